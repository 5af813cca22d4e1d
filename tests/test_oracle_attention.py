"""The attention oracles against differences and against each other (CPU)."""
import numpy as np
import pytest

from oracle import attention, decode


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("window", [0, 3])
@pytest.mark.parametrize("lens", [[(5, 5)], [(4, 9), (0, 3), (6, 2), (3, 3)]])
def test_prompt_gradient_is_the_difference(lens, window):
    cu, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(int) for x in zip(*lens))
    q, k, v = rnd(1, cu[-1], 4, 8), rnd(2, cu_k[-1], 2, 8), rnd(3, cu_k[-1], 2, 8)
    do, dlse = rnd(4, *q.shape), rnd(5, cu[-1], 4)
    f = lambda a, b, c: attention.prompt(a, b, c, cu, cu_k, 0.3, window)  # noqa: E731

    def loss(a, b, c):
        r = f(a, b, c)
        some = np.isfinite(r["lse"])
        return (r["o"] * do).sum() + (r["lse"][some] * dlse[some]).sum()

    got = attention.prompt(q, k, v, cu, cu_k, 0.3, window, do, dlse)
    eps = 1e-5  # differences are off by eps^2 f''' / 6 and 2^-52 |loss| / eps: some 1e-9
    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        for seed in range(3):
            step = rnd(10 + seed, *(q, k, v)[i].shape)
            up, down = ([x + (s * eps * step if n == i else 0) for n, x in enumerate((q, k, v))] for s in (1, -1))
            assert abs((loss(*up) - loss(*down)) / (2 * eps) - (got[name] * step).sum()) < 1e-7


def test_a_query_sees_its_own_key_and_earlier_ones():
    q, k, v = rnd(1, 4, 1, 8), rnd(2, 4, 1, 8), rnd(3, 4, 1, 8)
    r = attention.prompt(q, k, v, [0, 4], [0, 4], 1.0)
    assert np.allclose(r["o"][0], v[0]) and np.allclose(r["lse"][0, 0], q[0, 0] @ k[0, 0])
    v[3] += 100
    again = attention.prompt(q, k, v, [0, 4], [0, 4], 1.0)
    assert np.array_equal(again["o"][:3], r["o"][:3]) and not np.allclose(again["o"][3], r["o"][3])


@pytest.mark.parametrize("window", [0, 4, 9])
def test_a_chain_is_one_token_after_another(window):
    """A tree that is a chain is decoding: each token of it as the new one over a cache with those before it."""
    N, T, Hq, Hkv, D, ps = 2, 5, 4, 2, 8, 3
    lens = np.array([7, 0])
    table = np.arange(8).reshape(2, 4)
    kc, vc, kn, vn, q = rnd(1, 8, ps, Hkv, D), rnd(2, 8, ps, Hkv, D), rnd(3, N, T, Hkv, D), rnd(4, N, T, Hkv, D), rnd(5, N, T, Hq, D)
    parents = np.tile(np.arange(-1, T - 1), (N, 1))
    o, lse, _, _ = attention.tree(q, kn, vn, kc, vc, table, lens, parents, 0.4, window)
    kf, vf = kc.copy(), vc.copy()
    for t in range(T):
        for n in range(N):
            at = lens[n] + t
            kf[table[n, at // ps], at % ps], vf[table[n, at // ps], at % ps] = kn[n, t], vn[n, t]
        want = decode.paged(q[:, t], kf, vf, table, lens + t + 1, 0.4, window)
        assert np.allclose(o[:, t], want[0]) and np.allclose(lse[:, t], want[1])


def test_branches_do_not_see_one_another():
    assert attention.ancestors([-1, 0, 0, 2, -1]) == [[0], [1, 0], [2, 0], [3, 2, 0], [4]]
    assert attention.ancestors([-2, 0, -1, 3, 2]) == [None, None, [2], None, [4, 2]]


def test_trim_undoes_extend():
    rng = np.random.default_rng(0)
    for _ in range(50):
        page, N = int(rng.integers(1, 6)), int(rng.integers(1, 6))
        lens = rng.integers(0, 12, N).tolist()
        table = np.full((N, 12), -1)
        at = 0
        for n, x in enumerate(lens):
            u = -(-x // page)
            table[n, :min(u, 12)] = np.arange(at, at + u)[:12]
            at += u
        stack = list(range(at, at + 20))
        free = int(rng.integers(0, 20))
        new = rng.integers(0, 15, N).tolist()
        t2, l2, f2, slots, cu = attention.extend(table.tolist(), lens, new, stack, free, page, sum(new))
        live = [s for s in slots if s >= 0]
        assert len(set(live)) == len(live) and cu[-1] == sum(new)
        l3, s3, f3 = attention.trim(t2, l2, lens, stack, f2, page)
        width = 12 * page
        assert l3 == [min(x, width) for x in lens] and s3 == stack and f3 == free
