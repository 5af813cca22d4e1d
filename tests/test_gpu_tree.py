"""GPU parity of attention of drafted trees over a paged cache (gdn_paged_attn_tree) against its fp64 oracle.

Tolerances as in the tests of one new token: dz = 4 D 2^-24 reach for a score, so lse is off by dz plus its rounding, o by
2 dz mass plus what the types round: with bf16 queries the weights (2^-8 mass; under scales of the cache's values once more,
for the weight is multiplied by the scale before it is rounded: 2^-24 mass) and o (2^-8 |o|); sums over L tokens add L 2^-24 mass."""
import numpy as np
import pytest
import torch

from oracle import attention

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build, gdn
    build.build()
    return gdn


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def random_tree(rng, T, live=None):
    live = T if live is None else live
    return [int(rng.choice([t - 1, rng.integers(max(-1, t - 5), t)])) for t in range(live)] + [-2] * (T - live)


def make(lens, T, Hq, Hkv, D, page, cache=BF, seed=0, heads_first=False, trees=None, extra=2):
    """Caches hold NaN wherever no sequence has a token; the table out-of-range pages past each sequence's."""
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    used = [-(-x // page) for x in lens]
    pages = sum(used) + extra
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(lens), max(max(used), 1) + 1), -1, dtype=torch.int32)
    table[:, -1] = 1 << 30
    kc, vc = (torch.full((pages, page, Hkv, D), float("nan")) for _ in range(2))
    at = 0
    for n, (length, u) in enumerate(zip(lens, used)):
        mine = order[at:at + u]
        at += u
        table[n, :u] = torch.tensor(mine, dtype=torch.int32)
        for i, pg in enumerate(mine):
            m = min(page, length - i * page)
            for c in (kc, vc):
                c[pg, :m] = torch.randn(m, Hkv, D, generator=gen)
    act = F32 if cache == F32 else BF
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    kc, vc = kc.to(cache), vc.to(cache)
    if heads_first:
        kc, vc = (torch.empty_strided(c.shape, (page * Hkv * D, D, page * D, 1), dtype=cache, device="cuda").copy_(c) for c in (kc, vc))
    if trees is None:
        trees = [random_tree(rng, T, int(rng.integers(1, T + 1)) if n % 2 else T) for n in range(len(lens))]
    x = dict(q=(2 * rnd(len(lens), T, Hq, D)).to(act), kn=rnd(len(lens), T, Hkv, D).to(act), vn=rnd(len(lens), T, Hkv, D).to(act), k=kc, v=vc, table=table,
             lens=torch.tensor(lens, dtype=torch.int32), parents=torch.tensor(trees, dtype=torch.int32).view(len(lens), T))
    for name in ("ks", "vs"):
        x[name] = 0.5 + torch.rand(Hkv, generator=gen) if cache == FP8 else None
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def call(gdn, x, **kw):
    return gdn.paged_attention_tree(x["q"], x["kn"], x["vn"], x["k"], x["v"], x["table"], x["lens"], x["parents"], k_scale=x["ks"], v_scale=x["vs"], return_lse=True, **kw)


def check(x, o, lse, window=0):
    D = x["q"].shape[-1]
    ro, rl, mass, reach = attention.tree(np64(x["q"]), np64(x["kn"]), np64(x["vn"]), np64(x["k"].float()), np64(x["v"].float()), x["table"].cpu().numpy(),
                                         x["lens"].cpu().numpy(), x["parents"].cpu().numpy(), D ** -0.5, window, np64(x["ks"]), np64(x["vs"]))
    o, lse = np64(o), np64(lse)
    dz = 4 * D * 2.0 ** -24 * reach
    L = int(x["lens"].max()) + 64 if x["lens"].numel() else 64
    e = 2.0 ** -8 if x["q"].dtype == BF else 0.0
    tol = (2 * dz[..., None] + e + (64 + L) * 2.0 ** -24) * mass + e * np.abs(ro)
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= tol + 1e-30).all(), float((np.abs(o - ro) - tol).max())
    some = np.isfinite(rl)
    assert (np.isneginf(lse) == ~some).all()
    assert (np.abs(lse[some] - rl[some]) <= dz[some] + 2.0 ** -20 * (1 + np.abs(rl[some]))).all()


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page,T", [(1, 1, 1, 1), (8, 1, 16, 5), (6, 2, 7, 33), (4, 4, 32, 64), (40, 2, 48, 9)])
def test_lengths_and_heads(gdn, cache, D, Hq, Hkv, page, T):
    """Empty, one token, page and tile edges, blocks of rows that end inside a drafted token's heads."""
    x = make([0, 1, 15, 16, 65, 130], T, Hq, Hkv, D, page, cache, seed=Hq + page)
    check(x, *call(gdn, x))


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("lens", [[5000], [4097, 0, 1, 2047], [12011]])
def test_long_sequences_split_and_joined(gdn, cache, lens):
    x = make(lens, 6, 4, 2, 128, 64, cache, seed=len(lens))
    check(x, *call(gdn, x))


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("window", [1, 2, 3, 16, 100, 5000])
def test_window(gdn, cache, window):
    """Also shorter than the tree is deep."""
    x = make([1500, 1, 0, 99, 100, 101], 7, 4, 2, 64, 16, cache, seed=window, trees=[list(range(-1, 6))] * 3 + [[-1, 0, 1, 1, 3, -1, 5]] * 3)
    check(x, *call(gdn, x, window=window), window=window)


@pytest.mark.parametrize("cache", [BF, FP8])
@pytest.mark.parametrize("page", [5, 16, 48])
def test_heads_before_tokens(gdn, cache, page):
    x = make([300, 77, 0, 18], 11, 16, 4, 128, page, cache, seed=page, heads_first=True)
    check(x, *call(gdn, x))


@pytest.mark.parametrize("cache", [BF, FP8, F32])
def test_many_uneven_sequences(gdn, cache):
    rng = np.random.default_rng(3)
    x = make(rng.integers(0, 400, 40).tolist(), 4, 8, 2, 64, 16, cache, seed=9)
    check(x, *call(gdn, x))


@pytest.mark.parametrize("cache", [BF, F32])
def test_no_such_tokens(gdn, cache):
    """Parents that are no earlier token, whole sequences without a tree, and followers of missing tokens."""
    trees = [[-2, 0, -1, 2], [-2, -2, -2, -2], [0, 1, 5, 100], [-1, 0, 3, 2], [-(1 << 31), (1 << 31) - 1, -1, 1]]
    x = make([40, 30, 20, 0, 10], 4, 4, 2, 64, 16, cache, seed=4, trees=trees)
    for name in ("q", "kn", "vn"):  # what lies in the rows of missing tokens is not used
        for n, line in enumerate(trees):
            for t, seen in enumerate(attention.ancestors(line)):
                if seen is None:
                    x[name][n, t] = float("nan")
    keep = {n: x[n].clone() for n in ("q", "kn", "vn")}
    o, lse = call(gdn, x)
    for n in keep:
        x[n] = torch.nan_to_num(x[n])
    check(x, o, lse)


@pytest.mark.parametrize("cache", [BF, F32])
def test_a_bad_value_reaches_only_those_who_see_it(gdn, cache):
    """NaN and infinities in a drafted token's value: other branches are as without it."""
    x = make([50], 6, 4, 2, 64, 16, cache, seed=5, trees=[[-1, 0, 0, 1, 2, -1]])
    o, lse = call(gdn, x)
    for value in (float("nan"), float("inf")):
        y = dict(x, vn=x["vn"].clone())
        y["vn"][0, 1, 0, 7] = value
        ob, lb = call(gdn, y)
        assert torch.equal(lb, lse)
        sees = torch.tensor([1, 3], device="cuda")
        others = torch.tensor([0, 2, 4, 5], device="cuda")
        assert torch.equal(ob[0, others], o[0, others]) and torch.equal(ob[0, :, 2:], o[0, :, 2:])
        assert not torch.isfinite(ob[0, sees][:, :2, 7]).any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_8_bit_value(gdn, D):
    """A cached token that takes all the weight: its value comes back as it is, each of the 256."""
    every = torch.arange(256, dtype=torch.uint8, device="cuda").view(FP8)
    N = 256 // min(D, 256)
    v = every.view(torch.uint8).view(N, 1, 1, D).expand(N, 4, 1, D).contiguous().view(FP8)
    k = torch.full((N, 4, 1, D), 8.0, device="cuda").to(FP8)
    q = torch.full((N, 1, 1, D), 8.0, device="cuda", dtype=BF)
    table = torch.arange(N, dtype=torch.int32, device="cuda").view(N, 1)
    one = torch.ones(N, dtype=torch.int32, device="cuda")
    o = gdn.paged_attention_tree(q, -q, torch.ones_like(q), k, v, table, one, one[:, None] * -1)  # the drafted token's weight: 0
    want = every.float()
    got = o.float().flatten()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


@pytest.mark.parametrize("factor", [0.0, -1.0])
def test_scales_that_are_zero_or_negative(gdn, factor):
    x = make([300, 5, 0], 4, 4, 2, 64, 16, FP8, seed=11)
    x["ks"] = x["ks"] * factor
    x["vs"] = x["vs"] * factor
    check(x, *call(gdn, x))


def test_pages_out_of_range_and_long_lengths(gdn):
    x = make([100, 100, 64], 3, 4, 2, 64, 16, seed=6)
    x["table"][0, 2] = -1
    x["table"][1, 1] = 1 << 29
    x["table"] = x["table"][:, :4].contiguous()  # lengths past the table's 64 tokens
    check(x, *call(gdn, x))


def test_a_chain_is_one_token_after_another(gdn):
    """Drafted in a chain, then written to the cache: decoding each gives the same attention."""
    x = make([37, 5, 60], 4, 8, 2, 64, 16, seed=7, trees=[[-1, 0, 1, 2]] * 3)
    pages = torch.arange(3 * 6, dtype=torch.int32, device="cuda").view(3, 6)
    k, v = (torch.randn(18, 16, 2, 64, device="cuda").to(BF) for _ in range(2))
    lens = x["lens"]
    o, lse = gdn.paged_attention_tree(x["q"], x["kn"], x["vn"], k, v, pages, lens, x["parents"], return_lse=True)
    for t in range(4):
        a, l = gdn.paged_attention_decode(x["q"][:, t].contiguous(), k, v, pages, lens + t + 1, k_new=x["kn"][:, t].contiguous(), v_new=x["vn"][:, t].contiguous(), return_lse=True)
        assert (lse[:, t] - l).abs().max() <= 1e-4 and (o[:, t].float() - a.float()).abs().max() <= 2.0 ** -6 * a.float().abs().max()


@pytest.mark.parametrize("cache", [BF, FP8, F32])
def test_captured_call_serves_other_lengths_and_trees(gdn, cache):
    x = make([200, 3], 5, 4, 2, 64, 16, cache, seed=1, extra=20)
    y = make([7, 150], 5, 4, 2, 64, 16, cache, seed=2, extra=23)
    wide = max(x["table"].shape[1], y["table"].shape[1])
    for z in (x, y):
        z["table"] = torch.nn.functional.pad(z["table"], (0, wide - z["table"].shape[1]), value=-1)
    pages = max(x["k"].shape[0], y["k"].shape[0])
    bufs = {n: None if t is None else torch.empty((pages, *t.shape[1:]) if n in "kv" else t.shape, dtype=t.dtype, device="cuda") for n, t in x.items()}

    def fill(z):
        for n, t in z.items():
            if t is not None:
                bufs[n][:t.shape[0]].copy_(t)

    fill(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(gdn, bufs)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call(gdn, bufs)
    torch.cuda.current_stream().wait_stream(side)
    for z in (y, x):
        fill(z)
        graph.replay()
        torch.cuda.synchronize()
        check(z, *out)


def test_repeated_calls_and_workspaces_give_the_same_bits(gdn):
    x = make([3000, 100, 0, 700], 8, 8, 2, 128, 16, seed=3)
    o, lse = call(gdn, x)
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again = call(gdn, x, workspace=ws)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_two_calls_at_once(gdn):
    """On two streams, and as two captured graphs that share a workspace and run one after the other."""
    xs = [make([3000, 40, 900], 9, 8, 2, 128, 16, seed=s) for s in (1, 2)]
    want = [call(gdn, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                outs.append(call(gdn, x))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(outs, want) for a, b in zip(g, w))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=streams[0]):
            outs.append(call(gdn, x, workspace=ws))
    with torch.cuda.stream(streams[0]):
        for graph in graphs * 3:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(outs, want) for a, b in zip(g, w))


def test_long_offsets(gdn):
    """Pages whose offsets pass 32 bits of elements."""
    pages, page, Hkv, D = (1 << 31) // (64 * 128) + 40, 64, 1, 128
    k = torch.empty(pages, page, Hkv, D, dtype=FP8, device="cuda")
    v = torch.empty_like(k)
    small = make([150], 3, 4, Hkv, D, page, FP8, seed=8)
    far = torch.tensor([[pages - 1, pages - 7, 2]], dtype=torch.int32, device="cuda")
    for big, name in ((k, "k"), (v, "v")):
        big.view(torch.uint8)[far[0].long()] = small[name].view(torch.uint8)[small["table"][0, :3].long()]
    want = call(gdn, small)
    got = call(gdn, dict(small, k=k, v=v, table=far))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_wait_gave_up(gdn):
    for cache in (BF, FP8):
        call(gdn, make([500, 0, 77], 9, 8, 2, 128, 16, cache))
    assert gdn.gdn_attn_device_status() == gdn.GDN_OK
