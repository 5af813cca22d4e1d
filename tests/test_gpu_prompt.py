"""GPU parity of attention over prompts (gdn_prompt_attn_fwd, _bwd) against its fp64 oracle.

Tolerances, from the sizes the oracle returns.  u = 2^-24; e = 2^-8 with bf16 (half a step of a rounding), 0 with fp32.
A score's fp32 error is at most dz = 4 D u reach.
  lse  dz and its own rounding.
  o    the weights are off by 2 dz and rounded by e, the sums over L keys by L u: (2 dz + e + (64 + L) u) mass; o is
       rounded: e |o| (u |o| in fp32, within the former).
  In the gradient p = e^{z - lse} is off by E = the largest 2 dz + 8 u (1 + |lse|) and rounded by e:
  dv   (E + e + L u) dv_mass, and e |dv|.
  dz   = p (do v - D), where the product is off by D u, D by the error of o as it was returned (e (mass + |o|) and the
       former's smaller terms) and D u: dq is off by (E + e + L u) dq_size + (e + E + (D + 64 + L) u) dq_o + D u dq_v,
       and e |dq|; dk likewise."""
import numpy as np
import pytest
import torch

from oracle import attention

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build, gdn
    build.build()
    return gdn


def np64(t):
    return t.detach().double().cpu().numpy()


def make(lens, Hq, Hkv, D, dtype=BF, seed=0, front=0, behind=0, fused=False, q_std=2.0):
    """Packed sequences of (queries, keys); rows in front of and behind them, and between the heads' rows of a fused
    projection, hold NaN."""
    gen = torch.Generator().manual_seed(seed)
    cu, cu_k = ([front + sum(x[i] for x in lens[:n]) for n in range(len(lens) + 1)] for i in (0, 1))
    shapes = dict(q=(cu[-1] + behind, Hq, q_std), k=(cu_k[-1] + behind, Hkv, 1.0), v=(cu_k[-1] + behind, Hkv, 1.0))
    x = {}
    width = (Hq + 2 * Hkv) * D + 24
    for name, (rows, heads, std) in shapes.items():
        end = cu[-1] if name == "q" else cu_k[-1]
        t = torch.full((rows, heads, D), float("nan"))
        t[front:end] = std * torch.randn(end - front, heads, D, generator=gen)
        t = t.to(dtype).cuda()
        if fused:
            wide = torch.full((rows, width), float("nan"), dtype=dtype, device="cuda")
            at = {"q": 0, "k": Hq * D + 8, "v": (Hq + Hkv) * D + 16}[name]
            wide[:, at:at + heads * D] = t.flatten(1)
            t = wide[:, at:at + heads * D].unflatten(1, (heads, D))
        x[name] = t[None]
    do = torch.full((1, cu[-1] + behind, Hq, D), float("nan"))
    do[:, front:cu[-1]] = torch.randn(1, cu[-1] - front, Hq, D, generator=gen)
    dlse = torch.full((1, cu[-1] + behind, Hq), float("nan"))
    dlse[:, front:cu[-1]] = torch.randn(1, cu[-1] - front, Hq, generator=gen)
    x.update(cu=cu, cu_k=cu_k, do=do.to(dtype).cuda(), dlse=dlse.cuda(), scale=D ** -0.5, lens=lens)
    x["cu_seqlens"], x["cu_seqlens_k"] = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu, cu_k))
    return x


def oracle(x, window=0, back=False, dlse=False):
    q, k, v = (np64(x[n])[0] for n in ("q", "k", "v"))
    return attention.prompt(q, k, v, x["cu"], x["cu_k"], x["scale"], window, np64(x["do"])[0] if back else None, np64(x["dlse"])[0] if dlse else None)


def near(name, got, want, tol, rows=slice(None)):
    got, want, tol = np64(got)[0][rows], want[rows], tol[rows]
    assert np.isfinite(got).all(), name
    over = np.abs(got - want) - tol - 1e-30
    assert (over <= 0).all(), (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


def sizes(x, r):
    D, L = x["q"].shape[-1], max([b for _, b in x["lens"]] + [1])
    return D, L, 2.0 ** -8 if x["q"].dtype == BF else 0.0, 4 * D * U * r["reach"]


def check_fwd(x, r, o, lse):
    D, L, e, dz = sizes(x, r)
    rows = slice(x["cu"][0], x["cu"][-1])
    near("o", o, r["o"], (2 * dz[..., None] + e + (64 + L) * U) * r["mass"] + e * np.abs(r["o"]), rows)
    lse, want = np64(lse)[0][rows], r["lse"][rows]
    some = np.isfinite(want)
    assert (np.isneginf(lse) == ~some).all()
    assert (np.abs(lse[some] - want[some]) <= dz[rows][some] + 2.0 ** -20 * (1 + np.abs(want[some]))).all()


def check_bwd(x, r, dq, dk, dv):
    D, L, e, dz = sizes(x, r)
    some = np.isfinite(r["lse"])
    E = float((2 * dz[some] + 8 * U * (1 + np.abs(r["lse"][some]))).max()) if some.any() else 0.0
    L = max([L] + [a for a, _ in x["lens"]]) * (x["q"].shape[2] // x["k"].shape[2])  # a key's sum is over the group's queries
    rows, keys = slice(x["cu"][0], x["cu"][-1]), slice(x["cu_k"][0], x["cu_k"][-1])
    near("dv", dv, r["dv"], (E + e + L * U) * r["dv_mass"] + max(e, U) * np.abs(r["dv"]), keys)
    for name, got, at in (("dq", dq, rows), ("dk", dk, keys)):
        tol = (E + e + L * U) * r[name + "_size"] + (e + E + (D + 64 + L) * U) * r[name + "_o"] + D * U * r[name + "_v"] + max(e, U) * np.abs(r[name])
        near(name, got, r[name], tol, at)


def args(x, keys=True):
    return dict(scale=x["scale"], cu_seqlens=x["cu_seqlens"], cu_seqlens_k=x["cu_seqlens_k"] if keys else None)


def run(gdn, x, window=0, dlse=False):
    o, lse = gdn.prompt_attention(x["q"], x["k"], x["v"], window=window, return_lse=True, **args(x))
    grads = gdn.gdn_prompt_attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], window=window, dlse=x["dlse"] if dlse else None, **args(x))
    return o, lse, grads


def check(gdn, x, window=0, dlse=False):
    r = oracle(x, window, True, dlse)
    o, lse, grads = run(gdn, x, window, dlse)
    check_fwd(x, r, o, lse)
    check_bwd(x, r, *grads)
    # rows that no sequence covers
    for t, fill, cu in ((o, 0.0, x["cu"]), (lse, -np.inf, x["cu"]), (grads[0], 0.0, x["cu"]), (grads[1], 0.0, x["cu_k"]), (grads[2], 0.0, x["cu_k"])):
        t = np64(t)[0]
        assert (t[:cu[0]] == fill).all() and (t[cu[-1]:] == fill).all()


EDGES = [(1, 1), (0, 0), (63, 63), (64, 64), (65, 65), (2, 2), (127, 127), (128, 128), (129, 129), (1, 300), (7, 3), (300, 1), (0, 5), (6, 0), (131, 260), (257, 257)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (8, 1)])
def test_lengths_and_heads(gdn, dtype, D, Hq, Hkv):
    """Sequences of every length around the tiles', with other numbers of keys, empty ones among them."""
    check(gdn, make(EDGES, Hq, Hkv, D, dtype, seed=Hq + D))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("front,behind", [(0, 0), (0, 300), (5, 0)])
def test_no_sequence_at_all(gdn, dtype, front, behind):
    """Offsets of one element: rows, but no sequence that covers them."""
    x = make([], 4, 2, 128, dtype, front=front, behind=behind)
    o, lse, grads = run(gdn, x)
    assert o.shape == x["q"].shape and (o == 0).all() and torch.isneginf(lse).all()
    for g, t in zip(grads, (x["q"], x["k"], x["v"])):
        assert g.shape == t.shape and (g == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 200, 1 << 30])
def test_window(gdn, dtype, window):
    check(gdn, make([(300, 300), (130, 400), (5, 2), (0, 3), (400, 130)], 4, 2, 64, dtype, seed=window % 97), window)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_a_fused_projection_among_others(gdn, dtype, D):
    """Views of a projection's rows, with NaN in every row and column that is not theirs."""
    check(gdn, make([(70, 70), (3, 3), (129, 129)], 4, 2, D, dtype, seed=3, front=5, behind=140, fused=True))


@pytest.mark.parametrize("dtype,D,lens", [(BF, 128, [(1500, 1500)]), (BF, 64, [(900, 2100), (1100, 1100)]), (BF, 256, [(700, 1300)]), (F32, 128, [(500, 900)])])
def test_many_tiles(gdn, dtype, D, lens):
    check(gdn, make(lens, 4, 2, D, dtype, seed=D), dlse=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_gradient_of_lse(gdn, dtype):
    check(gdn, make([(40, 40), (140, 200), (9, 4)], 4, 2, 128, dtype, seed=8), dlse=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("std", [1e-3, 30.0])
def test_flat_and_peaked_scores(gdn, dtype, std):
    """Nearly equal weights, and one that takes all, with the maximum anywhere."""
    check(gdn, make([(260, 260)], 2, 1, 128, dtype, seed=4, q_std=std))


def test_growing_scores(gdn):
    """Every tile's maximum far above the one before: the accumulator is rescaled each time."""
    x = make([(600, 600)], 2, 1, 64, seed=5)
    x["k"] = (x["k"].float() * torch.linspace(0.1, 8, 600, device="cuda")[None, :, None, None]).to(BF)
    check(gdn, x)


def test_shared_lengths_and_a_batch_of_equal_ones(gdn):
    """One cu_seqlens for queries and keys, and [B, T] without any, give what packed sequences do."""
    x = make([(150, 150)] * 3, 4, 2, 64, seed=6)
    o, lse, grads = run(gdn, x)
    again = gdn.prompt_attention(x["q"], x["k"], x["v"], return_lse=True, **args(x, False))
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    q, k, v, do = (x[n].view(3, 150, -1, 64) for n in ("q", "k", "v", "do"))
    ob, lb = gdn.prompt_attention(q, k, v, return_lse=True)
    assert torch.equal(ob.view_as(o), o) and torch.equal(lb.view_as(lse), lse)
    for a, b in zip(gdn.gdn_prompt_attn_bwd(q, k, v, ob, lb, do, x["scale"]), grads):
        assert torch.equal(a.view_as(b), b)
    part = gdn.prompt_attention(q[:, 100:].contiguous(), k, v)  # more keys than queries
    assert torch.equal(part, ob[:, 100:]) or torch.allclose(part.float(), ob[:, 100:].float(), atol=2 ** -6)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_value_reaches_only_those_who_see_it(gdn, dtype, D, value):
    """Infinite and NaN values: earlier queries of the same tile, and other sequences, are as without them."""
    x = make([(100, 100), (50, 60), (300, 300)], 2, 1, D, dtype, seed=7)
    o, lse = gdn.prompt_attention(x["q"], x["k"], x["v"], return_lse=True, **args(x))
    v = x["v"].clone()
    bad = [(0, 37), (1, 59), (2, 130)]  # sequence, key
    for n, t in bad:
        v[0, x["cu_k"][n] + t, 0, 5] = value
    ob, lb = gdn.prompt_attention(x["q"], x["k"], v, return_lse=True, **args(x))
    assert torch.equal(lb, lse)
    for n, t in bad:
        lq, lk = x["lens"][n]
        rows = slice(x["cu"][n], x["cu"][n + 1])
        sees = torch.arange(lq, device="cuda") + lk - lq >= t
        a, b = ob[0, rows], o[0, rows]
        assert torch.equal(a[~sees], b[~sees])
        assert torch.equal(a[..., :5], b[..., :5]) and torch.equal(a[..., 6:], b[..., 6:])
        hit = a[sees][..., 5]
        assert not torch.isfinite(hit).any()


def test_bad_queries_and_keys_stay_in_their_rows(gdn):
    x = make([(100, 100), (130, 130)], 2, 1, 64, seed=9)
    o, lse = gdn.prompt_attention(x["q"], x["k"], x["v"], return_lse=True, **args(x))
    q, k = x["q"].clone(), x["k"].clone()
    q[0, 20, 1, 3] = float("nan")
    k[0, 100 + 70, 0, 2] = float("inf")
    ob, lb = gdn.prompt_attention(q, k, x["v"], return_lse=True, **args(x))
    touched = torch.zeros(230, 2, dtype=torch.bool, device="cuda")
    touched[20, 1] = True
    touched[170:] = True
    assert torch.equal(ob[0][~touched], o[0][~touched]) and torch.equal(lb[0][~touched], lse[0][~touched])
    assert torch.isnan(ob[0, 20, 1]).all() and torch.isnan(lb[0, 20, 1])


def test_a_given_output_keeps_what_no_sequence_covers(gdn):
    x = make([(30, 30)], 2, 1, 64, front=3, behind=9)
    want, wl = gdn.prompt_attention(x["q"], x["k"], x["v"], return_lse=True, **args(x))
    o, lse = torch.full_like(want, 7.0), torch.full_like(wl, 5.0)
    got = gdn.gdn_prompt_attn_fwd(x["q"], x["k"], x["v"], o=o, lse=lse, **args(x))
    assert got.data_ptr() == o.data_ptr()
    assert (o[0, :3] == 7).all() and (o[0, 33:] == 7).all() and (lse[0, :3] == 5).all() and (lse[0, 33:] == 5).all()
    assert torch.equal(o[0, 3:33], want[0, 3:33]) and torch.equal(lse[0, 3:33], wl[0, 3:33])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_autograd(gdn, dtype):
    """prompt_attention's gradients are gdn_prompt_attn_bwd's, with either output used or not."""
    x = make([(50, 50), (77, 140)], 4, 2, 64, dtype, seed=2)
    leaves = [x[n].clone().requires_grad_(True) for n in ("q", "k", "v")]
    o, lse = gdn.prompt_attention(*leaves, return_lse=True, **args(x))
    got = torch.autograd.grad((o, lse), leaves, (x["do"], x["dlse"]), retain_graph=True)
    raw = [t.detach() for t in leaves]
    again, _, rest = gdn.gdn_prompt_attn_fwd(*raw, lse=True, rest=True, **args(x))
    assert torch.equal(again, o) and (rest is None) == (dtype == F32)
    if rest is not None:  # o and its rest are o to 16 bits
        r = oracle(dict(x, **dict(zip("qkv", raw))))
        assert (rest.float().abs() <= 2.0 ** -8 * o.float().abs()).all()
        _, L, _, dz = sizes(x, r)
        near("o + rest", o.float() + rest.float(), r["o"], (2 * dz[..., None] + 2.0 ** -8 + (64 + L) * U) * r["mass"] + 2.0 ** -16 * np.abs(r["o"]))
    for a, b in zip(got, gdn.gdn_prompt_attn_bwd(*raw, o.detach(), lse.detach(), x["do"], dlse=x["dlse"], o_rest=rest, **args(x))):
        assert torch.equal(a, b)
    only_o = torch.autograd.grad(o, leaves, x["do"], retain_graph=True)
    for a, b in zip(only_o, gdn.gdn_prompt_attn_bwd(*raw, o.detach(), lse.detach(), x["do"], o_rest=rest, **args(x))):
        assert torch.equal(a, b)
    only_lse = torch.autograd.grad(lse, leaves, x["dlse"])
    for a, b in zip(only_lse, gdn.gdn_prompt_attn_bwd(*raw, o.detach(), lse.detach(), torch.zeros_like(o), dlse=x["dlse"], o_rest=rest, **args(x))):
        assert torch.equal(a, b)


def test_the_gradient_is_the_difference(gdn):
    """fp32, along a random direction, against central differences of the oracle's loss in fp64: what is left is the
    fp32 error of the gradient, some L u of its terms' sum."""
    x = make([(40, 40), (20, 33)], 2, 1, 64, F32, seed=12)
    grads = run(gdn, x)[2]
    gen = torch.Generator().manual_seed(1)
    for name, g in zip(("q", "k", "v"), grads):
        step = torch.randn(x[name].shape, generator=gen).double().cuda()

        def loss(s):
            y = dict(x, **{name: x[name].double() + s * 1e-4 * step})
            return float((oracle(y)["o"] * np64(x["do"])[0]).sum())

        diff, dot = (loss(1) - loss(-1)) / 2e-4, float((g.double() * step).sum())
        assert abs(diff - dot) <= 1e-5 * float((g.double() * step).abs().sum()), name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_repeated_calls_give_the_same_bits(gdn, dtype):
    x = make([(200, 260), (90, 90)], 8, 2, 128, dtype, seed=3)
    first = run(gdn, x)
    for _ in range(3):
        again = run(gdn, x)
        assert torch.equal(again[0], first[0]) and all(torch.equal(a, b) for a, b in zip(again[2], first[2]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_captured_calls_serve_other_lengths(gdn, dtype):
    x = make([(100, 100), (56, 56), (44, 44)], 4, 2, 64, dtype, seed=1)
    y = make([(3, 3), (150, 150), (40, 40)], 4, 2, 64, dtype, seed=2, behind=7)
    y["cu_seqlens_k"] = y["cu_seqlens"]
    bufs = {n: x[n].clone() for n in ("q", "k", "v", "do", "cu_seqlens")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        a = dict(scale=x["scale"], cu_seqlens=bufs["cu_seqlens"])
        o, lse = gdn.prompt_attention(bufs["q"], bufs["k"], bufs["v"], return_lse=True, **a)
        return o, lse, gdn.gdn_prompt_attn_bwd(bufs["q"], bufs["k"], bufs["v"], o, lse, bufs["do"], **a)

    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call()
    torch.cuda.current_stream().wait_stream(side)
    for z in (y, x):
        for n in bufs:
            bufs[n].copy_(z[n])
        graph.replay()
        torch.cuda.synchronize()
        r = oracle(z, 0, True)
        check_fwd(z, r, out[0], out[1])
        check_bwd(z, r, *out[2])


def test_captured_forward_and_gradient(gdn):
    """Autograd's own forward and backward in a graph, of leaves that were made for it."""
    x, y = (make([(190, 190), (66, 66)], 4, 2, 64, seed=s) for s in (1, 2))
    leaves = [x[n].clone().requires_grad_(True) for n in ("q", "k", "v")]
    do, cu = x["do"].clone(), x["cu_seqlens"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        o, lse = gdn.prompt_attention(*leaves, scale=x["scale"], cu_seqlens=cu, return_lse=True)
        return o, lse, torch.autograd.grad(o, leaves, do)

    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o, lse, grads = step()
    torch.cuda.current_stream().wait_stream(side)
    for z in (y, x):
        with torch.no_grad():
            for t, n in zip(leaves, ("q", "k", "v")):
                t.copy_(z[n])
        do.copy_(z["do"])
        graph.replay()
        torch.cuda.synchronize()
        r = oracle(z, 0, True)
        check_fwd(z, r, o, lse)
        check_bwd(z, r, *grads)


def test_a_gradient_that_begins_anywhere(gdn):
    """The gradient of a concatenation of flat tensors is a view at any offset."""
    x = make([(70, 70)], 2, 2, 64)
    grads = []
    for odd in (0, 3):
        leaf = x["v"].clone().requires_grad_(True)
        o = gdn.prompt_attention(x["q"], x["k"], leaf)
        w = torch.cat([x["do"].new_zeros(odd), x["do"].flatten()])
        (torch.cat([o.new_zeros(odd), o.flatten()]) * w).sum().backward()
        grads.append(leaf.grad)
    assert torch.equal(*grads)


def test_two_calls_at_once(gdn):
    """Calls on two streams, and two captured graphs with a workspace each, replayed together."""
    xs = [make([(900, 900), (300, 500)], 4, 2, 128, seed=s) for s in (1, 2)]
    want = [run(gdn, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]

    def same(got):
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1]) and all(torch.equal(a, b) for a, b in zip(g[2], w[2]))

    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                outs.append(run(gdn, x))
        same(outs)
    graphs, outs = [], []
    for x, st in zip(xs, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=st):
            outs.append(run(gdn, x))
    for _ in range(5):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        same(outs)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graphs_that_share_a_workspace(gdn, dtype):
    """Two captured gradients over one workspace, whatever it held before, replayed one after the other."""
    xs = [make([(300, 300), (40, 90)], 8, 2, 64, dtype, seed=s, behind=9) for s in (1, 2)]
    fwd = [gdn.prompt_attention(x["q"], x["k"], x["v"], return_lse=True, **args(x)) for x in xs]
    grad = lambda x, f, **kw: gdn.gdn_prompt_attn_bwd(x["q"], x["k"], x["v"], *f, x["do"], **args(x), **kw)  # noqa: E731
    want = [grad(x, f) for x, f in zip(xs, fwd)]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x, f in zip(xs, fwd):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                outs.append(grad(x, f, workspace=ws))
        for graph in graphs * 2:
            graph.replay()
    side.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(outs, want) for a, b in zip(g, w))


def test_on_another_stream(gdn):
    x = make([(300, 300)], 4, 2, 128, seed=4)
    want = run(gdn, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(gdn, x)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(got[2], want[2]))


def test_broadcast_leaves_sum_their_gradients(gdn):
    """A key shared by a batch, made whole before the call: autograd sums over its copies."""
    x = make([(60, 60)], 2, 1, 64, F32, seed=5)
    q = torch.cat([x["q"], x["q"] * 0.5])
    k = x["k"].clone().requires_grad_(True)
    v = torch.cat([x["v"], x["v"]])
    gdn.prompt_attention(q, k.expand(2, -1, -1, -1).contiguous(), v).sum().backward()
    parts = []
    for b in range(2):
        leaf = x["k"].clone().requires_grad_(True)
        gdn.prompt_attention(q[b:b + 1], leaf, v[b:b + 1]).sum().backward()
        parts.append(leaf.grad)
    assert torch.allclose(k.grad, parts[0] + parts[1], rtol=1e-6, atol=1e-6)


def test_no_wait_gave_up(gdn):
    run(gdn, make([(200, 300), (77, 77)], 4, 2, 128))
    assert gdn.gdn_attn_device_status() == gdn.GDN_OK
