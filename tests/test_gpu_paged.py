"""GPU parity of attention over a paged cache (gdn_paged_attn_decode) against its fp64 oracle.

Tolerances, from the sizes the oracle returns (mass = softmax(z) |v|, reach = max scale |q| |k|):
a score's fp32 error is at most dz = 4 D 2^-24 reach (D products and the scale), so lse is off by
dz plus its own rounding, and o by 2 dz mass plus what the types round: with bf16 queries the
weights are held in no fewer bits than bf16 (8 significant bits: 2^-8 mass) and o is rounded to
bf16 (2^-8 |o|); with fp32 queries the sum over L tokens adds L 2^-24 mass."""
import numpy as np
import pytest
import torch

from oracle import decode

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build
    build.build()


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(lens, Hq, Hkv, D, page, cache=BF, seed=0, heads_first=False, dirty=True, extra=2):
    """Queries, caches (NaN wherever no sequence has a token) and the table (out-of-range page
    numbers past each sequence's pages)."""
    gen = torch.Generator().manual_seed(seed)
    used = [-(-x // page) for x in lens]
    pages = sum(used) + extra
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(lens), max(max(used), 1) + 1), -1, dtype=torch.int32)
    table[:, -1] = 1 << 30
    kc, vc = (torch.full((pages, page, Hkv, D), float("nan") if dirty else 0.0) for _ in range(2))
    at = 0
    for n, (length, u) in enumerate(zip(lens, used)):
        mine = order[at:at + u]
        at += u
        table[n, :u] = torch.tensor(mine, dtype=torch.int32)
        for i, pg in enumerate(mine):
            m = min(page, length - i * page)
            for c in (kc, vc):
                c[pg, :m] = torch.randn(m, Hkv, D, generator=gen)
    q = torch.randn(len(lens), Hq, D, generator=gen) * 2
    scales = [0.5 + torch.rand(Hkv, generator=gen) for _ in range(2)] if cache == FP8 else [None, None]
    act = F32 if cache == F32 else BF
    kc, vc = kc.to(cache), vc.to(cache)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    if heads_first:
        kd, vd = (c.transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in (kc.float(), vc.float()))
        kd, vd = (torch.empty_strided(c.shape, c.stride(), dtype=cache, device="cuda").copy_(c) for c in (kd, vd))
    else:
        kd, vd = kc.cuda(), vc.cuda()
    return dict(q=q.to(act).cuda(), k=kd, v=vd, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                ks=dev(scales[0]), vs=dev(scales[1]), D=D)


def check(x, o, lse, window=0, scale=None):
    D, scale = x["D"], scale or x["D"] ** -0.5
    val = lambda c: np64(c.float())  # noqa: E731
    ro, rl, mass, reach = decode.paged(np64(x["q"]), val(x["k"]), val(x["v"]), x["table"].cpu().numpy(), x["lens"].cpu().numpy(),
                                       scale, window, np64(x["ks"]), np64(x["vs"]))
    o, lse = np64(o), np64(lse)
    dz = 4 * D * 2.0 ** -24 * reach
    if x["q"].dtype == BF:
        tol = (2 * dz[..., None] + 2.0 ** -8) * mass + 2.0 ** -8 * np.abs(ro)
    else:
        tol = (2 * dz[..., None] + (64 + x["lens"].max().item()) * 2.0 ** -24) * mass
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= tol + 1e-30).all(), float((np.abs(o - ro) - tol).max())
    some = np.isfinite(rl)
    assert (np.isneginf(lse) == ~some).all()
    assert (np.abs(lse[some] - rl[some]) <= dz[some] + 2.0 ** -20 * (1 + np.abs(rl[some]))).all()


def call(x, **kw):
    from chunked_prefill_gb300 import gdn
    return gdn.paged_attention_decode(x["q"], x["k"], x["v"], x["table"], x["lens"], k_scale=x["ks"], v_scale=x["vs"], return_lse=True, **kw)


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page", [(1, 1, 1), (8, 1, 16), (6, 2, 7), (16, 16, 32), (40, 2, 48)])
def test_lengths_and_heads(cache, D, Hq, Hkv, page):
    """Empty, one token, page and tile edges, in every type, head width and grouping."""
    x = make([0, 1, 15, 16, 17, 33, 130], Hq, Hkv, D, page, cache, seed=Hq + page)
    check(x, *call(x))


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("lens", [[5000], [4097, 0, 1, 2047], [20011]])
def test_long_sequences_split_and_joined(cache, lens):
    x = make(lens, 4, 2, 128, 64, cache, seed=len(lens))
    check(x, *call(x))


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page,window", [(12, 1, 1, 0), (40, 1, 32, 0), (66, 2, 5, 700)])
def test_many_heads_to_one_on_long_sequences(cache, D, Hq, Hkv, page, window):
    """More query heads to a kv-head than a block of heads holds, split sequences, small pages."""
    x = make([9001, 0, 733, 2, 4000], Hq, Hkv, D, page, cache, seed=Hq + D)
    check(x, *call(x, window=window), window=window)


@pytest.mark.parametrize("cache", [BF, FP8])
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
def test_window(cache, window):
    """Tokens before the window hold NaN as well."""
    lens = [3000, 1, 0, 99, 100, 101]
    x = make(lens, 8, 2, 128, 16, cache, seed=window)
    for n, length in enumerate(lens):
        for t in range(max(0, length - window)):
            pg = int(x["table"][n, t // 16])
            for c in (x["k"], x["v"]):
                c.view(torch.uint8)[pg, t % 16] = 0x7F if cache == FP8 else 0xFF
    check(x, *call(x, window=window), window=window)


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (36, 2)])
def test_new_token_is_written_and_attended_to(cache, Hq, Hkv):
    """The caches get the rounded rows at len - 1 and nothing else; the result is that of a cache
    that held them already."""
    lens, D, page = [1, 16, 17, 2500, 0], 128, 16
    x = make(lens, Hq, Hkv, D, page, cache, seed=7, heads_first=True)
    act = x["q"].dtype
    kn, vn = (torch.randn(len(lens), Hkv, D, device="cuda").mul(3).to(act) for _ in range(2))
    kn[0, 0, 0] = 1000.0  # past the 8-bit range
    want = {}
    for name, new, sc in (("k", kn, x["ks"]), ("v", vn, x["vs"])):
        c = x[name].float().clone()
        row = new.float() / (1.0 if sc is None else sc[:, None])
        if cache == FP8:
            row = row.clamp(-448, 448)
        for n, length in enumerate(lens):
            if length:
                c[int(x["table"][n, (length - 1) // page]), (length - 1) % page] = row[n].to(cache).float()
                x[name].view(torch.uint8)[int(x["table"][n, (length - 1) // page]), (length - 1) % page] = 0x7F  # NaN, or large
        want[name] = c
    got = call(x, k_new=kn, v_new=vn)
    for name in ("k", "v"):
        a, b = x[name].float(), want[name]
        assert torch.equal(torch.nan_to_num(a, nan=-7.0), torch.nan_to_num(b, nan=-7.0)), name
    check(x, *got)
    again = call(x)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("cache", [BF, FP8, F32])
def test_layouts_and_strided_queries(cache):
    """Heads before tokens and heads after tokens give equal bits, and so do query rows inside a
    wider projection."""
    a = make([700, 3, 64], 8, 4, 128, 24, cache, seed=3)
    b = make([700, 3, 64], 8, 4, 128, 24, cache, seed=3, heads_first=True)
    ra, rb = call(a), call(b)
    assert torch.equal(ra[0], rb[0]) and torch.equal(ra[1], rb[1])
    wide = torch.randn(3, 10, 128, device="cuda").to(a["q"].dtype)
    wide[:, 2:] = a["q"]
    a["q"] = wide[:, 2:]
    rc = call(a)
    assert torch.equal(ra[0], rc[0]) and torch.equal(ra[1], rc[1])
    check(a, *ra)


def test_pages_out_of_range_are_masked_and_lengths_cut():
    """A page number past the cache masks its tokens; a length past the table is cut to it."""
    x = make([100, 64, 48], 4, 2, 128, 16, BF, seed=5)
    x["table"][0, 2] = 10 ** 6
    x["table"][1, :4] = -1  # nothing left
    x["table"][2, 3:] = -5
    x["lens"][2] = 10 ** 9
    check(x, *call(x))


def test_extreme_scores():
    """Scores of +-3000 (weights of 0 and 1), all scores equal, and a value row of large numbers."""
    x = make([300, 20], 2, 1, 128, 16, BF, seed=11)
    x["q"][0] *= 500
    x["q"][1] = 0
    x["v"].mul_(1e4)
    check(x, *call(x))


def test_cache_past_32_bit_offsets():
    from chunked_prefill_gb300 import gdn
    page, Hkv, D = 64, 8, 128
    pages = (2 ** 31) // (page * Hkv * D) + 3
    k, v = (torch.zeros(pages, page, Hkv, D, dtype=FP8, device="cuda") for _ in range(2))
    small = make([130], 16, Hkv, D, page, FP8, seed=2, extra=0)
    top = torch.tensor([[pages - 1, 1, pages - 2]], dtype=torch.int32, device="cuda")
    for i in range(3):
        for big, c in ((k, small["k"]), (v, small["v"])):
            big.view(torch.uint8)[int(top[0, i])] = c.view(torch.uint8)[int(small["table"][0, i])]
    o, lse = gdn.paged_attention_decode(small["q"], k, v, top, small["lens"], k_scale=small["ks"], v_scale=small["vs"], return_lse=True)
    check(small, o, lse)


def test_graph_other_stream_and_determinism():
    """A captured call replayed with other lengths."""
    from chunked_prefill_gb300 import gdn
    x = make([3000, 500], 8, 2, 128, 16, BF, seed=4)
    lse = torch.empty(2, 8, device="cuda")
    o = torch.empty_like(x["q"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run = lambda: gdn.gdn_paged_attn_decode(x["q"], x["k"], x["v"], x["table"], x["lens"], 0.1, o=o, lse=lse)  # noqa: E731
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            run()
        for lens in ([3000, 500], [1, 0], [1030, 499]):
            x["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            graph.replay()
            first = (o.clone(), lse.clone())
            graph.replay()
            st.synchronize()
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
            check(x, o, lse, scale=0.1)


def test_refusals():
    from chunked_prefill_gb300 import gdn
    x = make([5], 4, 2, 128, 16, BF)
    f = gdn.paged_attention_decode
    args = [x["q"], x["k"], x["v"], x["table"], x["lens"]]

    def refuses(i, t, err=ValueError, **kw):
        a = list(args)
        if i is not None:
            a[i] = t
        with pytest.raises(err):
            f(*a, **kw)

    refuses(0, x["q"].cpu())
    refuses(0, x["q"].transpose(1, 2).contiguous().transpose(1, 2))
    refuses(2, x["v"][:, :8])
    refuses(2, x["v"].float())
    refuses(3, x["table"].long())
    refuses(4, x["lens"].long())
    refuses(None, None, k_new=x["q"][:, :2])
    refuses(None, None, err=gdn.GdnError, scale=-1.0)
    refuses(None, None, err=gdn.GdnError, window=-1)
    refuses(0, x["q"][:, :3].contiguous(), err=gdn.GdnError)       # 3 query heads over 2
    refuses(0, x["q"].float(), err=gdn.GdnError)                   # fp32 queries, bf16 cache
    refuses(0, x["q"].half(), err=TypeError)
    with pytest.raises(gdn.GdnError):                              # D = 96
        f(x["q"][..., :96].contiguous(), x["k"][..., :96].contiguous(), x["v"][..., :96].contiguous(), *args[3:])
    with pytest.raises(RuntimeError, match="differentiable"):
        f(x["q"].clone().requires_grad_(True), *args[1:])


@pytest.mark.parametrize("cache", [BF, FP8, F32])
def test_one_large_weight_beside_many_small_ones(cache):
    """A first token that takes most of the weight, and thousands of others at e^-12 of it, whose
    values agree: their sum still counts."""
    L = 6000
    x = make([L], 2, 1, 128, 16, cache, seed=13)
    scale = 128 ** -0.5
    x["q"].fill_(1.0)
    pages = [int(p) for p in x["table"][0, :L // 16]]
    x["k"][pages] = torch.zeros(1, device="cuda").to(x["k"].dtype) if cache != FP8 else 0
    x["k"].view(torch.uint8)[pages[0], 0] = torch.full((1, 128), 12 * 128 ** 0.5 / 128, device="cuda").to(cache).view(torch.uint8)
    x["v"].view(torch.uint8)[pages] = torch.full((375, 16, 1, 128), 2.0, device="cuda").to(cache).view(torch.uint8)
    x["v"].view(torch.uint8)[pages[0], 0] = torch.full((1, 128), -1.0, device="cuda").to(cache).view(torch.uint8)
    if x["ks"] is not None:
        x["ks"].fill_(1.0)
        x["vs"].fill_(1.0)
    check(x, *call(x), scale=scale)


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_not_finite_rows_stay_where_they_are(cache, bad):
    """An infinite or NaN query row, and a NaN value row that is attended to, give NaN in their own
    heads alone."""
    x = make([200, 50, 2000], 8, 2, 128, 16, cache, seed=17)
    x["q"][1, 2, 5] = bad
    page = int(x["table"][0, 3])
    x["v"].view(torch.uint8)[page, 7, 1] = 0x7F if cache == FP8 else 0xFF
    o, lse = call(x)
    nan = torch.isnan(o).any(-1)
    want = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    want[1, 2] = True
    want[0, 4:] = True
    assert torch.equal(nan, want)


def test_many_sequences_and_many_heads():
    """More (sequence, kv-head) pairs than multiprocessors hold CTAs, split and unsplit."""
    gen = torch.Generator().manual_seed(1)
    for most in (3, 3000):
        lens = torch.randint(0, most + 1, (90,), generator=gen).tolist()
        lens[0] = most
        x = make(lens, 8, 8, 64, 32, BF, seed=most)
        check(x, *call(x))


def some_lens(N, most, seed):
    edges = [most, 0, 1, min(15, most), min(16, most), min(17, most), most - 1]
    gen = torch.Generator().manual_seed(seed)
    return (edges + torch.randint(0, most + 1, (N,), generator=gen).tolist())[:N]


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,page,window", [(1, 16, 0), (6, 7, 0), (16, 16, 20), (12, 5, 9), (20, 32, 0)])
def test_many_short_sequences(cache, D, G, page, window):
    """More pairs than multiprocessors hold CTAs, of few tokens each, empty ones among them."""
    N, Hkv = 154, 4
    x = make(some_lens(N, 50, D + G), G * Hkv, Hkv, D, page, cache, seed=G, heads_first=G == 6)
    check(x, *call(x, window=window), window=window)


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("D,N,Hkv,most", [(128, 1, 2, 900), (128, 20, 2, 900), (128, 60, 2, 700), (128, 100, 2, 400), (128, 160, 2, 600),
                                          (64, 7, 2, 1500), (64, 170, 3, 300), (256, 5, 3, 500), (256, 140, 3, 130)])
def test_every_division_of_short_caches(cache, D, N, Hkv, most):
    """One to eight CTAs to a (sequence, kv-head), of one warp and of several; the last CTAs of a
    sequence have nothing where it is short."""
    x = make(some_lens(N, most, N), 4 * Hkv, Hkv, D, 16, cache, seed=N)
    check(x, *call(x))
    live = torch.nonzero(x["lens"] > 0).flatten()
    kn, vn = (torch.randn(N, Hkv, D, device="cuda").to(x["q"].dtype) for _ in range(2))
    before = x["k"].float().clone(), x["v"].float().clone()
    got = call(x, k_new=kn, v_new=vn)
    check(x, *got)  # against the caches as they are now
    t = x["lens"][live].long() - 1
    pages = x["table"][live, t // 16].long()
    for c, b, new, sc in ((x["k"], before[0], kn, x["ks"]), (x["v"], before[1], vn, x["vs"])):
        row = new[live].float() / (1.0 if sc is None else sc[:, None])
        b[pages, t % 16] = row.to(cache).float()
        assert torch.equal(torch.nan_to_num(c.float(), nan=-7.0), torch.nan_to_num(b, nan=-7.0))


def test_a_new_token_past_the_table_is_not_written():
    x = make([48, 20], 4, 2, 128, 16, BF, seed=19)
    x["table"] = x["table"][:, :3].contiguous()
    x["table"][1, 2] = 0
    x["lens"][0] = 49  # the table holds 48
    k, v = x["k"].clone(), x["v"].clone()
    new = torch.randn(2, 2, 128, device="cuda").to(BF)
    got = call(x, k_new=new, v_new=new)
    at = (int(x["table"][1, 1]), 3)
    k[at], v[at] = new[1], new[1]
    for a, b in ((x["k"], k), (x["v"], v)):
        assert torch.equal(torch.nan_to_num(a, nan=-7.0), torch.nan_to_num(b, nan=-7.0))
    check(x, *got)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,cache,lift", [(8, FP8, 0), (8, FP8, 120), (16, FP8, 0), (16, FP8, 120), (8, BF, 0)])
def test_queries_of_the_smallest_sizes(D, Hq, cache, lift):
    """Query rows down to the smallest subnormal of bf16, zeros among their features; with scales of 2^lift
    their scores are of ordinary size and have to be as exact."""
    x = make([300, 20, 1], Hq, 1, D, 16, cache, seed=D + Hq)
    down = torch.tensor([-112, -118, -119, -120, -121, -126, -130, -133] * 2)[:Hq]
    q = torch.randn(3, Hq, D, generator=torch.Generator().manual_seed(5)).double() * 2.0 ** down.double()[:, None]
    q[:, :, ::3] = 0
    x["q"] = q.float().to(BF).cuda()
    if x["ks"] is not None:
        x["ks"] *= 2.0 ** lift
    check(x, *call(x))
