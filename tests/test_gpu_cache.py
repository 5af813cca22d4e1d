"""The paged cache's own operators on the GPU: writing keys and values (gdn_paged_cache_write), page tables
(gdn_page_table_extend, _trim), and a run of them with the attention over prompts, trees and single tokens."""
import numpy as np
import pytest
import torch

from oracle import attention

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build, gdn
    build.build()
    return gdn


def caches(pages, page, Hkv, D, dtype, heads_first, gen):
    shape = (pages, Hkv, page, D) if heads_first else (pages, page, Hkv, D)
    c = [torch.randn(shape, generator=gen).to(dtype).cuda() for _ in range(2)]
    return [x.transpose(1, 2) for x in c] if heads_first else c


def bits(x):
    return x.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


@pytest.mark.parametrize("dtype", [BF, FP8, F32])
@pytest.mark.parametrize("Hkv,D,page,heads_first", [(1, 16, 1, False), (2, 64, 7, False), (8, 128, 16, True), (3, 256, 48, False), (16, 256, 64, True)])
@pytest.mark.parametrize("count", [1, 5, 333])
@pytest.mark.parametrize("picked", [False, True])
def test_write(gdn, dtype, Hkv, D, page, heads_first, count, picked):
    """Every slot gets the correctly rounded quotient, every other one keeps its bits; slots and rows out of range
    are skipped."""
    gen = torch.Generator().manual_seed(count + D)
    pages = -(-count // page) + 3
    kc, vc = caches(pages, page, Hkv, D, dtype, heads_first, gen)
    act = F32 if dtype == F32 else BF
    rows_n = 2 * count + 3 if picked else count + 2
    wide = torch.full((rows_n, 2 * Hkv * D + 32), float("nan"), dtype=act)
    wide[:, :Hkv * D] = (300 * torch.randn(rows_n, Hkv * D, generator=gen)).to(act)
    wide[:, Hkv * D + 16:2 * Hkv * D + 16] = torch.randn(rows_n, Hkv * D, generator=gen).to(act)
    wide = wide.cuda()
    k, v = wide[:, :Hkv * D].unflatten(1, (Hkv, D)), wide[:, Hkv * D + 16:2 * Hkv * D + 16].unflatten(1, (Hkv, D))
    slots = torch.randperm(pages * page, generator=gen)[:count]
    bad = [-1, pages * page, -(1 << 40), 1 << 40]
    for i in range(2, count, 7):
        slots[i] = bad[i % 4]
    rows = torch.randint(0, rows_n, (count,), generator=gen, dtype=I32) if picked else None
    if picked and count > 4:
        rows[3], rows[4] = -1, rows_n
    scales = [0.5 + torch.rand(Hkv, generator=gen).cuda() for _ in range(2)] if dtype == FP8 else [None, None]
    want = []
    for c, x, s in ((kc, k, scales[0]), (vc, v, scales[1])):
        c = c.clone()
        at = torch.arange(count) if rows is None else rows.long()
        ok = (slots >= 0) & (slots < pages * page) & (at >= 0) & (at < rows_n)
        y = x[at[ok].cuda()].float()
        if s is not None:
            y = (y / s[:, None]).clamp(-448, 448)
        sl = slots[ok].cuda()
        c.view(torch.uint8)[sl // page, sl % page] = y.to(dtype).view(torch.uint8)
        want.append(c)
    gdn.paged_cache_write(k, v, kc, vc, slots.cuda(), rows=None if rows is None else rows.cuda(), k_scale=scales[0], v_scale=scales[1])
    assert torch.equal(bits(kc), bits(want[0])) and torch.equal(bits(vc), bits(want[1]))


@pytest.mark.parametrize("scaled", [False, True])
def test_write_of_special_values(gdn, scaled):
    x = torch.tensor([0.0, -0.0, float("nan"), float("inf"), -float("inf"), 1e30, -1e30, 2.0 ** -130, 2.0 ** -9, 448.0, 464.0, 465.0, 1.0, -3.0, 0.0625, 17.0], dtype=BF, device="cuda")
    k = x.view(1, 1, 16)
    s = torch.full((1,), 0.75, device="cuda") if scaled else None
    for dtype in (BF, FP8):
        kc, vc = (torch.zeros(1, 2, 1, 16, dtype=dtype, device="cuda") for _ in range(2))
        gdn.paged_cache_write(k, k, kc, vc, torch.tensor([1], device="cuda"), k_scale=s, v_scale=s)
        y = x.float() / 0.75 if scaled else x.float()
        want = (y.clamp(-448, 448) if dtype == FP8 else y).to(dtype).float()
        for c in (kc, vc):
            assert torch.equal(torch.nan_to_num(c[0, 1, 0].float(), nan=77.0, posinf=1e38, neginf=-1e38), torch.nan_to_num(want, nan=77.0, posinf=1e38, neginf=-1e38))
            assert (c[0, 0].float() == 0).all()


def test_write_agrees_with_the_decoding_step(gdn):
    """The same bits as paged_attention_decode writes for a new token."""
    gen = torch.Generator().manual_seed(1)
    for dtype in (BF, FP8, F32):
        act = F32 if dtype == F32 else BF
        kn, vn, q = (torch.randn(3, h, 64, generator=gen).to(act).cuda() for h in (2, 2, 4))
        ks, vs = (0.5 + torch.rand(2, generator=gen).cuda() for _ in range(2)) if dtype == FP8 else (None, None)
        table = torch.arange(12, dtype=I32, device="cuda").view(3, 4)
        lens = torch.tensor([5, 16, 33], dtype=I32, device="cuda")
        a, b = caches(12, 16, 2, 64, dtype, False, gen), None
        b = [c.clone() for c in a]
        gdn.paged_attention_decode(q, a[0], a[1], table, lens, k_new=kn, v_new=vn, k_scale=ks, v_scale=vs)
        at = (lens - 1).long()
        slots = table.long().gather(1, (at // 16)[:, None])[:, 0] * 16 + at % 16
        gdn.paged_cache_write(kn, vn, b[0], b[1], slots, k_scale=ks, v_scale=vs)
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(bits(a[1]), bits(b[1]))


def test_write_past_32_bit_offsets(gdn):
    page, Hkv, D = 64, 1, 128
    pages = (1 << 32) // (page * D) + 5
    kc, vc = (torch.empty(pages, page, Hkv, D, dtype=FP8, device="cuda") for _ in range(2))
    last = pages * page
    slots = torch.tensor([last - 1, 3, last - 64], device="cuda")
    k = torch.randn(3, Hkv, D, device="cuda").to(BF)
    gdn.paged_cache_write(k, -k, kc, vc, slots)
    flat_k, flat_v = kc.view(-1, D), vc.view(-1, D)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(bits(flat_k[s]), bits(k[i, 0].to(FP8))) and torch.equal(bits(flat_v[s]), bits((-k[i, 0]).to(FP8)))


# ------------------------------------------------------------------------------------ page tables
def state(rng, N, width, page, stack_size, spare):
    lens = rng.integers(0, width * page + 1, N)
    lens[rng.random(N) < 0.2] = 0
    pages = rng.permutation(int(sum(-(-lens // page))) + stack_size + spare)
    table = rng.integers(-5, 1 << 20, (N, width))
    at = 0
    for n in range(N):
        u = -(-int(lens[n]) // page)
        table[n, :u] = pages[at:at + u]
        at += u
    stack = pages[at:at + stack_size]
    return table, lens, stack


def dev(x):
    return torch.tensor(np.asarray(x), dtype=I32, device="cuda")


@pytest.mark.parametrize("N,width,page", [(1, 1, 1), (3, 4, 16), (40, 7, 5), (256, 9, 16), (1500, 3, 7), (8192, 2, 3)])
@pytest.mark.parametrize("most", [1, 9, 60])
@pytest.mark.parametrize("share", [0.0, 0.5, 2.0])
def test_extend_and_trim(gdn, N, width, page, most, share):
    """Every number, with as many free pages as a share of what the sequences ask for."""
    rng = np.random.default_rng(N * 31 + most)
    new = rng.integers(-2, most + 1, N)
    size = max(1, int(share * sum(max(0, x) for x in new) / page))
    table, lens, stack = state(rng, N, width, page, size, 3)
    free = int(rng.integers(0, size + 1)) if share < 1 else size
    if N > 2:
        lens[2] = -7          # counts as 0
        lens[1] = width * page + 11  # as the row's
    total = max(0, int(np.maximum(new, 0).sum()) + int(rng.integers(-3, 4)))
    want = attention.extend(table.tolist(), lens.tolist(), new.tolist(), stack.tolist(), free, page, total)
    t, l, s, f = torch.full((N, width + 2), 9, dtype=I32, device="cuda")[:, :width], dev(lens), dev(stack), dev([free])
    t.copy_(dev(table))
    slots, cu = gdn.page_table_extend(t, l, dev(new), s, f, page, total)
    got = [t.tolist(), l.tolist(), int(f), slots.tolist(), cu.tolist()]
    assert got[4] == want[4] and got[2] == want[2] and got[0] == want[0] and got[3] == want[3]
    granted = [b if b != a else int(x) for a, b, x in zip(lens, want[1], l.tolist())]
    assert granted == l.tolist()
    assert s.tolist() == stack.tolist()
    # cut to anything, and everything given up
    for keep in (rng.integers(-1, width * page + 1, N), np.zeros(N, int)):
        want = attention.trim(t.tolist(), l.tolist(), keep.tolist(), s.tolist(), int(f), page)
        gdn.page_table_trim(t, l, dev(keep), s, f, page)
        assert l.tolist() == want[0] and int(f) == want[2] and s.tolist() == want[1]


@pytest.mark.parametrize("total", [0, 4096, 4097, 200000])
def test_slots_of_many_tokens(gdn, total):
    rng = np.random.default_rng(total)
    N, page, width = 37, 48, 200
    new = rng.multinomial(total, rng.dirichlet(np.ones(N)))
    table, lens, stack = state(rng, N, 5, page, 5000, 0)
    table = np.concatenate([table, np.zeros((N, width - 5), int)], 1)
    want = attention.extend(table.tolist(), lens.tolist(), new.tolist(), stack.tolist(), 5000, page, total)
    t, l, s, f = dev(table), dev(lens), dev(stack), dev([5000])
    slots, cu = gdn.page_table_extend(t, l, dev(new), s, f, page, total)
    assert slots.tolist() == want[3] and cu.tolist() == want[4] and t.tolist() == want[0] and l.tolist() == want[1] and int(f) == want[2]


def test_trim_undoes_extend(gdn):
    rng = np.random.default_rng(5)
    table, lens, stack = state(rng, 60, 12, 16, 300, 0)
    t, l, s, f = dev(table), dev(lens), dev(stack), dev([300])
    before = l.clone()
    gdn.page_table_extend(t, l, dev(rng.integers(0, 60, 60)), s, f, 16, 4000)
    gdn.page_table_trim(t, l, before, s, f, 16)
    assert torch.equal(l, before) and s.tolist() == stack.tolist() and int(f) == 300


def test_trim_of_more_pages_than_31_bits_count(gdn):
    """Every sequence gives up its whole row: the last ones' pages fill the stack, the others are dropped."""
    N, width, size = 8192, (1 << 18) + 5, 1000
    t = torch.full((N, width), -3, dtype=I32, device="cuda")
    t[-1] = torch.arange(width, device="cuda")
    l, s, f = torch.full((N,), width, dtype=I32, device="cuda"), torch.full((size + 64,), 77, dtype=I32, device="cuda"), dev([10])
    gdn.page_table_trim(t, l, torch.zeros_like(l), s[32:32 + size], f, 1)
    assert (l == 0).all() and int(f) == size
    assert (s[:42] == 77).all() and (s[32 + size:] == 77).all()
    assert s[42:32 + size].tolist() == list(range(width - 1, width - 1 - (size - 10), -1))


def test_no_sequences_and_no_pages(gdn):
    e = torch.zeros(0, dtype=I32, device="cuda")
    f = dev([3])
    slots, cu = gdn.page_table_extend(torch.zeros(0, 4, dtype=I32, device="cuda"), e, e, dev([1, 2]), f, 16, 5)
    assert slots.tolist() == [-1] * 5 and cu.tolist() == [0] and int(f) == 2
    slots, cu = gdn.page_table_extend(torch.zeros(2, 0, dtype=I32, device="cuda"), dev([0, 0]), dev([0, 3]), e, dev([0]), 16, 3)
    assert slots.tolist() == [-1] * 3 and cu.tolist() == [0, 0, 3]


def test_captured_table_steps(gdn):
    """A captured step run again and again: one more token a time until the pages run out."""
    N, page, width = 5, 4, 6
    table, lens, stack = np.zeros((N, width), int), np.zeros(N, int), np.arange(20)[::-1].copy()
    t, l, s, f, new = dev(table), dev(lens), dev(stack), dev([20]), dev([1] * N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            slots, cu = gdn.page_table_extend(t, l, new, s, f, page, N)
    torch.cuda.current_stream().wait_stream(side)
    model = (table.tolist(), lens.tolist(), 20)
    for _ in range(30):
        want = attention.extend(model[0], model[1], [1] * N, stack.tolist(), model[2], page, N)
        graph.replay()
        assert slots.tolist() == want[3] and l.tolist() == want[1] and int(f) == want[2] and t.tolist() == want[0]
        model = want[:3]


def test_captured_table_steps_of_many_tokens(gdn):
    """The form with two launches, twice in a graph, on another stream and again and again; then all that was taken is
    given back, in the order that giving back has."""
    rng = np.random.default_rng(3)
    N, page, width = 300, 16, 40
    table, lens, stack = state(rng, N, width, page, 9000, 0)
    lens = np.minimum(lens, 60)
    t, l, s, f = dev(table), dev(lens), dev(stack), dev([9000])
    new, before = [rng.multinomial(40000, rng.dirichlet(np.full(N, 20.0))) for _ in range(2)], l.clone()
    given, total = [dev(n) for n in new], 40000
    want, model = [], (table.tolist(), lens.tolist(), 9000)
    for n in new:
        want.append(attention.extend(model[0], model[1], n.tolist(), stack.tolist(), model[2], page, total))
        model = want[-1][:3]
    end = attention.trim(model[0], model[1], before.tolist(), stack.tolist(), model[2], page)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = []
            for n in given:
                out.append((*gdn.page_table_extend(t, l, n, s, f, page, total), l.clone(), f.clone(), t.clone()))
            gdn.page_table_trim(t, l, before, s, f, page)
        for _ in range(3):
            graph.replay()
            side.synchronize()
            for (slots, cu, length, free, pages), w in zip(out, want):
                assert slots.tolist() == w[3] and cu.tolist() == w[4] and length.tolist() == w[1] and int(free) == w[2] and pages.tolist() == w[0]
            assert l.tolist() == end[0] == before.tolist() and s.tolist() == end[1] and int(f) == end[2] == 9000
            t.copy_(dev(table))
            s.copy_(dev(stack))


# --------------------------------------------------------------------------- all of them together
@pytest.mark.parametrize("dtype,D", [(BF, 64), (BF, 128), (F32, 64)])
def test_from_a_prompt_to_accepted_drafts(gdn, dtype, D):
    """Room for packed prompts, their attention and keys into the pages; drafted trees verified; a branch accepted,
    written and decoded on: what attention over the whole text from the start gives for the same tokens.

    Both sides round weights and outputs (2^-8 each with bf16, of the values' size); fp32 2^-24 by the tokens."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    N, Hq, Hkv, page, width, T = 3, 8, 2, 16, 8, 5
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    prompts = [50, 16, 33]
    most = 80
    text = [dict(q=rnd(most, Hq, D), k=rnd(most, Hkv, D), v=rnd(most, Hkv, D)) for _ in range(N)]
    table, lens = torch.full((N, width), -1, dtype=I32, device="cuda"), torch.zeros(N, dtype=I32, device="cuda")
    stack, free = torch.randperm(30, generator=gen, device="cuda").to(I32), dev([30])
    kc, vc = (torch.full((30, page, Hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    slots, cu = gdn.page_table_extend(table, lens, dev(prompts), stack, free, page, sum(prompts))
    pack = lambda name, at: torch.cat([text[n][name][a:b] for n, (a, b) in enumerate(at)])  # noqa: E731
    first = [(0, p) for p in prompts]
    q, k, v = (pack(name, first)[None] for name in "qkv")
    got = [list(gdn.prompt_attention(q, k, v, cu_seqlens=cu)[0].split(prompts))]
    gdn.paged_cache_write(k, v, kc, vc, slots)
    # drafted: the tokens that the text goes on with at 0, 2 and 4, others in between
    line, trees = [0, 2, 4], [[-1, -1, 0, 1, 2]] * N
    dq, dk, dv = (rnd(N, T, h, D) for h in (Hq, Hkv, Hkv))
    for n in range(N):
        for i, t in enumerate(line):
            dq[n, t], dk[n, t], dv[n, t] = (text[n][x][prompts[n] + i] for x in "qkv")
    o = gdn.paged_attention_tree(dq, dk, dv, kc, vc, table, lens, dev(trees))
    slots, cu = gdn.page_table_extend(table, lens, dev([3] * N), stack, free, page, 3 * N)
    rows = dev([n * T + t for n in range(N) for t in line])
    gdn.paged_cache_write(dk, dv, kc, vc, slots, rows=rows)
    got.append([o[n, line] for n in range(N)])
    for i in range(4):  # and decoding
        slots, _ = gdn.page_table_extend(table, lens, dev([1] * N), stack, free, page, N)
        x = [torch.stack([text[n][name][prompts[n] + 3 + i] for n in range(N)]) for name in "qkv"]
        got.append(list(gdn.paged_attention_decode(x[0], kc, vc, table, lens, k_new=x[1], v_new=x[2])[:, None]))
    assert lens.tolist() == [p + 7 for p in prompts]
    for n in range(N):
        total = prompts[n] + 7
        want = gdn.prompt_attention(*(text[n][x][None, :total] for x in "qkv"))[0].float()
        mine = torch.cat([g[n] for g in got]).float()
        size = text[n]["v"][:total].float().abs().amax()
        tol = 4 * 2.0 ** -8 * size if dtype == BF else 1e-5 * size
        assert (mine - want).abs().max() <= tol
    gdn.page_table_trim(table, lens, dev([0] * N), stack, free, page)
    assert int(free) == 30 and sorted(stack.tolist()) == list(range(30))
