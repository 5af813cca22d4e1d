"""Infinite and NaN values behind masks of attention over prompts and drafted trees: they reach the rows that see them, and
leave every other number as it is, bit for bit.  And windows, whose edges are such masks, in every plan."""
import pytest
import torch

from oracle import attention
from tests.test_gpu_prompt import check as check_prompt, make as make_prompt
from tests.test_gpu_tree import call, check, make

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


def offsets(lens):
    return [sum(lens[:n]) for n in range(len(lens) + 1)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seed", [0, 1])
def test_tiles_of_queries_in_turn(gdn, D, seed):
    """Hundreds of short sequences, so that a CTA takes many tiles of queries in turn, some of which have no rows (50
    tokens), or see no keys (200 queries of 60 keys), in one half of a tile.  What a tile's warps know of its bad values
    may not be overwritten by those of a later one before they have used it."""
    gen = torch.Generator().manual_seed(seed)
    kinds = [(200, 200), (50, 50), (50, 50), (50, 50), (50, 90), (200, 60), (129, 129)]
    lens = [kinds[int(i)] for i in torch.randint(0, len(kinds), (320,), generator=gen)]
    cu, cu_k = (offsets([x[i] for x in lens]) for i in (0, 1))
    Hq, Hkv = 8, 2
    q, k, v = (torch.randn(1, n, h, D, generator=gen).to(BF).cuda() for n, h in ((cu[-1], Hq), (cu_k[-1], Hkv), (cu_k[-1], Hkv)))
    args = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), cu_seqlens_k=torch.tensor(cu_k, dtype=torch.int32, device="cuda"), return_lse=True)
    o, lse = gdn.prompt_attention(q, k, v, **args)
    # of two sequences in three the keys from one on are bad, in a column of the sequence's own
    bad, hit = v.clone(), torch.zeros_like(o, dtype=torch.bool)
    for n, (lq, lk) in enumerate(lens):
        if n % 3 == 2:
            continue
        first, column = int(torch.randint(0, lk, (1,), generator=gen)), n % D
        bad[0, cu_k[n] + first:cu_k[n + 1], :, column] = float("nan")
        sees = torch.arange(lq) + lk - lq >= first
        hit[0, cu[n]:cu[n + 1], :, column] = sees[:, None].cuda()
    for _ in range(10):
        ob, lb = gdn.prompt_attention(q, k, bad, **args)
        assert torch.equal(lb, lse)
        assert torch.equal(torch.isnan(ob), hit)
        assert torch.equal(torch.where(hit, o, ob), o)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 70, 130, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_windows_of_prompts(gdn, dtype, D, window, value):
    """Bad keys on either side of both edges of what queries see, and in tiles that all see; more keys than queries."""
    gen = torch.Generator().manual_seed(D + window)
    lens = [(300, 300), (130, 500), (257, 257), (700, 700), (1, 128), (140, 30)]
    cu, cu_k = (offsets([x[i] for x in lens]) for i in (0, 1))
    q, k, v = (torch.randn(1, n, h, D, generator=gen).to(dtype).cuda() for n, h in ((cu[-1], 4), (cu_k[-1], 2), (cu_k[-1], 2)))
    args = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), cu_seqlens_k=torch.tensor(cu_k, dtype=torch.int32, device="cuda"), return_lse=True, window=window)
    o, lse = gdn.prompt_attention(q, k, v, **args)
    bad, hit = v.clone(), torch.zeros_like(o, dtype=torch.bool)
    for n, (lq, lk) in enumerate(lens):
        at = torch.arange(lq) + lk - lq
        for i, t in enumerate(sorted({int(x) for x in torch.randint(0, lk, (5,), generator=gen)} | {0, lk - 1, min(127, lk - 1), min(128, lk - 1)})):
            head, column = i % 2, (7 * i + n) % D
            bad[0, cu_k[n] + t, head, column] = value
            sees = (at >= t) & (at < t + window if window else at >= 0)
            hit[0, cu[n]:cu[n + 1], 2 * head:2 * head + 2, column] |= sees[:, None].cuda()
    ob, lb = gdn.prompt_attention(q, k, bad, **args)
    assert torch.equal(lb, lse)
    assert torch.equal(~torch.isfinite(ob), hit)
    assert torch.equal(torch.where(hit, o, ob), o)


CHAIN, FORKS = list(range(-1, 63)), [t // 2 - 1 for t in range(64)]


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,T", [(2, 9), (2, 64), (8, 64), (32, 11)])
@pytest.mark.parametrize("window", [0, 5, 100, 2500])
def test_trees(gdn, cache, D, Hq, T, window):
    """Cached tokens on either side of the edge of every drafted token's window, in the middle and at the end, and
    drafted tokens; blocks of rows of one and of two tiles, edges in one and in two tiles of tokens, sequences in one CTA's
    part and in several."""
    lens = [300, 5300, 64, 0, 129]
    x = make(lens, T, Hq, 2, D, 16, cache, seed=T + window, trees=[(CHAIN if n % 2 == 0 else FORKS)[:T] for n in range(len(lens))])
    o, lse = call(gdn, x, window=window)
    assert torch.isfinite(o).all()
    value = float("nan") if cache == FP8 else float("inf")
    y, hit, G = dict(x, v=x["v"].clone(), vn=x["vn"].clone()), torch.zeros_like(o, dtype=torch.bool), Hq // 2
    lines = [attention.ancestors(p) for p in x["parents"].tolist()]
    table = x["table"].tolist()
    for n, length in enumerate(lens):
        first = [max(0, length + len(line) - window) if window else 0 for line in lines[n]]
        edges = {f + d for f in (first[0], first[T // 2], first[-1]) for d in (-1, 0, 1)}
        for i, pos in enumerate(sorted(p for p in edges | {0, 100, length // 2, length - 1} if 0 <= p < length)):
            head, column = i % 2, (5 * i + n) % D
            y["v"][table[n][pos // 16], pos % 16, head, column] = value
            for t in range(T):
                if pos >= first[t]:
                    hit[n, t, head * G:(head + 1) * G, column] = True
        for i, new in enumerate(sorted({0, T // 3, T - 1})):
            head, column = i % 2, D - 1 - i
            y["vn"][n, new, head, column] = float("inf")
            for t in range(T):
                if new in (lines[n][t][:window] if window else lines[n][t]):
                    hit[n, t, head * G:(head + 1) * G, column] = True
    for _ in range(2):
        ob, lb = call(gdn, y, window=window)
        assert torch.equal(lb, lse)
        assert torch.equal(~torch.isfinite(ob), hit)
        assert torch.equal(torch.where(hit, o, ob), o)


@pytest.mark.parametrize("cache", [BF, FP8, F32])
@pytest.mark.parametrize("D,Hq,T", [(64, 8, 64), (128, 8, 64), (128, 32, 11), (256, 2, 64), (256, 8, 9)])
@pytest.mark.parametrize("window", [1, 17, 64, 100, 2000])
def test_windows_of_trees(gdn, cache, D, Hq, T, window):
    """The outputs themselves, in the plans that the tests of one tile of rows do not reach."""
    x = make([3000, 1, 0, 63, 64, 130], T, Hq, 2, D, 24, cache, seed=window, trees=[CHAIN[:T]] * 3 + [FORKS[:T]] * 3)
    check(x, *call(gdn, x, window=window), window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [1, 64, 129, 200])
def test_windows_of_prompts_and_their_gradient(gdn, dtype, D, window):
    check_prompt(gdn, make_prompt([(300, 300), (130, 400), (5, 2), (0, 3), (400, 130)], 4, 2, D, dtype, seed=window), window)
