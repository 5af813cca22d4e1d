"""Infinite and NaN values behind masks, where the plans of attention over prompts keep records of them: they reach the rows
that see them, and leave every other number as it is, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
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
