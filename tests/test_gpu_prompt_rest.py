"""What rounding the output to bf16 leaves (o_rest of gdn_prompt_attn_fwd) and what the gradient gains by it.

Equal scores make weights of exactly 1, so that o is a mean of few bf16 values: its sum over L keys is off by
(64 + L) 2^-24 of the values' sizes (as in test_gpu_prompt.py), its quotient by 2^-22 of itself, and nothing else is rounded
before o is.  What that leaves is at most 2^-8 |o| and rounded by 2^-8 of itself: o + rest is off by 2^-16 |o|."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prompt import args, make, np64, oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build, gdn
    build.build()
    return gdn


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [3, 8])
def test_output_and_rest_are_the_output_to_16_bits(gdn, D, window):
    x = make([(300, 300), (40, 90), (5, 3)], 4, 2, D, seed=D + window, front=3, behind=20, q_std=0.0)
    r = oracle(x, window)
    o, lse, rest = gdn.gdn_prompt_attn_fwd(x["q"], x["k"], x["v"], lse=True, rest=True, window=window, **args(x))
    rows = slice(x["cu"][0], x["cu"][-1])
    o, rest, want, mass = np64(o)[0][rows], np64(rest)[0][rows], r["o"][rows], r["mass"][rows]
    tol = (2.0 ** -16 + 2.0 ** -22) * np.abs(want) + (64 + window) * 2.0 ** -24 * mass
    assert (np.abs(o + rest - want) <= tol).all()
    rounded = np.abs(o - want) > tol  # where o alone is not as near
    assert rounded.mean() > 0.25 and (rest[rounded] != 0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_gradient_is_nearer_with_the_rest(gdn, D):
    """Values far from zero: dz = p (do v - <do, o>) is a small difference of large terms, into which o's rounding goes."""
    x = make([(200, 200), (70, 150)], 4, 2, D, seed=D)
    x["v"] = (x["v"].float() + 16).to(torch.bfloat16)
    r = oracle(x, 0, True)
    o, lse, rest = gdn.gdn_prompt_attn_fwd(x["q"], x["k"], x["v"], lse=True, rest=True, **args(x))
    off = []
    for given in (None, rest):
        dq, dk, _ = gdn.gdn_prompt_attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], o_rest=given, **args(x))
        off.append([float(np.linalg.norm(np64(g)[0] - r[n]) / np.linalg.norm(r[n])) for n, g in (("dq", dq), ("dk", dk))])
    assert off[1][0] < off[0][0] and off[1][1] < off[0][1]
