"""The hybrid decoding example: its operators together.  Decoding token by token after a prompt gives
the logits of a prompt that held those tokens from the start.

Both ways round every layer's output to bf16 in other orders (chunked against recurrent rule, fp32
softmax against the paged kernel), half a unit of 2^-8 each, and the last norm to 8 bits (2^-4 of a
value, independent over 512 values): the logits, sums over 512 such values, are compared by their
relative 2-norm, 2^-4 sqrt(2) x 1/2 = 4.4e-2 for the roundings to 8 bits (two sides, uniformly
distributed: 1 / sqrt(3) of the half step) plus 3 layers x 2 roundings x 2^-8 = 2.4e-2."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
TOL = 4.4e-2 + 2.4e-2


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("hybrid_decode", PATH)
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod  # dataclasses look their module up there
    spec.loader.exec_module(mod)
    return mod


def test_decode_continues_the_prompt(ex):
    model = ex.HybridModel(ex.Config())
    N, T, more, pages = 3, 70, 4, 6
    gen = torch.Generator(device="cuda").manual_seed(2)
    tokens = torch.randint(0, model.cfg.vocab, (N, T + more), generator=gen, device="cuda")
    slots = torch.tensor([2, 0, 4], dtype=torch.int32, device="cuda")
    table = torch.randperm(N * pages, generator=gen, device="cuda").to(torch.int32).view(N, pages)
    want = model.prefill(tokens, model.new_cache(5, N * pages), slots, table)
    pools = model.new_cache(5, N * pages)
    model.prefill(tokens[:, :T], pools, slots, table)
    lens = torch.full((N,), T, dtype=torch.int32, device="cuda")
    for t in range(T, T + more):
        lens += 1
        got = model.decode(tokens[:, t], pools, slots, table, lens)
    err = ((got - want).norm() / want.norm()).item()
    assert err <= TOL, err
    # one sequence alone, in another batch
    pools = model.new_cache(5, N * pages)
    model.prefill(tokens[1:2, :T], pools, slots[1:2], table[1:2])
    lens = torch.full((1,), T, dtype=torch.int32, device="cuda")
    for t in range(T, T + more):
        lens += 1
        alone = model.decode(tokens[1:2, t], pools, slots[1:2], table[1:2], lens)
    assert ((alone - got[1:2]).norm() / got[1:2].norm()).item() <= TOL


def test_example_runs(ex, capsys):
    ex.main()
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 4 and all(len(eval(line.split(": ")[1])) == 33 for line in lines)
