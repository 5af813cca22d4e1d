"""GPU parity of the recurrent step (gdn_recurrent_step) against its fp64 oracle.

Tolerances: a token's sums run over K = 128 products in fp32, so their error is at most
128 x 2^-24 sum |h k| <= 128 x 2^-24 x sqrt(128) max |h| for unit keys, 8.6e-5 of the largest
state; the decay (<= 1) and unit keys do not amplify it from token to token.  That is FP32_TOL
(1e-4 of the largest value).  bf16 outputs (8 significant bits) add half a unit of their
last place, 2^-8."""
import numpy as np
import pytest
import torch

from oracle import decode
from tests.gpu_util import FP32_TOL, rel_err

pytestmark = pytest.mark.gpu
OUT_TOL = {torch.bfloat16: 2.0 ** -8 + FP32_TOL, torch.float32: FP32_TOL}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build
    build.build()


def inputs(T, Hqk, Hv, slots, seed, dtype, raw=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k, v = r(T, Hqk, 128), r(T, Hqk, 128), r(T, Hv, 128)
    g, beta = r(T, Hv), r(T, Hv)
    d = dict(state=0.3 * r(slots, Hv, 128, 128), A_log=None, dt_bias=None)
    if raw:
        d.update(A_log=0.5 * r(Hv), dt_bias=r(Hv))
    else:
        q, k = (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
        g, beta = -torch.nn.functional.softplus(2 * g - 2), torch.sigmoid(beta)
    d.update(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype), g=g, beta=beta)
    return d


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def oracle(d, slots, lens, scale):
    a = {n: np64(t) for n, t in d.items()}
    return decode.step(a["q"], a["k"], a["v"], a["g"], a["beta"], scale, a["state"], slots, lens, a["A_log"], a["dt_bias"])


def cuda(d, lead=None):
    x = {n: None if t is None else t.cuda() for n, t in d.items()}
    for n in ("q", "k", "v", "g", "beta"):
        x[n] = x[n].unflatten(0, lead or (1, -1))
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("N,L,Hqk,Hv", [(1, 1, 1, 1), (3, 1, 2, 8), (2, 5, 4, 12), (1, 33, 1, 3)])
def test_equal_lengths(dtype, raw, N, L, Hqk, Hv):
    from chunked_prefill_gb300 import gdn
    d = inputs(N * L, Hqk, Hv, N, 10 * N + L, dtype, raw)
    x = cuda(d, (N, L))
    state = x["state"].clone()
    o, new = gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state=state, A_log=x["A_log"],
                                       dt_bias=x["dt_bias"])
    assert new is state and o.shape == (N, L, Hv, 128)
    ro, rs = oracle(d, list(range(N)), [L] * N, 128 ** -0.5)
    assert rel_err(np64(o).reshape(ro.shape), ro) <= OUT_TOL[dtype]
    assert rel_err(np64(new), rs) <= FP32_TOL


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_with_slots(dtype, in_place):
    """Uneven token counts (none, one, many) in shuffled slots, a padding row and a slot past the
    pool; the other slots keep their contents."""
    from chunked_prefill_gb300 import gdn
    lens, slots, pool = [2, 0, 1, 7, 3, 2], [4, 1, 8, 0, -1, 9], 9
    T = sum(lens)
    d = inputs(T, 2, 6, pool, 21, dtype)
    x = cuda(d)
    out = x["state"] if in_place else torch.full_like(x["state"], 7.0)
    before = x["state"].clone()
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    o, new = gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=0.2, state=x["state"],
                                       state_out=out, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), cu_seqlens=cu)
    ro, rs = oracle(d, slots, lens, 0.2)
    assert rel_err(np64(o)[0], ro) <= OUT_TOL[dtype]
    assert (o[0, 10:] == 0).all()  # the two sequences without a slot
    named = [4, 1, 8, 0]
    assert rel_err(np64(new)[named], rs[named]) <= FP32_TOL
    assert torch.equal(new[1], before[1])  # no tokens: the state as it was
    for s in set(range(pool)) - set(named):
        assert torch.equal(new[s], before[s] if in_place else torch.full_like(new[s], 7.0))
    if not in_place:
        assert torch.equal(x["state"], before)


def test_strided_rows_and_zero_state():
    """q, k, v, a, b as views of a fused projection's rows (a, b on 4-byte boundaries), no entering
    state: the same bits as contiguous copies."""
    from chunked_prefill_gb300 import gdn
    N, Hqk, Hv = 3, 2, 5 * 2
    d = inputs(N, Hqk, Hv, N, 4, torch.bfloat16, raw=True)
    x = cuda(d, (N, 1))
    want = gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], A_log=x["A_log"], dt_bias=x["dt_bias"])
    rows = torch.randn(N, (2 * Hqk + Hv) * 128 + 8, device="cuda").to(torch.bfloat16)
    ab = torch.randn(N, 2 * Hv + 1, device="cuda")
    parts = [rows[:, 8:8 + Hqk * 128], rows[:, 8 + Hqk * 128:8 + 2 * Hqk * 128], rows[:, 8 + 2 * Hqk * 128:]]
    gates = [ab[:, 1:1 + Hv], ab[:, 1 + Hv:]]
    for p, n in zip(parts + gates, ("q", "k", "v", "g", "beta")):
        p.copy_(x[n].reshape(N, -1))
    q, k, v = (p.unflatten(-1, (-1, 128))[:, None] for p in parts)
    g, beta = (p[:, None] for p in gates)
    got = gdn.gated_delta_rule_step(q, k, v, g, beta, A_log=x["A_log"], dt_bias=x["dt_bias"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    zero = dict(d, state=torch.zeros_like(d["state"]))
    ro, rs = oracle(zero, list(range(N)), [1] * N, 128 ** -0.5)
    assert rel_err(np64(got[0]).reshape(ro.shape), ro) <= OUT_TOL[torch.bfloat16]
    assert rel_err(np64(got[1]), rs) <= FP32_TOL


def test_continues_the_chunked_prefill():
    """Prefill through chunk_gated_delta_rule, then single steps from its final state, against the
    oracle over the whole sequence."""
    from chunked_prefill_gb300 import gdn
    P, L, Hqk, Hv = 100, 4, 2, 4
    d = inputs(P + L, Hqk, Hv, 1, 9, torch.float32)
    x = cuda(d)
    part = lambda n, a, b: x[n][:, a:b].contiguous()  # noqa: E731
    names = ("q", "k", "v", "g", "beta")
    _, state = gdn.chunk_gated_delta_rule(*(part(n, 0, P) for n in names), initial_state=x["state"], output_final_state=True)
    outs = []
    for t in range(P, P + L):
        o, state = gdn.gated_delta_rule_step(*(part(n, t, t + 1) for n in names), state=state)
        outs.append(o)
    ro, rs = oracle(d, [0], [P + L], 128 ** -0.5)
    assert rel_err(np64(torch.cat(outs, 1))[0], ro[P:]) <= FP32_TOL
    assert rel_err(np64(state), rs) <= FP32_TOL


def test_decay_to_nothing_and_full_write():
    """g = -inf forgets the state entirely; beta = 1 with a unit key writes v at that key."""
    from chunked_prefill_gb300 import gdn
    d = inputs(1, 1, 1, 1, 2, torch.float32)
    d["g"].fill_(-float("inf"))
    d["beta"].fill_(1.0)
    x = cuda(d)
    _, new = gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"])
    want = np.outer(np64(d["k"])[0, 0], np64(d["v"])[0, 0])
    assert rel_err(np64(new)[0, 0], want) <= FP32_TOL


@pytest.mark.parametrize("gates", [[0.0, -0.01, -5.0, -40.0, 0.0], [-3.0], [0.7], [-100.0, 0.0], [0.0, -float("inf"), -0.5, 20.0, -20.0]])
def test_decays_of_every_size_over_many_tokens(gates):
    """Decays that add up past any factor kept aside of the state, down and up.  A growing state's errors
    grow with it: each token adds at most |k_i| <= 0.3 times 1e-4 of its largest value."""
    from chunked_prefill_gb300 import gdn
    T = 43
    d = inputs(T, 2, 4, 1, 12, torch.float32)
    d["g"] = torch.tensor(gates)[torch.arange(T) % len(gates)][:, None].repeat(1, 4) * (1 + 0.1 * torch.arange(4))
    x = cuda(d)
    o, new = gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"].clone())
    ro, rs = oracle(d, [0], [T], 128 ** -0.5)
    tol = 0.3 * T * FP32_TOL
    assert rel_err(np64(new), rs) <= tol
    o = np64(o)[0]
    assert all(rel_err(o[t], ro[t]) <= tol for t in range(T))


def test_other_stream_graph_and_determinism():
    """A captured step replayed with other lengths and slots, on a stream of its own; repeated
    calls give equal bits."""
    from chunked_prefill_gb300 import gdn
    d = inputs(4, 1, 2, 4, 6, torch.bfloat16)
    x = cuda(d)
    cu = torch.tensor([0, 1, 2, 4], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    out, o = torch.zeros_like(x["state"]), torch.empty_like(x["v"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def call():
        gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], scale=1.0, state=x["state"], state_out=out,
                                  slots=slots, cu_seqlens=cu, o=o)

    with torch.cuda.stream(st):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            call()
        for lens, sl in (([1, 1, 2], [2, 0, 1]), ([3, 0, 1], [3, -1, 2])):
            cu.copy_(torch.tensor(np.cumsum([0] + lens), dtype=torch.int32))
            slots.copy_(torch.tensor(sl, dtype=torch.int32))
            out.zero_()
            graph.replay()
            first = (o.clone(), out.clone())
            graph.replay()
            st.synchronize()
            assert torch.equal(o, first[0]) and torch.equal(out, first[1])
            ro, rs = oracle(d, sl, lens, 1.0)
            live = [s for s in sl if s >= 0]
            assert rel_err(np64(o)[0], ro) <= OUT_TOL[torch.bfloat16]
            assert rel_err(np64(out)[live], rs[live]) <= FP32_TOL


def test_pool_past_32_bit_offsets():
    """A slot whose state starts past 2^31 values."""
    from chunked_prefill_gb300 import gdn
    Hv, slot = 64, 2100
    pool = torch.empty(slot + 1, Hv, 128, 128, device="cuda")
    assert slot * Hv * 128 * 128 > 2 ** 31
    d = inputs(1, 16, Hv, 1, 8, torch.bfloat16)
    pool[slot] = d["state"][0].cuda()
    x = cuda(d)
    o, _ = gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state=pool,
                                     slots=torch.tensor([slot], dtype=torch.int32, device="cuda"))
    ro, rs = oracle(d, [0], [1], 128 ** -0.5)
    assert rel_err(np64(o)[0], ro) <= OUT_TOL[torch.bfloat16]
    assert rel_err(np64(pool[slot]), rs[0]) <= FP32_TOL


def test_refusals():
    from chunked_prefill_gb300 import gdn
    d = inputs(2, 2, 2, 2, 1, torch.bfloat16)
    x = cuda(d, (2, 1))
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    bad = lambda: pytest.raises(ValueError)  # noqa: E731
    with bad():
        gdn.gated_delta_rule_step(*a[:3], a[3].half(), a[4], state=x["state"])
    with bad():
        gdn.gated_delta_rule_step(*a, state=x["state"].double())
    with bad():
        gdn.gated_delta_rule_step(*a, state=x["state"][:1])  # fewer slots than sequences
    with bad():
        gdn.gated_delta_rule_step(*a, state=x["state"], slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with bad():
        gdn.gated_delta_rule_step(*a, state=x["state"], cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with bad():
        gdn.gated_delta_rule_step(x["q"].cpu(), *a[1:], state=x["state"])
    with bad():
        gdn.gated_delta_rule_step(x["q"].transpose(2, 3).contiguous().transpose(2, 3), *a[1:], state=x["state"])
    with pytest.raises(gdn.GdnError):
        gdn.gated_delta_rule_step(*a, state=x["state"], A_log=torch.zeros(2, device="cuda"))  # dt_bias missing
    with pytest.raises(gdn.GdnError):
        gdn.gated_delta_rule_step(*a, state=x["state"], scale=float("nan"))
    with pytest.raises(RuntimeError, match="differentiable"):
        gdn.gated_delta_rule_step(a[0].requires_grad_(True), *a[1:], state=x["state"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu,slots", [([3, 4, 4, 9], [1, 0, 2]), ([0, 9], [0]), ([5, 6], [-1]), ([0, 0, 0], [0, 1]), ([0], [])])
def test_tokens_of_no_sequence_get_zeros(dtype, cu, slots):
    """Tokens before the first offset and past the last one: 0 in an o that the call makes (not what lay in
    that memory before), untouched in a given one."""
    from chunked_prefill_gb300 import gdn
    T = 21
    d = inputs(T, 2, 6, 3, 33, dtype)
    x = cuda(d)
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    covered = torch.zeros(T, dtype=torch.bool, device="cuda")
    covered[cu[0]:cu[-1]] = True
    state, given = x["state"], torch.full_like(x["v"], 7.0)
    poison = torch.full_like(x["v"], float("nan"))
    del poison  # the next allocation of this size gets its memory
    o, _ = gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state=state.clone(), slots=sl, cu_seqlens=offsets)
    assert (o[0, ~covered] == 0).all() and torch.isfinite(o).all()
    gdn.gated_delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state=state.clone(), slots=sl, cu_seqlens=offsets, o=given)
    assert (given[0, ~covered] == 7.0).all() and torch.equal(given[0, covered], o[0, covered])
    live = [b - a for a, b in zip(cu, cu[1:])]
    shifted = {k: v[cu[0]:] if k in ("q", "k", "v", "g", "beta") else v for k, v in d.items()}
    if sum(live):
        ro, _ = oracle(shifted, slots, live, 128 ** -0.5)
        assert rel_err(np64(o)[0, cu[0]:cu[-1]], ro[:sum(live)]) <= OUT_TOL[dtype]
