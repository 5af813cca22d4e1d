"""Measured cases of the operators that a decoding step of a gated-delta-rule model is made of:

  step   gdn.gated_delta_rule_step    the recurrent gated delta rule over a pool of states
  attn   gdn.paged_attention_decode   one new token per sequence over a paged key-value cache
  norm   gdn.rms_norm, gdn.rms_norm_quant, gdn.gdn_rmsnorm_bwd
                                      root-mean-square norm with the residual's addition, its
                                      8-bit form and its backward pass

``run`` makes the library's calls where ``own`` is true and computes the same results from
elementary tensor operations in fp32 elsewhere; ``exact`` computes them in fp64 from the
definitions.  All inputs come from ``prepare``'s seed; head counts are those of the library's
workloads and head sweep.
"""
import math
import random

import torch

own = False
DEVICE = "cuda"

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
FP8_TINY = 2.0 ** -126  # smallest 8-bit output scale
EPS = 1e-6
K = V = 128
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": FP8}
BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}


def listed():
    step = dict(op="step", ragged=False, raw=False, packed=False, dtype="bf16")
    attn = dict(op="attn", ragged=True, append=False, window=0, heads_first=False, dtype="bf16")
    norm = dict(op="norm", residual=True, backward=False, dtype="bf16", out="bf16", group=0, offset=0.0)
    return [
        # one user's next token, two q/k and eight v heads: latency alone
        dict(step, name="step_single", seqs=1, tokens=1, hqk=2, hv=8, pool=1),
        # a served batch fed by the layer's raw projections, views of the fused projection's rows
        dict(step, name="step_batch", seqs=32, tokens=1, hqk=8, hv=24, pool=40, raw=True, packed=True),
        # one to six drafted tokens per sequence, packed, fp32 activations
        dict(step, name="step_draft", seqs=48, tokens=6, hqk=16, hv=48, pool=48, ragged=True, dtype="fp32"),
        # a full batch of every head: 1 GB of states in, 1 GB out
        dict(step, name="step_large", seqs=256, tokens=1, hqk=16, hv=64, pool=320),
        # a few short chats, wide heads, the new token's key and value written by the call
        dict(attn, name="attn_short", seqs=4, most=700, hq=16, hkv=2, dim=256, page=16, append=True),
        # one long document, an odd number of tokens
        dict(attn, name="attn_long", seqs=1, most=131071, hq=32, hkv=4, dim=128, page=64, ragged=False),
        # a served batch of uneven lengths, one of its rows empty
        dict(attn, name="attn_batch", seqs=64, most=8192, hq=32, hkv=8, dim=128, page=16),
        # a large batch over an 8-bit cache, pages that are no power of two, heads before tokens
        dict(attn, name="attn_fp8", seqs=128, most=16384, hq=64, hkv=8, dim=128, page=48, dtype="e4m3",
             heads_first=True),
        # a decoding step's rows, quantised for an 8-bit product
        dict(norm, name="norm_few", rows=16, dim=2048, out="e4m3"),
        # a prompt's rows
        dict(norm, name="norm_prompt", rows=32768, dim=4096),
        # an odd number of rows, 8 bits with one scale to 128 values
        dict(norm, name="norm_groups", rows=8191, dim=5120, out="e4m3", group=128),
        # a training step's gradient
        dict(norm, name="norm_grad", rows=32768, dim=2048, backward=True, offset=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "attn", "norm"])
    if op == "step":
        hqk, hv = rng.choice([(1, 1), (2, 4), (2, 8), (4, 16), (8, 24), (16, 16), (16, 48), (16, 64)])
        tokens = rng.choice([1, 1, rng.randint(2, 8)])
        seqs = _log(rng, 1, min(512, 12000 // (hv * (1 if tokens == 1 else 3))))
        return dict(op=op, seqs=seqs, tokens=tokens, hqk=hqk, hv=hv, pool=seqs + rng.randint(0, 1 + seqs // 4),
                    ragged=tokens > 1 and rng.random() < 0.7, raw=rng.random() < 0.5, packed=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "attn":
        hq, hkv = rng.choice([(4, 4), (8, 1), (16, 2), (24, 8), (32, 4), (32, 8), (64, 8), (40, 1)])
        dim = rng.choice([64, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "bf16", "e4m3", "e4m3", "fp32"])
        room = (3 << 29) // (hkv * dim * 2 * BYTES[dtype]) // (4 if dtype == "fp32" else 1)  # tokens over all sequences
        seqs = _log(rng, 1, 256)
        most = _log(rng, 1, min(200000, max(1, room // seqs), max(1, (1 << 30) // (seqs * hkv * dim))))
        return dict(op=op, seqs=seqs, most=most, hq=hq, hkv=hkv, dim=dim, page=rng.choice([1, 16, 24, 32, 64, 100, 256]),
                    ragged=rng.random() < 0.7, append=seqs * most < 20000 and rng.random() < 0.5,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), heads_first=rng.random() < 0.3, dtype=dtype)
    dim = rng.choice([64 * _log(rng, 1, 128), 128 * _log(rng, 1, 64), _log(rng, 1, 8192)])
    out = rng.choice(["same", "e4m3"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    backward = out == "same" and rng.random() < 0.5
    return dict(op=op, rows=_log(rng, 1, (1 << 26) // max(dim, 512) // (2 if dtype == "fp32" else 1)), dim=dim,
                residual=rng.random() < 0.7, backward=backward, dtype=dtype, out=dtype if out == "same" else out,
                group=rng.choice([g for g in (0, 0, 32, 64, 128) if g == 0 or dim % g == 0]) if out == "e4m3" else 0,
                offset=rng.choice([0.0, 1.0]))


def _lengths(case, most):
    """The case's lengths per sequence: `most` throughout, or between nothing and `most`."""
    n = case["seqs"]
    if not case["ragged"]:
        return [most] * n
    r = random.Random(n * 1000003 + most)
    least = 1 if case["op"] == "step" or case["append"] else 0
    got = [r.randint(max(1, least), most) for _ in range(n)]
    got[0] = most
    if n > 2 and least == 0:
        got[1] = 0  # a padding row of a captured batch
    return got


def _ordered(case, most, seed):
    got = _lengths(case, most)
    random.Random(seed).shuffle(got)
    return got


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=DEVICE)  # noqa: E731
    return {"step": _prepare_step, "attn": _prepare_attn, "norm": _prepare_norm}[case["op"]](case, seed, gen, randn)


def _prepare_step(c, seed, gen, randn):
    dt, n, hqk, hv = TYPES[c["dtype"]], c["seqs"], c["hqk"], c["hv"]
    lens = _ordered(c, c["tokens"], seed)
    total = sum(lens)
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    B, T = (1, total) if c["ragged"] else (n, c["tokens"])
    x, ab = randn(total, (2 * hqk + hv) * K), randn(total, 2 * hv)
    x[:, (2 * hqk) * K:] *= 0.5
    if not c["raw"]:
        qk = x[:, :2 * hqk * K].view(total, 2 * hqk, K)
        qk /= (qk.square().sum(-1, keepdim=True) + EPS).sqrt()
        # the decays of a trained layer: most heads keep what they hold for many tokens
        ab[:, :hv] = -torch.nn.functional.softplus(2 * ab[:, :hv] - 2)
        ab[:, hv:] = torch.sigmoid(ab[:, hv:])
    x = x.to(dt)
    parts = [x[:, :hqk * K], x[:, hqk * K:2 * hqk * K], x[:, 2 * hqk * K:], ab[:, :hv], ab[:, hv:]]
    if not c["packed"]:
        parts = [p.contiguous() for p in parts]
    q, k, v = (p.unflatten(-1, (-1, K)).unflatten(0, (B, T)) for p in parts[:3])
    g, beta = (p.unflatten(0, (B, T)) for p in parts[3:])
    slots = torch.randperm(c["pool"], generator=gen, device=DEVICE)[:n].to(torch.int32)
    return dict(case=c, q=q, k=k, v=v, g=g, beta=beta, scale=K ** -0.5,
                state=0.3 * randn(c["pool"], hv, K, V), state_out=torch.zeros(c["pool"], hv, K, V, device=DEVICE),
                slots=slots, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEVICE) if c["ragged"] else None,
                A_log=torch.log(1 + 15 * torch.rand(hv, generator=gen, device=DEVICE)) - 3 if c["raw"] else None,
                dt_bias=randn(hv) if c["raw"] else None, lens=lens)


def _prepare_attn(c, seed, gen, randn):
    n, hq, hkv, D, page = c["seqs"], c["hq"], c["hkv"], c["dim"], c["page"]
    lens = _ordered(c, c["most"], seed)
    used = [-(-x // page) for x in lens]
    pages = sum(used) + 1 + n // 8
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.zeros(n, max(max(used), 1), dtype=torch.int32, device=DEVICE)
    have = torch.arange(table.shape[1], device=DEVICE) < torch.tensor(used, device=DEVICE)[:, None]
    table[have] = order[:sum(used)]
    act = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16

    def cache(std):
        shape = (pages, hkv, page, D) if c["heads_first"] else (pages, page, hkv, D)
        x = torch.empty(shape, dtype=TYPES[c["dtype"]], device=DEVICE)
        step = max(1, (1 << 27) // x[0].numel())
        for i in range(0, pages, step):  # in parts: the fp32 draws of a whole cache need not fit beside it
            m = min(step, pages - i)
            x[i:i + m] = (std * torch.randn(m, *shape[1:], generator=gen, device=DEVICE)).to(x.dtype)
        return x.transpose(1, 2) if c["heads_first"] else x

    s = dict(case=c, q=(1.5 * randn(n, hq, D)).to(act), k_cache=cache(1.0), v_cache=cache(1.0), table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE), scale=D ** -0.5, window=c["window"],
             k_new=None, v_new=None, k_scale=None, v_scale=None)
    if c["dtype"] == "e4m3":
        s["k_scale"], s["v_scale"] = (0.5 + torch.rand(hkv, generator=gen, device=DEVICE) for _ in range(2))
    if c["append"]:
        s["k_new"], s["v_new"] = (randn(n, hkv, D).to(act) for _ in range(2))
    return s


def _prepare_norm(c, seed, gen, randn):
    dt, rows, dim = TYPES[c["dtype"]], c["rows"], c["dim"]
    s = dict(case=c, x=randn(rows, dim).to(dt), weight=((1 - c["offset"]) + 0.2 * randn(dim)).to(dt), residual=None,
             dy=None, dsum=None)
    if c["residual"]:
        r = (2 * randn(rows, dim)).to(dt)
        if c["backward"]:
            s["x"], s["dsum"] = s["x"] + r, randn(rows, dim).to(dt)
        else:
            s["residual"] = r
    if c["backward"]:
        s["dy"] = randn(rows, dim).to(dt)
    return s


# ------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return {"step": _own_step, "attn": _own_attn, "norm": _own_norm}[state["case"]["op"]](state)
    return {"step": _plain_step, "attn": _plain_attn, "norm": _plain_norm}[state["case"]["op"]](state)


def _own_step(s):
    from chunked_prefill_gb300 import gdn
    o, state = gdn.gated_delta_rule_step(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"],
                                         state=s["state"], state_out=s["state_out"], slots=s["slots"],
                                         cu_seqlens=s["cu_seqlens"], A_log=s["A_log"], dt_bias=s["dt_bias"])
    return {"o": o, "state": state}


def _own_attn(s):
    from chunked_prefill_gb300 import gdn
    o, lse = gdn.paged_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], scale=s["scale"],
                                        window=s["window"], k_new=s["k_new"], v_new=s["v_new"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
    return _with_caches(s, {"o": o, "lse": lse})


def _own_norm(s):
    from chunked_prefill_gb300 import gdn
    c = s["case"]
    if c["backward"]:
        dx, dw = gdn.gdn_rmsnorm_bwd(s["x"], s["weight"], s["dy"], dsum=s["dsum"], eps=EPS, weight_offset=c["offset"])
        return {"dx": dx, "dweight": dw}
    if c["out"] == "e4m3":
        y, scale, total = gdn.rms_norm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                                             weight_offset=c["offset"], group=c["group"])
        return {"y": y, "scale": scale, "sum": total}
    y, total = gdn.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, weight_offset=c["offset"])
    return {"y": y, "sum": total}


def _with_caches(s, out):
    if s["k_new"] is not None:
        out["k_cache"], out["v_cache"] = s["k_cache"], s["v_cache"]
    return out


def _plain_step(s):
    dt = s["q"].dtype
    q, k, v = (s[n].flatten(0, 1).float() for n in ("q", "k", "v"))
    g, beta = (s[n].flatten(0, 1) for n in ("g", "beta"))
    if s["A_log"] is not None:
        q, k = (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
        pre = g + s["dt_bias"]
        g = -torch.exp(s["A_log"]) * torch.where(pre > 20, pre, torch.log1p(torch.exp(pre.clamp(max=20))))
        beta = 1 / (1 + torch.exp(-beta))
    N, Hv = s["slots"].numel(), v.shape[1]
    G = Hv // q.shape[1]
    cu = s["cu_seqlens"]
    if cu is None:
        cu = torch.arange(N + 1, device=q.device) * (q.shape[0] // N)
    first, lens = cu[:-1].long(), (cu[1:] - cu[:-1])
    slots = s["slots"].long()
    h = s["state"][slots]
    o = torch.zeros_like(v)
    for t in range(s["case"]["tokens"]):  # the recurrence itself
        live = lens > t
        at = (first + t).clamp(max=q.shape[0] - 1)
        qt, kt = (x[at].repeat_interleave(G, 1) for x in (q, k))
        eg, b = torch.exp(g[at]), beta[at]
        u = b[..., None] * (v[at] - eg[..., None] * torch.matmul(kt[:, :, None, :], h)[:, :, 0])
        new = eg[..., None, None] * h + kt[..., :, None] * u[..., None, :]
        ot = s["scale"] * torch.matmul(qt[:, :, None, :], new)[:, :, 0]
        h = torch.where(live[:, None, None, None], new, h)
        o[at] = torch.where(live[:, None, None], ot, o[at])
    s["state_out"][slots] = h
    return {"o": o.to(dt).view(s["v"].shape), "state": s["state_out"]}


def _rows(cache, page, slot):
    """cache[page, slot] (8-bit types are gathered as bytes)."""
    if cache.element_size() == 1:
        return cache.view(torch.uint8)[page, slot].view(cache.dtype)
    return cache[page, slot]


def _plain_attn(s):
    q, lens, ps = s["q"], s["lens"].long(), s["k_cache"].shape[1]
    N, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    ks = s["k_scale"] if s["k_scale"] is not None else torch.ones(Hkv, device=q.device)
    vs = s["v_scale"] if s["v_scale"] is not None else torch.ones(Hkv, device=q.device)
    if s["k_new"] is not None:
        at = (lens - 1).clamp(min=0)
        page = s["table"].long().gather(1, (at // ps)[:, None])[:, 0]
        for cache, new, scale in ((s["k_cache"], s["k_new"], ks), (s["v_cache"], s["v_new"], vs)):
            row = new.float() / scale[:, None]
            if cache.dtype == FP8:
                cache.view(torch.uint8)[page, at % ps] = row.clamp(-FP8_MAX, FP8_MAX).to(FP8).view(torch.uint8)
            else:
                cache[page, at % ps] = row.to(cache.dtype)
    pos = torch.arange(s["case"]["most"], device=q.device)
    page = s["table"].long()[:, pos // ps]
    keys = _rows(s["k_cache"], page, pos % ps).float().permute(0, 2, 3, 1)  # [N, Hkv, D, L]
    score = torch.matmul(q.float().view(N, Hkv, Hq // Hkv, D), keys) * (ks[:, None, None] * s["scale"])
    seen = pos < lens[:, None]
    if s["window"]:
        seen &= pos >= lens[:, None] - s["window"]
    score = torch.where(seen[:, None, None], score, -torch.inf)
    some = (lens > 0)[:, None, None, None]
    top = torch.where(some, score.amax(-1, keepdim=True), 0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    values = _rows(s["v_cache"], page, pos % ps).float().permute(0, 2, 1, 3)  # [N, Hkv, L, D]
    o = torch.matmul(p, values) * vs[:, None, None] / torch.where(some, total, 1)
    lse = top + torch.log(total)
    return _with_caches(s, {"o": o.view(N, Hq, D).to(q.dtype), "lse": lse.view(N, Hq)})


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["weight"].float() + c["offset"]
    if s["residual"] is not None:
        x = x + s["residual"].float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    if c["backward"]:
        dy = s["dy"].float()
        xn, wdy = x * inv, dy * w
        dx = inv * (wdy - xn * (wdy * xn).mean(-1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        return {"dx": dx.to(dt), "dweight": (dy * xn).sum(0)}
    y = x * inv * w
    total = x.to(dt) if s["residual"] is not None else None
    if c["out"] == "e4m3":
        yg = y.view(c["rows"], -1, c["group"] or c["dim"])
        scale = (yg.abs().amax(-1) / FP8_MAX).clamp(min=FP8_TINY)
        return {"y": (yg / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).view_as(y).to(FP8), "scale": scale, "sum": total}
    return {"y": y.to(dt), "sum": total}


# ------------------------------------------------------------------------ bytes and flops
def work(case):
    c, e = case, BYTES[case["dtype"]]
    if c["op"] == "step":
        T, items = sum(_lengths(c, c["tokens"])), c["seqs"] * c["hv"]
        per_token = 2 * c["hqk"] * K * e + 2 * c["hv"] * V * e + 2 * c["hv"] * 4
        return {"bytes": items * 2 * K * V * 4 + T * per_token + 4 * c["seqs"],
                "flops": T * c["hv"] * 7 * K * V}
    if c["op"] == "attn":
        lens = _lengths(c, c["most"])
        seen = sum(min(x, c["window"]) if c["window"] else x for x in lens)
        act = 4 if c["dtype"] == "fp32" else 2
        rows = c["seqs"] * (2 * c["hq"] * c["dim"] * act + 4 * c["hq"])
        if c["append"]:  # the new rows are read from k_new and v_new, and written to the cache
            rows += c["seqs"] * 2 * c["hkv"] * c["dim"] * act
        pages = sum(-(-x // c["page"]) for x in lens)
        return {"bytes": seen * c["hkv"] * c["dim"] * 2 * e + rows + 4 * pages + 4 * c["seqs"],
                "flops": 4 * seen * c["hq"] * c["dim"]}
    n = c["rows"] * c["dim"]
    if c["backward"]:
        return {"bytes": n * e * (4 if c["residual"] else 3) + c["dim"] * (e + 4), "flops": 10 * n}
    scales = 4 * c["rows"] * (c["dim"] // c["group"] if c["group"] else 1) if c["out"] == "e4m3" else 0
    return {"bytes": n * (e * (3 if c["residual"] else 1) + BYTES[c["out"]]) + c["dim"] * e + scales, "flops": 6 * n}


# --------------------------------------------------------------------------------- fp64
def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "attn": _exact_attn, "norm": _exact_norm}[case["op"]](s)


def _exact_step(s):
    """S_t = e^g S (I - beta k k^T) + beta v k^T, o_t = scale S_t q_t with S = state^T, one
    sequence after another."""
    hqk, hv = s["q"].shape[2], s["v"].shape[2]
    out, o = s["state_out"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device=DEVICE).flatten(0, 1)
    t = 0
    for n, length in enumerate(s["lens"]):
        slot = int(s["slots"][n])
        S = s["state"][slot].double().transpose(1, 2)  # [Hv, V, K]
        for _ in range(length):
            q, k, v, g, b = (s[x].flatten(0, 1)[t].double() for x in ("q", "k", "v", "g", "beta"))
            if s["A_log"] is not None:
                q, k = (x / torch.sqrt(x.pow(2).sum(1, keepdim=True) + EPS) for x in (q, k))
                g = -s["A_log"].double().exp() * torch.logaddexp(g + s["dt_bias"].double(), torch.zeros_like(g))
                b = torch.sigmoid(b)
            q, k = (x.view(hqk, 1, K).expand(hqk, hv // hqk, K).reshape(hv, K) for x in (q, k))
            S = g.exp()[:, None, None] * S
            S = S + torch.einsum("hv,hk->hvk", b[:, None] * (v - torch.einsum("hvk,hk->hv", S, k)), k)
            o[t] = s["scale"] * torch.einsum("hvk,hk->hv", S, q)
            t += 1
        out[slot] = S.transpose(1, 2)
    return {"o": o.view(s["v"].shape), "state": out}


def _exact_attn(s):
    """softmax(scale q K^T) V, one sequence after another."""
    N, Hq, D = s["q"].shape
    ps, hkv = s["k_cache"].shape[1], s["k_cache"].shape[2]
    o = torch.zeros(N, Hq, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device=DEVICE)
    scales = {n: s[n].double() if s[n] is not None else torch.ones(hkv, dtype=torch.float64, device=DEVICE)
              for n in ("k_scale", "v_scale")}
    caches = [s["k_cache"], s["v_cache"]]
    for n, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        if s["k_new"] is not None:
            page, slot = int(s["table"][n, (length - 1) // ps]), (length - 1) % ps
            for cache, new, sc in ((caches[0], s["k_new"], "k_scale"), (caches[1], s["v_new"], "v_scale")):
                row = new[n].double() / scales[sc][:, None]
                if cache.dtype == FP8:
                    row = row.clamp(-FP8_MAX, FP8_MAX)
                cache[page, slot] = row.float().to(cache.dtype)
        first = max(0, length - s["window"]) if s["window"] else 0
        pages = s["table"][n, first // ps:-(-length // ps)].long()
        skip = first - first // ps * ps
        k, v = (_whole(c, pages)[skip:skip + length - first].double() * scales[sc][:, None]
                for c, sc in zip(caches, ("k_scale", "v_scale")))
        qn = s["q"][n].double().view(hkv, Hq // hkv, D)
        z = s["scale"] * torch.einsum("hgd,lhd->hgl", qn, k)
        lse[n] = torch.logsumexp(z, -1).flatten()
        o[n] = torch.einsum("hgl,lhd->hgd", torch.softmax(z, -1), v).reshape(Hq, D)
    out = {"o": o, "lse": lse}
    if s["k_new"] is not None:
        out["k_cache"], out["v_cache"] = (c.to(torch.float64) for c in caches)
    return out


def _whole(cache, pages):
    """The given pages' tokens, one after another: [tokens, Hkv, D]."""
    if cache.element_size() == 1:
        return cache.view(torch.uint8)[pages].view(cache.dtype).flatten(0, 1)
    return cache[pages].flatten(0, 1)


def _exact_norm(s):
    c = s["case"]
    rows, dim = c["rows"], c["dim"]
    w = s["weight"].double() + c["offset"]
    parts, dw = [], torch.zeros(dim, dtype=torch.float64, device=DEVICE)
    step = max(1, (1 << 25) // dim)
    for i in range(0, rows, step):
        x = s["x"][i:i + step].double()
        if s["residual"] is not None:
            x = x + s["residual"][i:i + step].double()
        r = torch.sqrt(x.pow(2).sum(1, keepdim=True) / dim + EPS)
        if c["backward"]:
            dy = s["dy"][i:i + step].double()
            dx = dy * w / r - x * (dy * w * x).sum(1, keepdim=True) / (dim * r ** 3)
            if s["dsum"] is not None:
                dx = dx + s["dsum"][i:i + step].double()
            dw += (dy * x / r).sum(0)
            parts.append((dx,))
            continue
        y = x / r * w
        total = x if s["residual"] is not None else None
        if c["out"] == "e4m3":
            y = y.view(y.shape[0], -1, c["group"] or dim)
            scale = (y.abs().amax(2) / FP8_MAX).clamp(min=FP8_TINY)
            parts.append(((y / scale[:, :, None]).reshape(-1, dim), scale, total))
        else:
            parts.append((y, total))
    got = [None if p[0] is None else torch.cat(p) for p in zip(*parts)]
    if c["backward"]:
        return {"dx": got[0], "dweight": dw}
    return dict(zip(("y", "scale", "sum") if c["out"] == "e4m3" else ("y", "sum"), got))
