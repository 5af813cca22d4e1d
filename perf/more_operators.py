"""Measured cases of the operators around a key-value cache, from a prompt to drafted tokens:

  prompt  gdn.prompt_attention        causal attention over whole prompts, with its backward pass
  tree    gdn.paged_attention_tree    a tree of drafted tokens over a paged key-value cache
  write   gdn.paged_cache_write       keys and values written to slots of a paged cache
  table   gdn.page_table_extend, gdn.page_table_trim
                                      page tables and slots from the requests' lengths

``run`` makes the library's calls where ``own`` is true and computes the same results from
elementary tensor operations in fp32 elsewhere; ``exact`` computes them in fp64 from the
definitions.  All inputs come from ``prepare``'s seed; head counts, features and pages are those of
the library's workloads and of its decoding operators' cases.
"""
import math
import random

import torch

own = False
DEVICE = "cuda"

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": FP8}
BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}
ROOM = 1 << 28  # values of a temporary of the plain forms


def listed():
    prompt = dict(op="prompt", ragged=False, prior=0, window=0, packed=False, backward=False, dtype="bf16")
    tree = dict(op="tree", ragged=True, window=0, heads_first=False, dtype="bf16")
    write = dict(op="write", heads_first=False, picked=False)
    return [
        # two short questions in full precision: latency counts
        dict(prompt, name="prompt_short", seqs=2, most=100, hq=8, hkv=2, dim=64, dtype="fp32"),
        # a served batch of prompts of uneven lengths, views of the fused projection's rows
        dict(prompt, name="prompt_packed", seqs=24, most=4000, ragged=True, hq=32, hkv=8, dim=128, packed=True),
        # the last part of a long document whose earlier keys are there, wide heads
        dict(prompt, name="prompt_long", seqs=1, most=8192, prior=24001, hq=16, hkv=2, dim=256),
        # a training step of one long row
        dict(prompt, name="prompt_grad", seqs=1, most=8192, hq=32, hkv=4, dim=128, backward=True),
        # a training step of packed documents of uneven lengths
        dict(prompt, name="prompt_grad_packed", seqs=16, most=2047, ragged=True, hq=24, hkv=8, dim=64, packed=True, backward=True),
        # a few chats with eight drafted tokens each, wide heads
        dict(tree, name="tree_few", seqs=4, nodes=8, most=700, hq=16, hkv=2, dim=256, page=16),
        # a served batch of uneven lengths, sixteen drafted tokens
        dict(tree, name="tree_batch", seqs=32, nodes=16, most=8192, hq=32, hkv=8, dim=128, page=16),
        # a large batch over an 8-bit cache, pages that are no power of two, heads before tokens
        dict(tree, name="tree_fp8", seqs=64, nodes=31, most=16384, hq=64, hkv=8, dim=128, page=48, dtype="e4m3", heads_first=True),
        # the accepted ones of a batch's drafted tokens
        dict(write, name="write_accepted", tokens=96, hkv=8, dim=128, page=16, dtype="bf16", picked=True),
        # a prompt's keys and values into an 8-bit cache
        dict(write, name="write_prompt", tokens=32767, hkv=8, dim=128, page=48, dtype="e4m3", heads_first=True),
        # one more token for each of a batch
        dict(op="table", name="table_step", seqs=256, most=8192, new=1, page=16, short=False),
        # prompts of uneven lengths, more than there are pages for
        dict(op="table", name="table_prompts", seqs=500, most=0, new=2000, page=64, short=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "write", "table"])
    heads = [(4, 4), (8, 1), (16, 2), (24, 8), (32, 4), (32, 8), (64, 8), (40, 1)]
    if op == "prompt":
        hq, hkv = rng.choice(heads)
        dim = rng.choice([64, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        backward = rng.random() < 0.5
        seqs = _log(rng, 1, 64)
        # a pass's products stay below the largest listed case's
        room = (1 << 38) // (hq * dim) // (4 if backward else 1) // (8 if dtype == "fp32" else 1)
        prior = rng.choice([0, 0, _log(rng, 1, math.sqrt(room / seqs) + 1)])
        most = _log(rng, 1, min(60000 // seqs, math.sqrt(room / seqs + prior * prior / 4) - prior / 2 + 1))
        return dict(op=op, seqs=seqs, most=most, hq=hq, hkv=hkv, dim=dim, prior=prior, ragged=rng.random() < 0.6,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), packed=prior == 0 and rng.random() < 0.5,
                    backward=backward, dtype=dtype)
    if op == "tree":
        hq, hkv = rng.choice(heads)
        dim = rng.choice([64, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "bf16", "e4m3", "e4m3", "fp32"])
        nodes = rng.choice([_log(rng, 1, 64), rng.randint(2, 32)])
        seqs = _log(rng, 1, 128)
        tokens = min((3 << 28) // (hkv * dim * BYTES[dtype]), (1 << 35) // (nodes * hq * dim) // (4 if dtype == "fp32" else 1))
        return dict(op=op, seqs=seqs, nodes=nodes, most=_log(rng, 1, min(130000, tokens // seqs)), hq=hq, hkv=hkv, dim=dim,
                    page=rng.choice([1, 16, 24, 32, 64, 100, 256]), ragged=rng.random() < 0.7,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), heads_first=rng.random() < 0.3, dtype=dtype)
    if op == "write":
        hkv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, (1 << 25) // (hkv * dim)), hkv=hkv, dim=dim, page=rng.choice([1, 16, 24, 48, 64, 100, 256]),
                    heads_first=rng.random() < 0.3, picked=rng.random() < 0.4, dtype=rng.choice(["bf16", "e4m3", "fp32"]))
    seqs = _log(rng, 1, 2000)
    return dict(op=op, seqs=seqs, most=rng.choice([0, _log(rng, 1, 20000)]), new=rng.choice([1, rng.randint(2, 64), _log(rng, 1, 1 + 400000 // seqs)]),
                page=rng.choice([1, 16, 24, 48, 64, 100, 256]), short=rng.random() < 0.3)


def _some(n, most, least, key):
    """n whole numbers between `least` and `most`, the first of them `most`."""
    r = random.Random(key)
    got = [r.randint(min(least, most), most) for _ in range(n)]
    if n:
        got[0] = most
    return got


def _lengths(case):
    """Tokens per sequence: `most` throughout, or uneven, a row of a captured batch empty."""
    n = case["seqs"]
    if not case["ragged"]:
        return [case["most"]] * n
    got = _some(n, case["most"], 0, n * 1000003 + case["most"])
    if n > 2:
        got[1] = 0
    return got


def _priors(case):
    """Keys that each sequence has before its first query."""
    if not case["ragged"]:
        return [case["prior"]] * case["seqs"]
    return _some(case["seqs"], case["prior"], 0, case["seqs"] * 7919 + case["prior"])


def _prompt_lengths(case, seed=None):
    got = list(zip(_lengths(case), _priors(case)))
    if seed is not None:
        random.Random(seed).shuffle(got)
    return got


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=DEVICE)  # noqa: E731
    return {"prompt": _prepare_prompt, "tree": _prepare_tree, "write": _prepare_write, "table": _prepare_table}[case["op"]](case, seed, gen, randn)


def _starts(lens):
    got = [0]
    for x in lens:
        got.append(got[-1] + x)
    return got


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _prepare_prompt(c, seed, gen, randn):
    dt, n, hq, hkv, D = TYPES[c["dtype"]], c["seqs"], c["hq"], c["hkv"], c["dim"]
    lens = _prompt_lengths(c, seed)
    cu, cu_k = _starts([x for x, _ in lens]), _starts([x + y for x, y in lens])
    B, T, Tk = (1, cu[-1], cu_k[-1]) if c["ragged"] else (n, c["most"], c["most"] + c["prior"])
    if c["packed"]:
        x = randn(B * T, (hq + 2 * hkv) * D)
        x[:, :hq * D] *= 1.5
        q, k, v = (p.unflatten(-1, (-1, D)).unflatten(0, (B, T)) for p in x.to(dt).split([hq * D, hkv * D, hkv * D], -1))
    else:
        q, k, v = (1.5 * randn(B, T, hq, D)).to(dt), randn(B, Tk, hkv, D).to(dt), randn(B, Tk, hkv, D).to(dt)
    s = dict(case=c, q=q, k=k, v=v, scale=D ** -0.5, lens=lens, cu=cu, cu_k=cu_k, cu_seqlens=None, cu_seqlens_k=None, do=None)
    if c["ragged"]:
        s["cu_seqlens"] = _int32(cu)
        if c["prior"]:
            s["cu_seqlens_k"] = _int32(cu_k)
    if c["backward"]:
        s["do"] = randn(B, T, hq, D).to(dt)
    return s


def _pages(gen, used, spare):
    """A table of `used` pages per row, drawn without order, and the number of pages."""
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.zeros(len(used), max(max(used), 1), dtype=torch.int32, device=DEVICE)
    have = torch.arange(table.shape[1], device=DEVICE) < torch.tensor(used, device=DEVICE)[:, None]
    table[have] = order[:sum(used)]
    return table, pages


def _cache(c, pages, randn):
    shape = (pages, c["hkv"], c["page"], c["dim"]) if c["heads_first"] else (pages, c["page"], c["hkv"], c["dim"])
    x = torch.empty(shape, dtype=TYPES[c["dtype"]], device=DEVICE)
    step = max(1, (1 << 27) // max(1, x[0].numel()))
    for i in range(0, pages, step):  # in parts: the fp32 draws of a whole cache need not fit beside it
        m = min(step, pages - i)
        x[i:i + m] = randn(m, *shape[1:]).to(x.dtype)
    return x.transpose(1, 2) if c["heads_first"] else x


def _trees(c, seed):
    """Parents of every sequence's drafted tokens: -1 below the cached ones, -2 where there are fewer."""
    r = random.Random(seed)
    nodes = _some(c["seqs"], c["nodes"], 1, c["seqs"] * 31 + c["nodes"]) if c["ragged"] else [c["nodes"]] * c["seqs"]
    r.shuffle(nodes)
    return [[r.choice([t - 1, r.randint(max(-1, t - 6), t - 1)]) for t in range(m)] + [-2] * (c["nodes"] - m) for m in nodes]


def _prepare_tree(c, seed, gen, randn):
    n, T, hq, hkv, D = c["seqs"], c["nodes"], c["hq"], c["hkv"], c["dim"]
    lens = _lengths(c)
    random.Random(seed).shuffle(lens)
    table, pages = _pages(gen, [-(-x // c["page"]) for x in lens], 1 + n // 8)
    act = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    trees = _trees(c, seed)
    s = dict(case=c, q=(1.5 * randn(n, T, hq, D)).to(act), k_new=randn(n, T, hkv, D).to(act), v_new=randn(n, T, hkv, D).to(act),
             k_cache=_cache(c, pages, randn), v_cache=_cache(c, pages, randn), table=table, lens=_int32(lens), parents=_int32(trees),
             scale=D ** -0.5, window=c["window"], k_scale=None, v_scale=None, host_lens=lens, host_parents=trees)
    if c["dtype"] == "e4m3":
        s["k_scale"], s["v_scale"] = (0.5 + torch.rand(hkv, generator=gen, device=DEVICE) for _ in range(2))
    return s


def _prepare_write(c, seed, gen, randn):
    n, hkv, D = c["tokens"], c["hkv"], c["dim"]
    pages = -(-n // c["page"]) + 8
    act = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    slots = torch.randperm(pages, generator=gen, device=DEVICE)[:, None] * c["page"] + torch.arange(c["page"], device=DEVICE)
    slots = slots.flatten()[:n].contiguous()
    slots[3::97] = -1  # tokens of a request that there were no pages for
    rows = n
    if c["picked"]:
        rows = 2 * n + 1
    s = dict(case=c, k=randn(rows, hkv, D).to(act), v=randn(rows, hkv, D).to(act), slots=slots, rows=None,
             k_cache=_cache(c, pages, randn), v_cache=_cache(c, pages, randn), k_scale=None, v_scale=None)
    if c["picked"]:
        s["rows"] = torch.randperm(rows, generator=gen, device=DEVICE)[:n].sort().values.to(torch.int32)
    if c["dtype"] == "e4m3":
        s["k_scale"], s["v_scale"] = (0.5 + torch.rand(hkv, generator=gen, device=DEVICE) for _ in range(2))
    return s


def _table_lengths(c):
    have = _some(c["seqs"], c["most"], 0, c["seqs"] * 13 + c["most"])
    new = [c["new"]] * c["seqs"] if c["new"] == 1 else _some(c["seqs"], c["new"], 0, c["seqs"] * 17 + c["new"])
    need = sum(-(-(x + y) // c["page"]) - -(-x // c["page"]) for x, y in zip(have, new))
    return have, new, need * 3 // 4 if c["short"] else need + 5


def _prepare_table(c, seed, gen, randn):
    have, new, free = _table_lengths(c)
    both = list(zip(have, new))
    random.Random(seed).shuffle(both)
    have, new = [x for x, _ in both], [y for _, y in both]
    used = [-(-x // c["page"]) for x in have]
    table, pages = _pages(gen, used, free)
    most = max(-(-(x + y) // c["page"]) for x, y in both)
    wide = torch.zeros(c["seqs"], max(most, 1), dtype=torch.int32, device=DEVICE)
    wide[:, :min(table.shape[1], wide.shape[1])] = table[:, :wide.shape[1]]
    taken = torch.zeros(pages, dtype=torch.bool, device=DEVICE)
    inside = torch.arange(table.shape[1], device=DEVICE) < torch.tensor(used, device=DEVICE)[:, None]
    taken[table[inside].long()] = True
    stack = torch.zeros(pages, dtype=torch.int32, device=DEVICE)
    left = (~taken).nonzero()[:, 0].to(torch.int32)
    stack[:left.numel()] = left[torch.randperm(left.numel(), generator=gen, device=DEVICE)]
    return dict(case=c, table=wide, lens=_int32(have), new=_int32(new), before=_int32(have), stack=stack, free=_int32([free]), total=sum(new))


# ------------------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "tree": _own_tree, "write": _own_write, "table": _own_table}[kind](state)
    return {"prompt": _plain_prompt, "tree": _plain_tree, "write": _plain_write, "table": _plain_table}[kind](state)


def _own_prompt(s):
    from chunked_prefill_gb300 import gdn
    c = s["case"]
    args = dict(scale=s["scale"], window=c["window"], cu_seqlens=s["cu_seqlens"], cu_seqlens_k=s["cu_seqlens_k"])
    if not c["backward"]:
        o, lse = gdn.prompt_attention(s["q"], s["k"], s["v"], return_lse=True, **args)
        return {"o": o, "lse": lse}
    q, k, v = (s[n].detach().requires_grad_() for n in ("q", "k", "v"))
    o = gdn.prompt_attention(q, k, v, **args)
    dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["do"])
    return {"o": o.detach(), "dq": dq, "dk": dk, "dv": dv}


def _own_tree(s):
    from chunked_prefill_gb300 import gdn
    o, lse = gdn.paged_attention_tree(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["parents"],
                                      scale=s["scale"], window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], return_lse=True)
    return {"o": o, "lse": lse}


def _own_write(s):
    from chunked_prefill_gb300 import gdn
    gdn.paged_cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], rows=s["rows"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_table(s):
    """Room for the new tokens, and the same pages given back: all of them were refused."""
    from chunked_prefill_gb300 import gdn
    page = s["case"]["page"]
    slots, cu = gdn.page_table_extend(s["table"], s["lens"], s["new"], s["stack"], s["free"], page, s["total"])
    grown = s["lens"].clone()
    gdn.page_table_trim(s["table"], s["lens"], s["before"], s["stack"], s["free"], page)
    return {"slots": slots, "cu_seqlens": cu, "grown": grown, "table": s["table"], "lens": s["lens"], "stack": s["stack"], "free": s["free"]}


def _plain_prompt(s):
    c, dt = s["case"], s["q"].dtype
    q, k, v = (s[n].flatten(0, 1) for n in ("q", "k", "v"))
    do = s["do"].flatten(0, 1) if c["backward"] else None
    T, hq, D = q.shape
    hkv, G = k.shape[1], hq // k.shape[1]
    o = torch.zeros(T, hq, D, device=q.device)
    lse = torch.full((T, hq), -torch.inf, device=q.device)
    if c["backward"]:
        dq, dk, dv = (torch.zeros(x.shape, device=q.device) for x in (q, k, v))
    for n, (length, prior) in enumerate(s["lens"]):
        Lk = length + prior
        if length == 0:
            continue
        ks = slice(s["cu_k"][n], s["cu_k"][n] + Lk)
        kf, vf = (x[ks].float().transpose(0, 1) for x in (k, v))  # [hkv, Lk, D]
        at = torch.arange(Lk, device=q.device)
        step = max(1, ROOM // (hq * Lk))
        for i in range(0, length, step):
            m = min(step, length - i)
            rows = slice(s["cu"][n] + i, s["cu"][n] + i + m)
            heads = lambda x: x[rows].float().view(m, hkv, G, D).permute(1, 2, 0, 3).reshape(hkv, G * m, D)  # noqa: E731
            back = lambda x: x.view(hkv, G, m, D).permute(2, 0, 1, 3).reshape(m, hq, D)  # noqa: E731
            qf = heads(q)
            z = (torch.matmul(qf, kf.transpose(1, 2)) * s["scale"]).view(hkv, G, m, Lk)
            own_at = torch.arange(i, i + m, device=q.device)[:, None] + prior
            seen = at <= own_at
            if c["window"]:
                seen &= at > own_at - c["window"]
            z = torch.where(seen, z, -torch.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - top)
            total = p.sum(-1, keepdim=True)
            p = (p / total).view(hkv, G * m, Lk)
            o[rows] = back(torch.matmul(p, vf))
            lse[rows] = (top + torch.log(total)).view(hq, m).t()
            if c["backward"]:
                dof = heads(do)
                dp = torch.matmul(dof, vf.transpose(1, 2))
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
                dq[rows] = back(torch.matmul(ds, kf))
                dk[ks] += torch.matmul(ds.transpose(1, 2), qf).transpose(0, 1)
                dv[ks] += torch.matmul(p.transpose(1, 2), dof).transpose(0, 1)
    if not c["backward"]:
        return {"o": o.to(dt).view(s["q"].shape), "lse": lse.view(s["q"].shape[:3])}
    return {"o": o.to(dt).view(s["q"].shape), "dq": dq.to(dt).view(s["q"].shape), "dk": dk.to(dt).view(s["k"].shape), "dv": dv.to(dt).view(s["v"].shape)}


def _rows(cache, page, slot):
    """cache[page, slot] (8-bit types are gathered as bytes)."""
    if cache.element_size() == 1:
        return cache.view(torch.uint8)[page, slot].view(cache.dtype)
    return cache[page, slot]


def _plain_tree(s):
    c = s["case"]
    N, T, Hq, D = s["q"].shape
    Hkv, page = c["hkv"], c["page"]
    G, dev = Hq // Hkv, s["q"].device
    ks = s["k_scale"] if s["k_scale"] is not None else torch.ones(Hkv, device=dev)
    vs = s["v_scale"] if s["v_scale"] is not None else torch.ones(Hkv, device=dev)
    # which drafted tokens each sees, and how deep it lies
    nodes = torch.arange(T, device=dev)
    parents = s["parents"].long()
    live = parents >= -1
    sees = torch.zeros(N, T, T, dtype=torch.bool, device=dev)
    depth = torch.zeros(N, T, dtype=torch.long, device=dev)
    up = nodes.expand(N, T)
    for _ in range(T):
        sees |= (up[..., None] == nodes) & live[..., None]
        up = torch.where(up >= 0, parents.gather(1, up.clamp(min=0)), up)
        depth += (up >= 0) & live
    L = c["most"]
    o = torch.zeros(N, T, Hq, D, device=dev)
    lse = torch.full((N, T, Hq), -torch.inf, device=dev)
    step = max(1, 4 * ROOM // max(1, L * Hkv * max(D, T * G)))
    for i in range(0, N, step):
        m = min(step, N - i)
        sl = slice(i, i + m)
        pos = torch.arange(L, device=dev)
        pages = s["table"][sl].long()[:, pos // page] if L else pos.expand(m, 0)
        gather = lambda cache: _rows(cache, pages, pos % page).float()  # noqa: E731
        keys = torch.cat([gather(s["k_cache"]) * ks[:, None], s["k_new"][sl].float()], 1).permute(0, 2, 3, 1)  # [m, Hkv, D, L + T]
        qf = s["q"][sl].float().view(m, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(m, Hkv, T * G, D)
        z = (torch.matmul(qf, keys) * s["scale"]).view(m, Hkv, T, G, L + T)
        lens, deep, lv = s["lens"][sl].long(), depth[sl], live[sl]
        cached = (pos < lens[:, None])[:, None, :] & lv[..., None]
        new = sees[sl]
        if c["window"]:
            own_at = (lens[:, None] + deep)[..., None]
            cached = cached & (pos > own_at - c["window"])
            new = new & (deep[:, None, :] > deep[..., None] - c["window"])
        seen = torch.cat([cached, new], -1)[:, None, :, None, :]
        z = torch.where(seen, z, -torch.inf)
        top = z.amax(-1, keepdim=True)
        top = torch.where(lv[:, None, :, None, None], top, 0)
        p = torch.exp(z - top)
        total = p.sum(-1, keepdim=True)
        values = torch.cat([gather(s["v_cache"]) * vs[:, None], s["v_new"][sl].float()], 1).permute(0, 2, 1, 3)  # [m, Hkv, L + T, D]
        x = torch.matmul(p.view(m, Hkv, T * G, L + T), values).view(m, Hkv, T, G, D) / torch.where(total > 0, total, 1)
        o[sl] = x.permute(0, 2, 1, 3, 4).reshape(m, T, Hq, D)
        lse[sl] = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(m, T, Hq)
    return {"o": o.to(s["q"].dtype), "lse": lse}


def _plain_write(s):
    page = s["case"]["page"]
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    rows = (s["rows"].long() if s["rows"] is not None else torch.arange(keep.numel(), device=keep.device))[keep]
    for name in ("k", "v"):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        x = s[name][rows].float()
        if scale is not None:
            x = x / scale[:, None]
        if cache.dtype == FP8:
            cache.view(torch.uint8)[at // page, at % page] = x.clamp(-FP8_MAX, FP8_MAX).to(FP8).view(torch.uint8)
        else:
            cache[at // page, at % page] = x.to(cache.dtype)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_table(s):
    page, table, dev = s["case"]["page"], s["table"], s["table"].device
    lens, new, stack, free = s["lens"].long(), s["new"].long(), s["stack"], s["free"].long()
    N, width = table.shape
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), new.cumsum(0)])
    had = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - had
    need = torch.where(lens + new <= width * page, need, 0)
    upto = need.cumsum(0)
    first = upto - need  # pages taken before
    granted = (lens + new <= width * page) & ((need == 0) | (upto <= free))
    # pages: the top of the stack goes to the first sequence's first one
    columns = torch.arange(width, device=dev)
    mine = granted[:, None] & (columns >= had[:, None]) & (columns < (had + need)[:, None])
    order = (free - 1 - first[:, None] - (columns - had[:, None])).clamp(min=0)
    table.copy_(torch.where(mine, stack[order], table))
    t = torch.arange(s["total"], device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = lens[seq] + t - cu[seq]
    slots = torch.where(granted[seq], table[seq, (at // page).clamp(max=width - 1)].long() * page + at % page, -1)
    s["lens"].copy_(torch.where(granted, lens + new, lens))
    grown = s["lens"].clone()
    taken = torch.where(granted, need, 0)
    # and given back, the last one first: the stack is as it was
    keep = torch.minimum(s["lens"], s["before"]).long()
    kept, has = (keep + page - 1) // page, (grown.long() + page - 1) // page
    give = has - kept
    behind = give.flip(0).cumsum(0).flip(0) - give  # pages given by the sequences after
    mine = (columns >= kept[:, None]) & (columns < has[:, None])
    left = free - taken.sum()
    order = left + behind[:, None] + (has[:, None] - 1 - columns)
    stack[order[mine]] = table[mine]
    s["free"].copy_(left + give.sum())
    s["lens"].copy_(keep)
    return {"slots": slots, "cu_seqlens": cu.to(torch.int32), "grown": grown, "table": table, "lens": s["lens"], "stack": stack, "free": s["free"]}


# ------------------------------------------------------------------------ bytes and flops
def _seen(length, prior, window):
    """(query, key) pairs of a sequence."""
    if window == 0:
        return length * prior + length * (length + 1) // 2
    full = max(0, min(length, window - prior))  # queries that see everything before them
    return full * prior + full * (full + 1) // 2 + (length - full) * window


def work(case):
    c = case
    if c["op"] == "prompt":
        e, lens = BYTES[c["dtype"]], _prompt_lengths(c)
        pairs = sum(_seen(x, y, c["window"]) for x, y in lens)
        q, k = (sum(n) * h * c["dim"] * e for n, h in (([x for x, _ in lens], c["hq"]), ([x + y for x, y in lens], c["hkv"])))
        if c["backward"]:  # q, k, v, do in; o, dq, dk, dv out
            return {"bytes": 4 * q + 4 * k, "flops": 14 * pairs * c["hq"] * c["dim"]}
        return {"bytes": 2 * q + 2 * k + 4 * c["hq"] * sum(x for x, _ in lens), "flops": 4 * pairs * c["hq"] * c["dim"]}
    if c["op"] == "tree":
        lens, act = _lengths(c), 4 if c["dtype"] == "fp32" else 2
        seen = [min(x, c["window"]) if c["window"] else x for x in lens]
        rows = c["seqs"] * c["nodes"] * (c["dim"] * act * (2 * c["hq"] + 2 * c["hkv"]) + 4 * c["hq"] + 4)
        nodes = _some(c["seqs"], c["nodes"], 1, c["seqs"] * 31 + c["nodes"]) if c["ragged"] else [c["nodes"]] * c["seqs"]
        return {"bytes": sum(seen) * c["hkv"] * c["dim"] * 2 * BYTES[c["dtype"]] + rows + 4 * sum(-(-x // c["page"]) for x in seen),
                "flops": 4 * c["hq"] * c["dim"] * sum(seen) * sum(nodes) // c["seqs"]}
    if c["op"] == "write":
        act = 4 if c["dtype"] == "fp32" else 2
        per = c["hkv"] * c["dim"]
        return {"bytes": c["tokens"] * (2 * per * (act + BYTES[c["dtype"]]) + 8 + (4 if c["picked"] else 0)), "flops": 2 * per * c["tokens"]}
    have, new, free = _table_lengths(c)
    need = min(free, sum(-(-(x + y) // c["page"]) - -(-x // c["page"]) for x, y in zip(have, new)))
    return {"bytes": 8 * sum(new) + 4 * 4 * need + 8 * 4 * c["seqs"], "flops": 4 * sum(new) + 16 * c["seqs"]}


# --------------------------------------------------------------------------------- fp64
def exact(case, seed):
    if case["op"] == "prompt" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "tree": _exact_tree, "write": _exact_write, "table": _exact_table}[case["op"]](s)


def _exact_prompt(s):
    """Per sequence and head: softmax(scale q K^T) V over the keys up to the query's own, and the
    gradients of <o, do>."""
    c = s["case"]
    q, k, v = (s[n].flatten(0, 1) for n in ("q", "k", "v"))
    T, hq, D = q.shape
    G = hq // k.shape[1]
    double = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=DEVICE)  # noqa: E731
    o, dq, dk, dv = double(q), double(q), double(k), double(v)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=DEVICE)
    q0 = k0 = 0
    for length, prior in s["lens"]:
        for h in range(hq if length else 0):
            j = h // G
            K, V = k[k0:k0 + length + prior, j].double(), v[k0:k0 + length + prior, j].double()
            step = 4096
            for i in range(0, length, step):
                a, b = i, min(length, i + step)
                end = prior + b  # no query of this part sees a later key
                start = max(0, prior + a + 1 - c["window"]) if c["window"] else 0
                Q = q[q0 + a:q0 + b, h].double()
                z = s["scale"] * (Q @ K[start:end].T)
                ahead = (torch.arange(start, end, device=DEVICE) - prior)[None, :] - torch.arange(a, b, device=DEVICE)[:, None]
                hidden = ahead > 0
                if c["window"]:
                    hidden |= ahead <= -c["window"]
                z.masked_fill_(hidden, -math.inf)
                w = torch.softmax(z, 1)
                lse[q0 + a:q0 + b, h] = torch.logsumexp(z, 1)
                out = w @ V[start:end]
                o[q0 + a:q0 + b, h] = out
                if c["backward"]:
                    g = s["do"].flatten(0, 1)[q0 + a:q0 + b, h].double()
                    dv[k0 + start:k0 + end, j] += w.T @ g
                    dz = s["scale"] * w * (g @ V[start:end].T - (g * out).sum(1, keepdim=True))
                    dq[q0 + a:q0 + b, h] = dz @ K[start:end]
                    dk[k0 + start:k0 + end, j] += dz.T @ Q
        q0 += length
        k0 += length + prior
    if c["backward"]:
        return {"o": o.view(s["q"].shape), "dq": dq.view(s["q"].shape), "dk": dk.view(s["k"].shape), "dv": dv.view(s["v"].shape)}
    return {"o": o.view(s["q"].shape), "lse": lse.view(s["q"].shape[:3])}


def _exact_tree(s):
    """Per sequence: every drafted token over the cached ones, its ancestors and itself."""
    c = s["case"]
    N, T, Hq, D = s["q"].shape
    Hkv, W = c["hkv"], c["window"]
    one = torch.ones(Hkv, dtype=torch.float64, device=DEVICE)
    ks, vs = (one if s[n] is None else s[n].double() for n in ("k_scale", "v_scale"))
    o = torch.zeros(N, T, Hq, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((N, T, Hq), -math.inf, dtype=torch.float64, device=DEVICE)
    for n, length in enumerate(s["host_lens"]):
        pages = s["table"][n, :-(-length // c["page"])].long()

        def whole(cache, scale, new):
            got = cache.view(torch.uint8)[pages].view(cache.dtype) if cache.element_size() == 1 else cache[pages]
            return torch.cat([got.flatten(0, 1)[:length].double() * scale[:, None], new[n].double()])

        k, v = whole(s["k_cache"], ks, s["k_new"]), whole(s["v_cache"], vs, s["v_new"])
        hide, depths = [], []
        for t, parent in enumerate(s["host_parents"][n]):
            line = [t]
            while parent >= 0:
                line.append(parent)
                parent = s["host_parents"][n][parent]
            depths.append(len(line) - 1)
            hide.append([x not in line or (W and depths[x] <= depths[t] - W) for x in range(T)])
        rows = [t for t in range(T) if s["host_parents"][n][t] >= -1]
        if not rows:
            continue
        mask = torch.zeros(len(rows), length + T, dtype=torch.bool, device=DEVICE)
        mask[:, length:] = torch.tensor(hide, device=DEVICE)[rows]
        if W:
            at = length + torch.tensor(depths, device=DEVICE)[rows]
            mask[:, :length] |= torch.arange(length, device=DEVICE) <= at[:, None] - W
        z = s["scale"] * torch.einsum("thgd,lhd->hgtl", s["q"][n, rows].double().view(len(rows), Hkv, -1, D), k)
        z = z.masked_fill(mask, -math.inf)
        lse[n, rows] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(len(rows), Hq)
        o[n, rows] = torch.einsum("hgtl,lhd->thgd", torch.softmax(z, -1), v).reshape(len(rows), Hq, D)
    return {"o": o, "lse": lse}


def _exact_write(s):
    page, out = s["case"]["page"], {}
    for name in ("k", "v"):
        cache = s[name + "_cache"].to(torch.float64)
        x = s[name].double() if s["rows"] is None else s[name].double()[s["rows"].long()]
        if s[name + "_scale"] is not None:
            x = x / s[name + "_scale"].double()[:, None]
        if s[name + "_cache"].dtype == FP8:
            x = x.clamp(-FP8_MAX, FP8_MAX)
        there = torch.nonzero(s["slots"] >= 0)[:, 0]
        cache[torch.div(s["slots"][there], page, rounding_mode="floor"), s["slots"][there] % page] = x[there]
        out[name + "_cache"] = cache
    return out


def _exact_table(s):
    """One request after another, with the free pages as a list."""
    page = s["case"]["page"]
    table, lens, new, stack = s["table"].tolist(), s["lens"].tolist(), s["new"].tolist(), s["stack"].tolist()
    free = int(s["free"])
    cu, slots, asked, top, grown = [0], [], 0, free, []
    for n in range(len(lens)):
        have, want = -(-lens[n] // page), -(-(lens[n] + new[n]) // page)
        fits = lens[n] + new[n] <= len(table[n]) * page
        asked += want - have if fits else 0
        granted = fits and (want == have or asked <= free)
        if granted:
            for column in range(have, want):
                top -= 1
                table[n][column] = stack[top]
            slots += [table[n][x // page] * page + x % page for x in range(lens[n], lens[n] + new[n])]
        else:
            slots += [-1] * new[n]
        grown.append(lens[n] + new[n] if granted else lens[n])
        cu.append(cu[-1] + new[n])
    # giving the same pages back leaves lengths, stack and count as they were
    return {"slots": torch.tensor(slots, dtype=torch.int64, device=DEVICE), "cu_seqlens": _int32(cu), "grown": _int32(grown),
            "table": _int32(table), "lens": s["lens"], "stack": s["stack"], "free": s["free"]}
