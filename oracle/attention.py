"""fp64 NumPy oracles of attention over prompts with its gradient, of drafted trees over a paged cache, of
writing that cache and of its page tables.  Written from the definitions; test infrastructure only."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _visible(lq, lk, window):
    at = np.arange(lq)[:, None] + lk - lq
    t = np.arange(lk)[None, :]
    seen = t <= at
    return seen & (t > at - window) if window else seen


def prompt(q, k, v, cu, cu_k, scale, window=0, do=None, dlse=None):
    """q [Tq,Hq,D], k, v [Tk,Hkv,D] packed by cu, cu_k.  Returns a dict of o, lse (and dq, dk, dv with do) and of
    the sizes that their rounding errors go with:
      reach [Tq,Hq]     max_t scale sum_d |q_d k_td| over the keys seen
      mass  [Tq,Hq,D]   softmax(z) |v|
      dv_mass           sum_i p_ij |do_i|
      dq_size, dk_size  sum |dz| |k|, sum |dz| |q| with scale
      dq_o, dk_o        the same with p sum_d |do| (mass + |o|) in the place of dz
      dq_v, dk_v        the same with p sum_d |do v|"""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    Tq, Hq, D = q.shape
    G = Hq // k.shape[1]
    r = dict(o=np.zeros_like(q), lse=np.full((Tq, Hq), -np.inf), reach=np.zeros((Tq, Hq)), mass=np.zeros_like(q))
    if do is not None:
        do = np.asarray(do, np.float64)
        for name, like in (("dq", q), ("dk", k), ("dv", v), ("dv_mass", v), ("dq_size", q), ("dk_size", k), ("dq_o", q), ("dk_o", k), ("dq_v", q), ("dk_v", k)):
            r[name] = np.zeros_like(like)
    for n in range(len(cu) - 1):
        a, b = slice(cu[n], cu[n + 1]), slice(cu_k[n], cu_k[n + 1])
        lq, lk = cu[n + 1] - cu[n], cu_k[n + 1] - cu_k[n]
        if lq <= 0 or lk <= 0:
            continue
        seen = _visible(lq, lk, window)
        some = seen.any(1)
        for h in range(Hq):
            j = h // G
            Q, K, V = q[a, h], k[b, j], v[b, j]
            z = np.where(seen, scale * (Q @ K.T), -np.inf)
            top = np.where(some, z.max(1), 0.0)
            e = np.exp(z - top[:, None])
            total = np.where(some, e.sum(1), 1.0)
            p = e / total[:, None]
            r["o"][a, h] = p @ V
            with np.errstate(divide="ignore"):
                r["lse"][a, h] = np.where(some, top + np.log(total), -np.inf)
            r["reach"][a, h] = np.where(seen, scale * (np.abs(Q) @ np.abs(K).T), 0.0).max(1)
            r["mass"][a, h] = p @ np.abs(V)
            if do is None:
                continue
            dO, O = do[a, h], r["o"][a, h]
            drop = (dO * O).sum(1) - (0.0 if dlse is None else np.asarray(dlse, np.float64)[a, h])
            dz = p * (dO @ V.T - drop[:, None])
            r["dq"][a, h] = scale * dz @ K
            r["dk"][b, j] += scale * dz.T @ Q
            r["dv"][b, j] += p.T @ dO
            r["dv_mass"][b, j] += p.T @ np.abs(dO)
            r["dq_size"][a, h] = scale * np.abs(dz) @ np.abs(K)
            r["dk_size"][b, j] += scale * np.abs(dz).T @ np.abs(Q)
            of_o = p * (np.abs(dO) * (r["mass"][a, h] + np.abs(O))).sum(1)[:, None]
            of_v = p * (np.abs(dO) @ np.abs(V).T)
            for name, x in (("_o", of_o), ("_v", of_v)):
                r["dq" + name][a, h] = scale * x @ np.abs(K)
                r["dk" + name][b, j] += scale * x.T @ np.abs(Q)
    return r


def ancestors(parents):
    """Of each drafted token, the tokens it sees (itself first, then upwards), None where there is no such token."""
    out = []
    for t in range(len(parents)):
        line, at = [], t
        while at >= 0:
            line.append(at)
            up = int(parents[at])
            if up < -1 or up >= at:
                line = None
                break
            at = up
        out.append(line)
    return out


def tree(q, k_new, v_new, k_cache, v_cache, table, lens, parents, scale, window=0, k_scale=None, v_scale=None):
    """q [N,T,Hq,D], k_new, v_new [N,T,Hkv,D], caches [pages,page,Hkv,D] as values (any NaN outside the sequences).
    Returns (o, lse, mass, reach) as decode.paged does."""
    q, kn, vn, kc, vc = (np.asarray(x, np.float64) for x in (q, k_new, v_new, k_cache, v_cache))
    N, T, Hq, D = q.shape
    pages, ps, Hkv = kc.shape[:3]
    ks = np.ones(Hkv) if k_scale is None else np.asarray(k_scale, np.float64)
    vs = np.ones(Hkv) if v_scale is None else np.asarray(v_scale, np.float64)
    o, mass = np.zeros((N, T, Hq, D)), np.zeros((N, T, Hq, D))
    lse, reach = np.full((N, T, Hq), -np.inf), np.zeros((N, T, Hq))
    for n in range(N):
        length = min(max(int(lens[n]), 0), table.shape[1] * ps)
        for t, line in enumerate(ancestors(parents[n])):
            if line is None:
                continue
            at = length + len(line) - 1
            first = max(0, at - window + 1) if window else 0
            pos = [x for x in range(first, length) if 0 <= table[n, x // ps] < pages]
            new = line[:window] if window else line
            where = (np.array([table[n, x // ps] for x in pos], int), np.array([x % ps for x in pos], int))
            kk = np.concatenate([kc[where] * ks[:, None], kn[n, new]])
            vv = np.concatenate([vc[where] * vs[:, None], vn[n, new]])
            for h in range(Hq):
                j = h // (Hq // Hkv)
                z = scale * (kk[:, j] @ q[n, t, h])
                p = np.exp(z - z.max())
                lse[n, t, h] = z.max() + np.log(p.sum())
                p /= p.sum()
                o[n, t, h] = p @ vv[:, j]
                mass[n, t, h] = p @ np.abs(vv[:, j])
                reach[n, t, h] = scale * (np.abs(kk[:, j]) @ np.abs(q[n, t, h])).max()
    return o, lse, mass, reach


def extend(table, lens, new, stack, free, page, total):
    """Lists and whole numbers.  Returns (table, lens, free, slots, cu)."""
    table, lens = [list(r) for r in table], list(lens)
    slots, cu, asked = [-1] * total, [0], 0
    free = top = min(max(free, 0), len(stack))
    at = 0
    for n in range(len(lens)):
        width = len(table[n]) * page
        have, more = min(max(lens[n], 0), width), max(new[n], 0)
        had, want = -(-have // page), -(-(have + more) // page)
        fits = have + more <= width
        asked += want - had if fits else 0
        if fits and (want == had or asked <= free):
            for c in range(had, want):
                top -= 1
                table[n][c] = stack[top]
            for i in range(have, have + more):
                if at + i - have < total:
                    slots[at + i - have] = table[n][i // page] * page + i % page
            lens[n] = have + more
        at += more
        cu.append(at)
    return table, lens, top, slots, cu


def trim(table, lens, keep, stack, free, page):
    """Returns (lens, stack, free)."""
    lens, stack = list(lens), list(stack)
    free = min(max(free, 0), len(stack))
    for n in reversed(range(len(lens))):
        have = min(max(lens[n], 0), len(table[n]) * page)
        kept = min(have, max(keep[n], 0))
        for c in reversed(range(-(-kept // page), -(-have // page))):
            if free < len(stack):
                stack[free] = table[n][c]
                free += 1
        lens[n] = kept
    return lens, stack, free
