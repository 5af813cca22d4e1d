"""fp64 NumPy oracles of the decoding operators: the recurrent step, attention of one new token
over a paged cache, the RMS norm with the residual's addition and its gradient.  Written from the
definitions; test infrastructure only."""
from __future__ import annotations

import numpy as np

from oracle import prologue as pro

E4M3_MAX = 448.0


def step(q, k, v, g, beta, scale, state, slots, lengths, A_log=None, dt_bias=None):
    """q, k [T,Hqk,K], v [T,Hv,V], g, beta [T,Hv], state [slots,Hv,K,V].  Returns (o, new state);
    slots outside the pool give o = 0."""
    q, k, v, g, beta, state = (np.asarray(x, np.float64) for x in (q, k, v, g, beta, state))
    if A_log is not None:
        q, k, g, beta = pro.fwd(q, k, g, beta, np.asarray(A_log, np.float64), np.asarray(dt_bias, np.float64))
    G = v.shape[1] // q.shape[1]
    o, out, t = np.zeros_like(v), state.copy(), 0
    for n, length in enumerate(lengths):
        slot = int(slots[n])
        for i in range(t, t + int(length)):
            if not 0 <= slot < len(state):
                continue
            for j in range(v.shape[1]):
                S = out[slot, j].T  # [V, K]
                kt, qt = k[i, j // G], q[i, j // G]
                S = np.exp(g[i, j]) * (S - beta[i, j] * np.outer(S @ kt, kt)) + beta[i, j] * np.outer(v[i, j], kt)
                o[i, j] = scale * (S @ qt)
                out[slot, j] = S.T
        t += int(length)
    return o, out


def paged(q, k_cache, v_cache, table, lens, scale, window=0, k_scale=None, v_scale=None):
    """q [N,Hq,D], caches [pages,page,Hkv,D] as values (any NaN outside the sequences).  Returns
    (o, lse, mass, reach): mass = softmax(z) |v| and reach = max_t scale sum_d |q_d k_td|, the sizes
    that the rounding errors of o and lse go with."""
    q, kc, vc = (np.asarray(x, np.float64) for x in (q, k_cache, v_cache))
    N, Hq, D = q.shape
    pages, ps, Hkv = kc.shape[:3]
    ks = np.ones(Hkv) if k_scale is None else np.asarray(k_scale, np.float64)
    vs = np.ones(Hkv) if v_scale is None else np.asarray(v_scale, np.float64)
    o, mass = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    lse, reach = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    for n in range(N):
        length = min(max(int(lens[n]), 0), table.shape[1] * ps)
        first = max(0, length - window) if window else 0
        pos = [t for t in range(first, length) if 0 <= table[n, t // ps] < pages]
        if not pos:
            continue
        at = (np.array([table[n, t // ps] for t in pos]), np.array([t % ps for t in pos]))
        kk, vv = kc[at] * ks[:, None], vc[at] * vs[:, None]
        for h in range(Hq):
            j = h // (Hq // Hkv)
            z = scale * (kk[:, j] @ q[n, h])
            p = np.exp(z - z.max())
            lse[n, h] = z.max() + np.log(p.sum())
            p /= p.sum()
            o[n, h] = p @ vv[:, j]
            mass[n, h] = p @ np.abs(vv[:, j])
            reach[n, h] = scale * (np.abs(kk[:, j]) @ np.abs(q[n, h])).max()
    return o, lse, mass, reach


def norm(x, weight, residual=None, eps=1e-6, offset=0.0):
    """(y, s)."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s * r * (np.asarray(weight, np.float64) + offset), s


def norm_scales(y, group=0):
    """One scale per row, or per `group` values of it: [rows, dim / group]."""
    rows, dim = y.shape
    return np.maximum(np.abs(y.reshape(rows, -1, group or dim)).max(-1) / E4M3_MAX, 2.0 ** -126)


def norm_bwd(s, weight, dy, dsum=None, eps=1e-6, offset=0.0):
    """Gradients of <y, dy> + <s, dsum> at s: (dx, dweight, size of dx's terms, size of dweight's)."""
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    w = np.asarray(weight, np.float64) + offset
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    n = s * r
    c = (w * dy * n).mean(-1, keepdims=True)
    dx = r * (w * dy - n * c)
    size = r * (np.abs(w * dy) + np.abs(n) * np.abs(w * dy * n).mean(-1, keepdims=True))
    if dsum is not None:
        dx, size = dx + dsum, size + np.abs(dsum)
    return dx, (dy * n).sum(0), size, np.abs(dy * n).sum(0)
