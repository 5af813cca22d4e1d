"""Thin Python binding of libgdn.so (argument marshalling only; every step of the
computation runs in the library's CUDA kernels).

The names follow the C ABI (``gdn_chunk_fwd``, ``gdn_chunk_bwd``, ``*_workspace_size``)
and, on top, the FlashQLA pages' high-level call (aisparkup page, "usage":
``chunk_gated_delta_rule(q, k, v, g, beta, scale, initial_state, output_final_state,
cu_seqlens) -> (o, final_state)``) as a ``torch.autograd.Function``.

PyTorch supplies device memory and the stream; the library never allocates.  When
libgdn.so is missing this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_LIB selects another in-tree build of the same library (the checked variant
# libgdn_check.so in the bounds tests); the default is the release build
LIB_PATH = os.environ.get("GDN_LIB") or os.path.join(_HERE, "libgdn.so")

(GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA, GDN_ERR_TIMEOUT,
 GDN_ERR_BOUNDS) = range(7)
GDN_BF16, GDN_FP32, GDN_E4M3 = 0, 1, 2
CP_AUTO, CP_OFF, CP_EXACT, CP_WARMUP, CP_EXACT_FULL = 0, 1, 2, 3, 4
_STATUS = {1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED", 3: "GDN_ERR_WORKSPACE",
           4: "GDN_ERR_CUDA"}


class GdnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class GdnProblem(ctypes.Structure):
    """Mirror of ``gdn_problem`` in include/gdn.h."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hqk", ctypes.c_int32),
                ("Hv", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_host", ctypes.c_void_p),
                ("num_seqs", ctypes.c_int32), ("cp_mode", ctypes.c_int32),
                ("cp_segment_chunks", ctypes.c_int32), ("warmup_chunks", ctypes.c_int32),
                ("cp_lambda", ctypes.c_float)]


class GdnStepProblem(ctypes.Structure):
    """Mirror of ``gdn_step_problem``."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int32),
                ("Hqk", ctypes.c_int32), ("Hv", ctypes.c_int32), ("K", ctypes.c_int32),
                ("V", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("cu_seqlens", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("num_slots", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("g_stride", ctypes.c_int64), ("beta_stride", ctypes.c_int64),
                ("clear_rest", ctypes.c_int32)]


class GdnPagedProblem(ctypes.Structure):
    """Mirror of ``gdn_paged_problem``."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("cache_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("window", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("new_stride", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("k_page_stride", ctypes.c_int64), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64)]


class GdnNormProblem(ctypes.Structure):
    """Mirror of ``gdn_norm_problem``."""
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("group", ctypes.c_int32), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64), ("dy_stride", ctypes.c_int64),
                ("dsum_stride", ctypes.c_int64)]


class GdnKernelTime(ctypes.Structure):
    """Mirror of ``gdn_kernel_time``."""
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_float)]


_lib = None


def lib():
    """Load libgdn.so (built in-tree by ``chunked_prefill_gb300.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m chunked_prefill_gb300.build` (no fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        vp, P = ctypes.c_void_p, ctypes.POINTER(GdnProblem)
        L.gdn_chunk_fwd_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.gdn_chunk_bwd_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.gdn_chunk_fwd.argtypes = [P] + [vp] * 9 + [ctypes.c_size_t, vp]
        L.gdn_chunk_bwd.argtypes = [P] + [vp] * 15 + [ctypes.c_size_t, vp]
        L.gdn_chunk_layout.argtypes = [P, ctypes.POINTER(ctypes.c_int32),
                                       ctypes.POINTER(ctypes.c_int64)]
        L.gdn_debug_plan.argtypes = [P, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                                     ctypes.POINTER(ctypes.c_int32)]
        L.gdn_chunk_fwd_saved.argtypes = [P] + [vp] * 12 + [ctypes.c_size_t, vp]
        L.gdn_chunk_bwd_saved.argtypes = [P] + [vp] * 15 + [ctypes.c_size_t, vp]
        L.gdn_prologue_fwd.argtypes = [P] + [vp] * 10 + [vp]
        L.gdn_prologue_bwd_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.gdn_prologue_bwd.argtypes = [P] + [vp] * 17 + [ctypes.c_size_t, vp]
        S, A, N = (ctypes.POINTER(c) for c in (GdnStepProblem, GdnPagedProblem, GdnNormProblem))
        L.gdn_recurrent_step.argtypes = [S] + [vp] * 11
        L.gdn_paged_attn_workspace_size.argtypes = [A, ctypes.POINTER(ctypes.c_size_t)]
        L.gdn_paged_attn_decode.argtypes = [A] + [vp] * 12 + [ctypes.c_size_t, vp]
        L.gdn_rmsnorm_fwd.argtypes = [N] + [vp] * 7
        L.gdn_rmsnorm_bwd_workspace_size.argtypes = [N, ctypes.POINTER(ctypes.c_size_t)]
        L.gdn_rmsnorm_bwd.argtypes = [N] + [vp] * 7 + [ctypes.c_size_t, vp]
        for f in ("gdn_recurrent_step", "gdn_paged_attn_workspace_size", "gdn_paged_attn_decode",
                  "gdn_rmsnorm_fwd", "gdn_rmsnorm_bwd_workspace_size", "gdn_rmsnorm_bwd"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("gdn_chunk_fwd_workspace_size", "gdn_chunk_bwd_workspace_size",
                  "gdn_chunk_fwd", "gdn_chunk_bwd", "gdn_chunk_layout", "gdn_chunk_fwd_saved",
                  "gdn_chunk_bwd_saved", "gdn_prologue_fwd", "gdn_prologue_bwd_workspace_size",
                  "gdn_prologue_bwd"):
            getattr(L, f).restype = ctypes.c_int
        L.gdn_device_status.argtypes = [vp, vp]
        L.gdn_device_status.restype = ctypes.c_int
        L.gdn_debug_wait_timeout.argtypes = [vp, ctypes.c_int32, vp]
        L.gdn_debug_wait_timeout.restype = ctypes.c_int
        L.gdn_last_error.restype = ctypes.c_char_p
        L.gdn_timing_enable.argtypes = [ctypes.c_int32]
        L.gdn_timing_enable.restype = ctypes.c_int
        L.gdn_timing_collect.argtypes = [ctypes.POINTER(GdnKernelTime), ctypes.c_int32,
                                         ctypes.POINTER(ctypes.c_int32)]
        L.gdn_timing_collect.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int):
    if rc != GDN_OK:
        raise GdnError(rc, lib().gdn_last_error().decode())


def gdn_device_status(workspace, stream=None) -> int:
    """Wait for the stream and read the error word of a call's workspace: GDN_OK,
    GDN_ERR_BOUNDS when a checked build skipped an out-of-range store, or GDN_ERR_TIMEOUT
    when a device-side wait of that call gave up (see include/gdn.h)."""
    return lib().gdn_device_status(_ptr(workspace), _stream(stream))


def gdn_debug_wait_timeout(workspace, limit_us: int, stream=None):
    """Test hook: a kernel whose bounded wait runs out after limit_us, setting its bit in the
    error word of `workspace`."""
    _check(lib().gdn_debug_wait_timeout(_ptr(workspace), int(limit_us), _stream(stream)))


def gdn_timing_enable(on: bool = True):
    """Bracket every library kernel launch with CUDA events (see include/gdn.h)."""
    _check(lib().gdn_timing_enable(1 if on else 0))


def gdn_timing_collect() -> dict:
    """{kernel name: (launches, total ms)} since the last collect; waits on the events."""
    buf = (GdnKernelTime * 64)()
    n = ctypes.c_int32(0)
    _check(lib().gdn_timing_collect(buf, 64, ctypes.byref(n)))
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms))
            for i in range(min(n.value, 64))}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return GDN_BF16
    if dt == torch.float32:
        return GDN_FP32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {dt}")


class Problem:
    """A ``gdn_problem`` plus the host copy of cu_seqlens it points to (kept alive)."""

    def __init__(self, q, v, scale, cu_seqlens=None, cu_seqlens_host=None, cp_mode=CP_AUTO,
                 cp_segment_chunks=0, warmup_chunks=0, cp_lambda=0.0):
        B, T, Hqk, K = q.shape
        Hv, V = v.shape[2], v.shape[3]
        p = GdnProblem(B=B, T=T, Hqk=Hqk, Hv=Hv, K=K, V=V, dtype=_dtype_code(q.dtype),
                       scale=float(scale), cp_mode=cp_mode, cp_segment_chunks=cp_segment_chunks,
                       warmup_chunks=warmup_chunks, cp_lambda=cp_lambda)
        self._cu_host = None
        self.num_seqs = B
        if cu_seqlens is not None:
            if cu_seqlens_host is None:
                cu_seqlens_host = cu_seqlens.detach().to("cpu")
            self._cu_host = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
            self._cu_dev = cu_seqlens
            p.cu_seqlens = cu_seqlens.data_ptr()
            p.cu_seqlens_host = self._cu_host.data_ptr()
            p.num_seqs = self._cu_host.numel() - 1
            self.num_seqs = p.num_seqs
        self.p = p
        self.Hv, self.K, self.V = Hv, K, V

    def ref(self):
        return ctypes.byref(self.p)


def gdn_chunk_fwd_workspace_size(prob: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().gdn_chunk_fwd_workspace_size(prob.ref(), ctypes.byref(n)))
    return n.value


def gdn_chunk_bwd_workspace_size(prob: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().gdn_chunk_bwd_workspace_size(prob.ref(), ctypes.byref(n)))
    return n.value


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _workspace(nbytes, device, workspace):
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def _validate_tensors(q, k, v, g, beta):
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if k.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q and k must match in shape; q, k, v in dtype")
    if g.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("g and beta must be float32")
    if g.shape != v.shape[:3] or beta.shape != v.shape[:3]:
        raise ValueError("g and beta must be [B, T, Hv]")


def gdn_chunk_fwd(q, k, v, g, beta, scale, h0=None, output_final_state=True, cu_seqlens=None,
                  cu_seqlens_host=None, cp_mode=CP_AUTO, cp_segment_chunks=0, warmup_chunks=0,
                  cp_lambda=0.0, o=None, ht=None, workspace=None, stream=None):
    """Forward through the C ABI.  Returns (o, ht); ht is None unless requested."""
    _validate_tensors(q, k, v, g, beta)
    prob = Problem(q, v, scale, cu_seqlens, cu_seqlens_host, cp_mode, cp_segment_chunks,
                   warmup_chunks, cp_lambda)
    if o is None:
        o = torch.empty_like(v)
    if ht is None and output_final_state:
        ht = torch.empty(prob.num_seqs, prob.Hv, prob.K, prob.V, device=q.device,
                         dtype=torch.float32)
    if h0 is not None:
        h0 = h0.contiguous().float()
    nbytes = gdn_chunk_fwd_workspace_size(prob)
    ws = _workspace(nbytes, q.device, workspace)
    _check(lib().gdn_chunk_fwd(prob.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                               _ptr(h0), _ptr(o), _ptr(ht), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)))
    return o, ht


def gdn_chunk_bwd(q, k, v, g, beta, scale, dO, h0=None, dht=None, cu_seqlens=None,
                  cu_seqlens_host=None, cp_mode=CP_AUTO, cp_segment_chunks=0, warmup_chunks=0,
                  cp_lambda=0.0, want_dh0=True, workspace=None, stream=None, out=None):
    """Backward through the C ABI.  Returns (dq, dk, dv, dg, dbeta, dh0)."""
    _validate_tensors(q, k, v, g, beta)
    if dO.shape != v.shape or dO.dtype != v.dtype or not dO.is_contiguous():
        raise ValueError("dO must be contiguous and match v")
    prob = Problem(q, v, scale, cu_seqlens, cu_seqlens_host, cp_mode, cp_segment_chunks,
                   warmup_chunks, cp_lambda)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dg, db = torch.empty_like(g), torch.empty_like(beta)
        dh0 = (torch.empty(prob.num_seqs, prob.Hv, prob.K, prob.V, device=q.device)
               if want_dh0 else None)
    else:
        dq, dk, dv, dg, db, dh0 = out
    if h0 is not None:
        h0 = h0.contiguous().float()
    if dht is not None:
        dht = dht.contiguous().float()
    nbytes = gdn_chunk_bwd_workspace_size(prob)
    ws = _workspace(nbytes, q.device, workspace)
    _check(lib().gdn_chunk_bwd(prob.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                               _ptr(h0), _ptr(dO), _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(dg), _ptr(db), _ptr(dh0), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)))
    return dq, dk, dv, dg, db, dh0


def gdn_chunk_layout(prob: Problem):
    """(chunk size C, chunks over all sequences) of the per-chunk saved outputs."""
    c, n = ctypes.c_int32(0), ctypes.c_int64(0)
    _check(lib().gdn_chunk_layout(prob.ref(), ctypes.byref(c), ctypes.byref(n)))
    return c.value, n.value


def gdn_debug_plan(prob: Problem, sms: int):
    """Test hook: (chunks per segment, segments) the planner picks for `prob` on `sms` SMs."""
    L, n = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().gdn_debug_plan(prob.ref(), int(sms), ctypes.byref(L), ctypes.byref(n)))
    return L.value, n.value


def gdn_chunk_fwd_saved(q, k, v, g, beta, scale, h0=None, output_final_state=True,
                        cu_seqlens=None, cu_seqlens_host=None, cp_mode=CP_AUTO,
                        cp_segment_chunks=0, cp_lambda=0.0, want_g_cum=True, want_A=True,
                        workspace=None, stream=None, o=None, ht=None, h=None):
    """Low-level forward through the C ABI.  Returns (g_cum, A, o, h, ht, ctx): the in-chunk
    cumulative gate [B,T,Hv] (or None), every token's row of its chunk's (I + A)^-1
    [B,T,Hv,C] (or None), the output, the state entering every chunk [total_chunks,Hv,K,V],
    the final state (or None) and the workspace that gdn_chunk_bwd_saved reads back."""
    _validate_tensors(q, k, v, g, beta)
    prob = Problem(q, v, scale, cu_seqlens, cu_seqlens_host, cp_mode, cp_segment_chunks, 0,
                   cp_lambda)
    C, nchunks = gdn_chunk_layout(prob)
    B, T, Hv = v.shape[:3]
    if o is None:
        o = torch.empty_like(v)
    if ht is None and output_final_state:
        ht = torch.empty(prob.num_seqs, Hv, prob.K, prob.V, device=q.device, dtype=torch.float32)
    g_cum = torch.empty_like(g) if want_g_cum else None
    A = torch.empty(B, T, Hv, C, device=q.device, dtype=q.dtype) if want_A else None
    if h is None:
        h = torch.empty(max(nchunks, 0), Hv, prob.K, prob.V, device=q.device, dtype=q.dtype)
    if h0 is not None:
        h0 = h0.contiguous().float()
    nbytes = gdn_chunk_bwd_workspace_size(prob)
    ws = _workspace(nbytes, q.device, workspace)
    _check(lib().gdn_chunk_fwd_saved(prob.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                     _ptr(h0), _ptr(o), _ptr(ht), _ptr(g_cum), _ptr(A), _ptr(h),
                                     _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
    return g_cum, A, o, h, ht, ws


def gdn_chunk_bwd_saved(q, k, v, g, beta, scale, h, ctx, dO, dht=None, cu_seqlens=None,
                        cu_seqlens_host=None, cp_mode=CP_AUTO, cp_segment_chunks=0,
                        cp_lambda=0.0, want_dh0=True, stream=None, out=None):
    """Backward from the saved states h and workspace ctx of gdn_chunk_fwd_saved (same
    problem arguments).  Returns (dq, dk, dv, dg, dbeta, dh0)."""
    _validate_tensors(q, k, v, g, beta)
    if dO.shape != v.shape or dO.dtype != v.dtype or not dO.is_contiguous():
        raise ValueError("dO must be contiguous and match v")
    prob = Problem(q, v, scale, cu_seqlens, cu_seqlens_host, cp_mode, cp_segment_chunks, 0,
                   cp_lambda)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dg, db = torch.empty_like(g), torch.empty_like(beta)
        dh0 = (torch.empty(prob.num_seqs, prob.Hv, prob.K, prob.V, device=q.device)
               if want_dh0 else None)
    else:
        dq, dk, dv, dg, db, dh0 = out
    if dht is not None:
        dht = dht.contiguous().float()
    _check(lib().gdn_chunk_bwd_saved(prob.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                     _ptr(h), _ptr(dO), _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv),
                                     _ptr(dg), _ptr(db), _ptr(dh0), _ptr(ctx),
                                     ctx.numel() * ctx.element_size(), _stream(stream)))
    return dq, dk, dv, dg, db, dh0


def chunk_gated_delta_rule_fwd(q, k, v, g, beta, scale=None, initial_state=None,
                               output_final_state=True, cu_seqlens=None, stream=None):
    """Low-level forward under the FlashQLA name (usage page, "low-level API"): returns
    (g_cum, A, o, h, final_state) -- the in-chunk cumulative gate, every token's row of its
    chunk's (I + A)^-1, the output, the state entering every chunk and the final state (None
    unless output_final_state).  The chunk records that chunk_gated_delta_rule_bwd reads back
    stay attached to h (attribute gdn_ctx), so h must be passed to it unchanged."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    g_cum, A, o, h, ht, ctx = gdn_chunk_fwd_saved(q, k, v, g, beta, scale, h0=initial_state,
                                                  output_final_state=output_final_state,
                                                  cu_seqlens=cu_seqlens, stream=stream)
    h.gdn_ctx = ctx
    return g_cum, A, o, h, ht


def chunk_gated_delta_rule_bwd(q, k, v, g, beta, h, do, dht=None, scale=None,
                               cu_seqlens=None, stream=None):
    """Low-level backward from chunk_gated_delta_rule_fwd's h (same q, k, v, g, beta, scale and
    cu_seqlens): returns (dq, dk, dv, dg, dbeta, dh0).  g and beta are the forward's inputs,
    not its cumulative gate."""
    ctx = getattr(h, "gdn_ctx", None)
    if ctx is None:
        raise ValueError("h must be the state tensor returned by chunk_gated_delta_rule_fwd")
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return gdn_chunk_bwd_saved(q, k, v, g, beta, scale, h, ctx, do, dht=dht,
                               cu_seqlens=cu_seqlens, stream=stream)


def _prologue_problem(q_raw, a):
    if q_raw.dim() != 4 or a.dim() != 3 or a.shape[:2] != q_raw.shape[:2]:
        raise ValueError("q_raw must be [B,T,Hqk,K] and a [B,T,Hv]")
    B, T, Hqk, K = q_raw.shape
    Hv = a.shape[2]
    return GdnProblem(B=B, T=T, Hqk=Hqk, Hv=Hv, K=K, V=K, dtype=_dtype_code(q_raw.dtype),
                      scale=1.0, cp_mode=CP_AUTO)


def _check_prologue_inputs(q_raw, k_raw, a, b, A_log, dt_bias):
    for name, t in (("q_raw", q_raw), ("k_raw", k_raw), ("a", a), ("b", b), ("A_log", A_log),
                    ("dt_bias", dt_bias)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if k_raw.shape != q_raw.shape or k_raw.dtype != q_raw.dtype:
        raise ValueError("q_raw and k_raw must match in shape and dtype")
    for name, t in (("a", a), ("b", b), ("A_log", A_log), ("dt_bias", dt_bias)):
        if t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    if b.shape != a.shape or A_log.shape != (a.shape[2],) or dt_bias.shape != (a.shape[2],):
        raise ValueError("b must match a; A_log and dt_bias must be [Hv]")


def gdn_prologue_fwd(q_raw, k_raw, a, b, A_log, dt_bias, stream=None):
    """Fused prologue through the C ABI: (q, k, g, beta) from the raw projections."""
    _check_prologue_inputs(q_raw, k_raw, a, b, A_log, dt_bias)
    p = _prologue_problem(q_raw, a)
    q, k = torch.empty_like(q_raw), torch.empty_like(k_raw)
    g, beta = torch.empty_like(a), torch.empty_like(b)
    _check(lib().gdn_prologue_fwd(ctypes.byref(p), _ptr(q_raw), _ptr(k_raw), _ptr(a), _ptr(b),
                                  _ptr(A_log), _ptr(dt_bias), _ptr(q), _ptr(k), _ptr(g),
                                  _ptr(beta), _stream(stream)))
    return q, k, g, beta


def gdn_prologue_bwd(q_raw, k_raw, a, b, A_log, dt_bias, dq, dk, dg, dbeta, stream=None):
    """Reverse mode of the prologue: (dq_raw, dk_raw, da, db, dA_log, ddt_bias)."""
    _check_prologue_inputs(q_raw, k_raw, a, b, A_log, dt_bias)
    p = _prologue_problem(q_raw, a)
    dq, dk = dq.contiguous(), dk.contiguous()
    dg, dbeta = dg.contiguous().float(), dbeta.contiguous().float()
    dq_raw, dk_raw = torch.empty_like(q_raw), torch.empty_like(k_raw)
    da, db = torch.empty_like(a), torch.empty_like(b)
    dA_log, ddt_bias = torch.empty_like(A_log), torch.empty_like(dt_bias)
    n = ctypes.c_size_t(0)
    _check(lib().gdn_prologue_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device=q_raw.device)
    _check(lib().gdn_prologue_bwd(ctypes.byref(p), _ptr(q_raw), _ptr(k_raw), _ptr(a), _ptr(b),
                                  _ptr(A_log), _ptr(dt_bias), _ptr(dq), _ptr(dk), _ptr(dg),
                                  _ptr(dbeta), _ptr(dq_raw), _ptr(dk_raw), _ptr(da), _ptr(db),
                                  _ptr(dA_log), _ptr(ddt_bias), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)))
    return dq_raw, dk_raw, da, db, dA_log, ddt_bias


class _Prologue(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q_raw, k_raw, a, b, A_log, dt_bias):
        ctx.save_for_backward(q_raw, k_raw, a, b, A_log, dt_bias)
        return gdn_prologue_fwd(q_raw, k_raw, a, b, A_log, dt_bias)

    @staticmethod
    def backward(ctx, dq, dk, dg, dbeta):
        q_raw, k_raw, a, b, A_log, dt_bias = ctx.saved_tensors
        zero = lambda t, like: torch.zeros_like(like) if t is None else t
        return gdn_prologue_bwd(q_raw, k_raw, a, b, A_log, dt_bias, zero(dq, q_raw),
                                zero(dk, k_raw), zero(dg, a), zero(dbeta, b))


def gated_delta_rule_prologue(q_raw, k_raw, a, b, A_log, dt_bias):
    """Differentiable fused prologue: q, k L2-normalised over K; g = -exp(A_log)
    softplus(a + dt_bias); beta = sigmoid(b).  Returns (q, k, g, beta)."""
    return _Prologue.apply(q_raw, k_raw, a, b, A_log, dt_bias)


class _ChunkGDN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0, scale, output_final_state, cu_seqlens, save_states):
        if save_states:
            _, _, o, h, ht, ws = gdn_chunk_fwd_saved(q, k, v, g, beta, scale, h0=h0,
                                                     output_final_state=output_final_state,
                                                     cu_seqlens=cu_seqlens, want_g_cum=False,
                                                     want_A=False)
            ctx.save_for_backward(q, k, v, g, beta, h0, cu_seqlens, h, ws)
        else:
            o, ht = gdn_chunk_fwd(q, k, v, g, beta, scale, h0=h0,
                                  output_final_state=output_final_state, cu_seqlens=cu_seqlens)
            ctx.save_for_backward(q, k, v, g, beta, h0, cu_seqlens)
        ctx.scale = scale
        ctx.save_states = save_states
        return o, ht

    @staticmethod
    def backward(ctx, do, dht):
        if ctx.save_states:
            q, k, v, g, beta, h0, cu, h, ws = ctx.saved_tensors
            grads = gdn_chunk_bwd_saved(q, k, v, g, beta, ctx.scale, h, ws, do.contiguous(),
                                        dht=dht, cu_seqlens=cu, want_dh0=h0 is not None)
        else:
            q, k, v, g, beta, h0, cu = ctx.saved_tensors
            grads = gdn_chunk_bwd(q, k, v, g, beta, ctx.scale, do.contiguous(), h0=h0, dht=dht,
                                  cu_seqlens=cu, want_dh0=h0 is not None)
        return (*grads, None, None, None, None)


def chunk_gated_delta_rule(q, k, v, g, beta, scale=None, initial_state=None,
                           output_final_state=False, cu_seqlens=None, save_states=False):
    """High-level call with the FlashQLA/FLA signature; differentiable.
    q, k [B,T,Hqk,K]; v [B,T,Hv,V]; g, beta [B,T,Hv] (fp32); initial_state [N,Hv,K,V].
    save_states=True keeps the state entering every chunk (and the chunk records) from the
    forward for the backward, which then skips its recompute of the forward."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return _ChunkGDN.apply(q, k, v, g, beta, initial_state, scale, output_final_state,
                           cu_seqlens, save_states)


# ---------------------------------------------------------------------------- decoding
# The checks and the marshalling of these calls are native (csrc/binding.cpp): a decoding step is
# made of many calls that take a few microseconds on the GPU.
_native = None


def _binding():
    """Load _binding.so (built in-tree next to libgdn.so) and hand it the library's functions."""
    global _native
    if _native is None:
        L = lib()
        path = os.path.join(_HERE, "_binding.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m chunked_prefill_gb300.build` (no fallback exists)")
        from chunked_prefill_gb300 import _binding as B
        B.bind(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "gdn_recurrent_step", "gdn_paged_attn_workspace_size", "gdn_paged_attn_decode",
            "gdn_rmsnorm_fwd", "gdn_rmsnorm_bwd_workspace_size", "gdn_rmsnorm_bwd")), _check)
        _native = B
    return _native


def gdn_recurrent_step(q, k, v, g, beta, scale, state_in=None, state_out=None, slots=None,
                       cu_seqlens=None, A_log=None, dt_bias=None, o=None, stream=None):
    """Recurrent step through the C ABI (see include/gdn.h).  q, k [B,T,Hqk,K], v [B,T,Hv,V],
    g, beta [B,T,Hv] fp32, each with contiguous rows at any token stride but 0; state_in, state_out
    [num_slots,Hv,K,V] fp32 pools; slots int32 [num_seqs]; cu_seqlens int32 [num_seqs+1] with
    B = 1, else B sequences of T tokens.  Returns o [B,T,Hv,V], 0 for tokens that no sequence
    covers (a given o keeps what it has there)."""
    return (_native or _binding()).step(q, k, v, g, beta, scale, state_in, state_out, slots,
                                        cu_seqlens, A_log, dt_bias, o, stream)


def gated_delta_rule_step(q, k, v, g, beta, scale=None, state=None, state_out=None, slots=None,
                          cu_seqlens=None, A_log=None, dt_bias=None, o=None, stream=None):
    """One decoding step of the gated delta rule: the recurrence of chunk_gated_delta_rule token
    by token, for the one or few new tokens of each sequence.  Returns (o, state_out).

    q, k [B,T,Hqk,K]; v [B,T,Hv,V]; g, beta [B,T,Hv] fp32 -- or, with A_log and dt_bias [Hv], the
    raw projections q, k, a, b of gated_delta_rule_prologue, whose activations are then fused in.
    state [num_slots,Hv,K,V] fp32 (None: zero), e.g. chunk_gated_delta_rule's final state, is
    updated in place unless state_out names another pool of the same shape; slots int32 [N] says
    which slot each sequence has (None: its own index; -1: a padding row, whose o is 0).
    cu_seqlens int32 [N+1] (device, B = 1) packs sequences of different token counts; the o of
    tokens that it does not cover is 0 (a given o keeps what it has there).  For inference:
    nothing is differentiated here."""
    if stream is not None:  # what is allocated here belongs to that stream, too
        with torch.cuda.stream(stream):
            return gated_delta_rule_step(q, k, v, g, beta, scale, state, state_out, slots, cu_seqlens,
                                         A_log, dt_bias, o)
    native = _native or _binding()
    if native.wants_grad(q, k, v, g, beta, state, state_out, A_log, dt_bias):
        raise RuntimeError("gated_delta_rule_step is not differentiable, but an argument requires a "
                           "gradient: train with chunk_gated_delta_rule")
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if state_out is None:
        state_out = state
        if state is None:
            if slots is not None:
                raise ValueError("slots need a state pool (state or state_out)")
            n = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            state_out = torch.empty(n, v.shape[2], q.shape[-1], v.shape[-1], dtype=torch.float32,
                                    device=q.device)
    return native.step(q, k, v, g, beta, scale, state, state_out, slots, cu_seqlens, A_log, dt_bias,
                       o, None), state_out


def gdn_paged_attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, k_new=None, v_new=None,
                          k_scale=None, v_scale=None, window=0, o=None, lse=None, workspace=None,
                          stream=None):
    """Paged decode attention through the C ABI (see include/gdn.h).  Returns o; lse is written
    when given."""
    return (_native or _binding()).paged(q, k_cache, v_cache, page_table, seq_lens, scale, k_new,
                                         v_new, k_scale, v_scale, window, o, lse, workspace, stream)


def paged_attention_decode(q, k_cache, v_cache, page_table, seq_lens, scale=None, k_new=None,
                           v_new=None, k_scale=None, v_scale=None, window=0, return_lse=False,
                           o=None, workspace=None, stream=None):
    """Attention of one new token per sequence over a paged key-value cache: o [N,Hq,D], or
    (o, lse [N,Hq] fp32) with return_lse.

    q [N,Hq,D]; caches [num_pages,page_size,Hkv,D] of any page, token and head strides, bf16 or
    e4m3 (with fp32 scales [Hkv]) under bf16 queries, fp32 under fp32 ones; page_table int32
    [N,max_pages]; seq_lens int32 [N], the new token counted.  k_new, v_new [N,Hkv,D]: the new
    token's key and value, which the call then writes to position seq_lens - 1 of the caches
    before it attends to them.  window > 0 attends to the last `window` tokens.  The weights are
    rounded to bf16 (fp16 under e4m3 caches) for their product with v under bf16 queries, their
    sum is not; a table no wider than the longest sequence may become is best, for the work is
    divided by its width.  For inference: nothing is differentiated here."""
    native = _native or _binding()
    if native.wants_grad(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale):
        raise RuntimeError("paged_attention_decode is not differentiable, but an argument requires "
                           "a gradient")
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return native.paged(q, k_cache, v_cache, page_table, seq_lens, scale, k_new, v_new, k_scale,
                        v_scale, window, o, True if return_lse else None, workspace, stream)


def gdn_rmsnorm_fwd(x, weight, residual=None, eps=1e-6, weight_offset=0.0, quant=False, group=0,
                    want_sum=True, stream=None):
    """Norm with the residual's addition through the C ABI (see include/gdn.h).  Returns
    (y, y_scale, sum): y_scale is None without quant, sum None without a residual (or want_sum)."""
    return (_native or _binding()).norm_fwd(x, weight, residual, eps, weight_offset, quant, group,
                                            want_sum, stream)


def gdn_rmsnorm_bwd(s, weight, dy, dsum=None, eps=1e-6, weight_offset=0.0, workspace=None, stream=None):
    """Gradients of the norm at its summed input s: (dx, dweight fp32).  dsum is the gradient
    with respect to the sum (None: zero)."""
    return (_native or _binding()).norm_bwd(s, weight, dy, dsum, eps, weight_offset, workspace, stream)


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, weight_offset):
        ctx.set_materialize_grads(False)  # an unused sum has no gradient to read
        y, _, total = gdn_rmsnorm_fwd(x, weight, residual, eps, weight_offset)
        ctx.save_for_backward(x if residual is None else total, weight)
        ctx.eps, ctx.weight_offset, ctx.residual = eps, weight_offset, residual is not None
        return y, total

    @staticmethod
    @once_differentiable  # a second derivative is refused, not zero
    def backward(ctx, dy, dtotal):
        s, weight = ctx.saved_tensors
        dim = s.shape[-1]
        if dy is None:
            dy = torch.zeros_like(s)
        flat = lambda t: None if t is None else t.contiguous().view(-1, dim)  # noqa: E731
        dx, dw = gdn_rmsnorm_bwd(flat(s), weight, flat(dy), flat(dtotal), ctx.eps, ctx.weight_offset)
        dx = dx.view(s.shape)
        return dx, dw.to(weight.dtype), dx if ctx.residual else None, None, None


def rms_norm(x, weight, residual=None, eps=1e-6, weight_offset=0.0):
    """Root-mean-square norm with the residual's addition: s = x + residual, y = s / sqrt(mean(s^2)
    + eps) * (weight + weight_offset) over the last dimension.  Returns (y, s), s None without a
    residual.  x, residual [..., dim] bf16 or fp32; weight [dim] bf16 or fp32.  Differentiable with
    respect to x, residual and weight (the backward pass takes s as it was rounded), once."""
    native = _native or _binding()
    if native.wants_grad(x, weight, residual):
        return _RMSNorm.apply(x, weight, residual, eps, weight_offset)
    y, _, total = native.norm_fwd(x, weight, residual, eps, weight_offset, False, 0, True, None)
    return y, total


def rms_norm_quant(x, weight, residual=None, eps=1e-6, weight_offset=0.0, group=0):
    """rms_norm with y in 8 bits (float8_e4m3fn): returns (y, scale, s) with the normed row
    approximately y * scale; scale fp32 [..., 1], or [..., dim / group] with one scale to `group`
    consecutive values: max |y| / 448, not below 2^-126, by a product with 1 / 448 as torch
    divides a GPU tensor by a number, and y by one with 1 / scale.  Nothing is differentiated here:
    to train through it, pass the gradient with respect to y * scale as gdn_rmsnorm_bwd's dy."""
    native = _native or _binding()
    if native.wants_grad(x, weight, residual):
        raise RuntimeError("rms_norm_quant is not differentiable, but an argument requires a gradient: "
                           "train with rms_norm or gdn_rmsnorm_bwd")
    return native.norm_fwd(x, weight, residual, eps, weight_offset, True, group, True, None)
