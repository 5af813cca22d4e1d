"""The decoding entry points without a GPU: bad arguments are refused before anything is launched,
and workspace sizes follow the problem."""
import ctypes

import pytest

from chunked_prefill_gb300 import build as gbuild

FAKE, ODD = 0x10000, 0x10002


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    from chunked_prefill_gb300 import gdn
    return gdn


def step(L, ptrs=None, **kw):
    f = dict(num_seqs=2, total_tokens=2, Hqk=1, Hv=2, K=128, V=128, dtype=0, scale=0.1, num_slots=2)
    f.update(kw)
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, A_log=None, dt_bias=None, state_in=FAKE, state_out=FAKE, o=FAKE)
    a.update(ptrs or {})
    return L.lib().gdn_recurrent_step(ctypes.byref(L.GdnStepProblem(**f)), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=64, V=64), 2), (dict(K=0), 1), (dict(Hv=3, Hqk=2), 1), (dict(Hqk=0), 1), (dict(dtype=2), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(num_seqs=-1), 1), (dict(total_tokens=3), 1), (dict(num_slots=-1), 1),
    (dict(q_stride=64), 1), (dict(q_stride=130), 1), (dict(g_stride=1), 1), (dict(num_seqs=1 << 29, total_tokens=1 << 29), 2),
    (dict(ptrs=dict(q=None)), 1), (dict(ptrs=dict(q=ODD)), 1), (dict(ptrs=dict(o=None)), 1), (dict(ptrs=dict(g=ODD)), 1),
    (dict(ptrs=dict(state_in=ODD)), 1), (dict(ptrs=dict(A_log=FAKE)), 1), (dict(ptrs=dict(dt_bias=FAKE)), 1),
])
def test_step_refusals(L, kw, code):
    assert step(L, **kw) == code and L.lib().gdn_last_error()


def test_step_of_no_sequences_is_fine(L):
    assert step(L, num_seqs=0, total_tokens=0, ptrs=dict(q=None, k=None, v=None, g=None, beta=None, o=None)) == 0


def paged(L, ptrs=None, ws=(FAKE, 1 << 40), **kw):
    f = dict(num_seqs=2, Hq=4, Hkv=2, D=128, dtype=0, cache_dtype=0, scale=0.1, window=0, page_size=16, max_pages=8, num_pages=20,
             k_page_stride=4096, k_token_stride=256, k_head_stride=128, v_page_stride=4096, v_token_stride=256, v_head_stride=128)
    f.update(kw)
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, k_new=None, v_new=None, ks=None, vs=None, o=FAKE, lse=None)
    a.update(ptrs or {})
    p = L.GdnPagedProblem(**f)
    n = ctypes.c_size_t(0)
    size = L.lib().gdn_paged_attn_workspace_size(ctypes.byref(p), ctypes.byref(n))
    return L.lib().gdn_paged_attn_decode(ctypes.byref(p), *a.values(), *ws, None), size, n.value


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), 2), (dict(D=0), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(dtype=1), 1), (dict(cache_dtype=1), 1), (dict(dtype=2), 1),
    (dict(scale=-1.0), 1), (dict(window=-1), 1), (dict(page_size=0), 1), (dict(max_pages=1 << 28), 2), (dict(num_seqs=70000), 2),
    (dict(q_stride=4), 1), (dict(q_stride=516), 1), (dict(k_token_stride=4), 1), (dict(v_page_stride=-4096), 1),
    (dict(table_stride=2), 1), (dict(num_pages=-1), 1),
])
def test_paged_refusals(L, kw, code):
    got, size, _ = paged(L, **kw)
    assert got == code and size == code


@pytest.mark.parametrize("ptrs", [dict(q=None), dict(q=ODD), dict(k=ODD), dict(v=None), dict(table=None), dict(table=ODD), dict(lens=None), dict(o=ODD),
                                  dict(k_new=FAKE), dict(v_new=FAKE), dict(k_new=FAKE, v_new=ODD), dict(ks=ODD), dict(lse=ODD)])
def test_paged_pointer_refusals(L, ptrs):
    assert paged(L, ptrs=ptrs)[0] == 1


def test_paged_workspace(L):
    """Nothing is needed where no sequence can be split; a split problem refuses a smaller one."""
    _, size, small = paged(L, num_seqs=0, max_pages=1)
    assert size == 0 and small == 0
    _, _, need = paged(L, num_seqs=0, max_pages=1 << 16)
    assert need == 0  # no sequences
    p = dict(max_pages=1 << 16, num_pages=1 << 17)
    got, _, need = paged(L, ws=(None, 0), **p)
    assert got == 3 and need > 0
    assert paged(L, ws=(FAKE, need - 1), **p)[0] == 3
    assert paged(L, ws=(ODD, need), **p)[0] == 1


def norm(L, ptrs=None, back=False, ws=(FAKE, 1 << 40), **kw):
    f = dict(rows=4, dim=64, dtype=0, weight_dtype=0, out_dtype=0, group=0, eps=1e-6)
    f.update(kw)
    p = L.GdnNormProblem(**f)
    if back:
        a = dict(s=FAKE, w=FAKE, dy=FAKE, dsum=None, dx=FAKE, dw=FAKE)
        a.update(ptrs or {})
        return L.lib().gdn_rmsnorm_bwd(ctypes.byref(p), *a.values(), *ws, None)
    a = dict(x=FAKE, r=None, w=FAKE, y=FAKE, scale=None, sum=None)
    a.update(ptrs or {})
    return L.lib().gdn_rmsnorm_fwd(ctypes.byref(p), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(dim=0), dict(dtype=2), dict(weight_dtype=3), dict(eps=-1.0), dict(eps=float("nan")), dict(weight_offset=float("inf")),
    dict(x_stride=63), dict(ptrs=dict(w=None)), dict(ptrs=dict(w=FAKE + 1)),
])
@pytest.mark.parametrize("back", [False, True])
def test_norm_refusals(L, kw, back):
    assert norm(L, back=back, **kw) == 1


def test_norm_direction_refusals(L):
    assert norm(L, out_dtype=1) == 1
    assert norm(L, out_dtype=2, group=48, ptrs=dict(scale=FAKE)) == 1
    assert norm(L, out_dtype=2) == 1                   # no place for the scales
    assert norm(L, ptrs=dict(y=FAKE + 1)) == 1
    assert norm(L, back=True, ptrs=dict(dx=None)) == 1
    assert norm(L, back=True, ptrs=dict(dw=ODD)) == 1
    p = L.GdnNormProblem(rows=4, dim=64, eps=1e-6)
    n = ctypes.c_size_t(0)
    assert L.lib().gdn_rmsnorm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value >= 64 * 4
    assert norm(L, back=True, ws=(FAKE, n.value - 1)) == 3
    assert norm(L, rows=0, ptrs=dict(x=None, y=None)) == 0


OTHER, THIRD = 0x40000, 0x80000


@pytest.mark.parametrize("rows,kw,ptrs", [
    (4, dict(x_stride=72), dict(y=OTHER, sum=FAKE)), (4, dict(x_stride=72), dict(y=FAKE)), (4, dict(residual_stride=72), dict(r=THIRD, y=OTHER, sum=THIRD)),
    (4, dict(out_dtype=2), dict(scale=OTHER, y=FAKE)), (1, dict(out_dtype=2), dict(scale=OTHER, y=FAKE)), (4, dict(residual_stride=72), dict(r=THIRD, y=THIRD)),
])
def test_norm_in_place_refusals(L, rows, kw, ptrs):
    """Outputs have contiguous rows of their own type: over an input whose rows lie elsewhere they would
    overwrite rows that are still to be read."""
    assert norm(L, rows=rows, ptrs=ptrs, **kw) == 1


@pytest.mark.parametrize("kw,ptrs", [(dict(dy_stride=72), dict(dy=OTHER, dx=OTHER)), (dict(dsum_stride=72), dict(dsum=OTHER, dx=OTHER)),
                                     (dict(x_stride=72), dict(dy=OTHER))])
def test_norm_gradient_in_place_refusals(L, kw, ptrs):
    assert norm(L, back=True, ptrs=ptrs, **kw) == 1
