"""Attention over prompts and drafted trees and the paged cache's operators without a GPU: bad arguments are
refused before anything is launched, in the C ABI and in Python."""
import ctypes

import pytest
import torch

from chunked_prefill_gb300 import build as gbuild

FAKE, ODD = 0x10000, 0x10002
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    from chunked_prefill_gb300 import gdn
    return gdn


def prompt(L, back=False, ptrs=None, ws=(FAKE, 1 << 40), **kw):
    f = dict(num_seqs=2, total_q=8, total_k=8, Hq=4, Hkv=2, D=64, dtype=0, scale=0.1)
    f.update(kw)
    p = L.GdnPromptProblem(**f)
    if back:
        a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, rest=None, do=FAKE, dlse=None, dq=FAKE, dk=FAKE, dv=FAKE)
        a.update(ptrs or {})
        return L.lib().gdn_prompt_attn_bwd(ctypes.byref(p), *a.values(), *ws, None)
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=None, rest=None)
    a.update({n: x for n, x in (ptrs or {}).items() if n in a})
    return L.lib().gdn_prompt_attn_fwd(ctypes.byref(p), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), 2), (dict(D=0), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(dtype=2), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(window=-1), 1), (dict(num_seqs=-1), 1), (dict(total_q=-2), 1), (dict(total_q=9), 1), (dict(total_k=9), 1), (dict(num_seqs=0), 1),
    (dict(num_seqs=70000), 2), (dict(cu_seqlens=ODD), 1), (dict(cu_seqlens_k=FAKE), 1), (dict(cu_seqlens=FAKE, total_k=9), 1),
    (dict(cu_seqlens=FAKE, cu_seqlens_k=ODD), 1), (dict(q_stride=128), 1), (dict(k_stride=130), 1), (dict(v_stride=132), 1),
    (dict(total_q=0x7fff0002, total_k=0x7fff0002), 2), (dict(Hq=1 << 16, Hkv=1), 2), (dict(q_stride=1 << 40), 2),
    (dict(ptrs=dict(q=None)), 1), (dict(ptrs=dict(k=ODD)), 1), (dict(ptrs=dict(v=None)), 1), (dict(ptrs=dict(o=ODD)), 1), (dict(ptrs=dict(lse=ODD)), 1),
    (dict(ptrs=dict(rest=ODD)), 1), (dict(ptrs=dict(rest=FAKE), dtype=1), 1),
])
@pytest.mark.parametrize("back", [False, True])
def test_prompt_refusals(L, kw, code, back):
    assert prompt(L, back, **kw) == code and L.lib().gdn_last_error()


def test_prompt_backward_refusals(L):
    for name in ("o", "lse", "do", "dq", "dk", "dv"):
        assert prompt(L, True, ptrs={name: None}) == 1, name
    assert prompt(L, True, ptrs=dict(dlse=ODD)) == 1
    n = ctypes.c_size_t(0)
    p = L.GdnPromptProblem(num_seqs=2, total_q=8, total_k=8, Hq=4, Hkv=2, D=64, scale=0.1)
    assert L.lib().gdn_prompt_attn_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value >= 8 * 4 * 8
    assert L.lib().gdn_prompt_attn_bwd_workspace_size(ctypes.byref(p), None) == 1
    assert prompt(L, True, ws=(FAKE, n.value - 1)) == 3 and prompt(L, True, ws=(None, 0)) == 3 and prompt(L, True, ws=(ODD, n.value)) == 1


def test_prompt_of_nothing_is_fine(L):
    none = dict(q=None, k=None, v=None, o=None)
    assert prompt(L, num_seqs=0, total_q=0, total_k=0, ptrs=none) == 0
    assert prompt(L, num_seqs=3, total_q=0, total_k=0, ptrs=none) == 0
    assert prompt(L, True, num_seqs=0, total_q=0, total_k=0, ws=(None, 0), ptrs=dict(none, lse=None, do=None, dq=None, dk=None, dv=None)) == 0


def tree(L, ptrs=None, ws=(FAKE, 1 << 40), **kw):
    f = dict(num_seqs=2, T=4, Hq=4, Hkv=2, D=128, dtype=0, cache_dtype=0, scale=0.1, window=0, page_size=16, max_pages=8, num_pages=20,
             k_page_stride=4096, k_token_stride=256, k_head_stride=128, v_page_stride=4096, v_token_stride=256, v_head_stride=128)
    f.update(kw)
    a = dict(q=FAKE, k_new=FAKE, v_new=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, parents=FAKE, ks=None, vs=None, o=FAKE, lse=None)
    a.update(ptrs or {})
    p = L.GdnTreeProblem(**f)
    n = ctypes.c_size_t(0)
    size = L.lib().gdn_paged_attn_tree_workspace_size(ctypes.byref(p), ctypes.byref(n))
    return L.lib().gdn_paged_attn_tree(ctypes.byref(p), *a.values(), *ws, None), size, n.value


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), 2), (dict(D=0), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(dtype=1), 1), (dict(cache_dtype=1), 1), (dict(dtype=2), 1), (dict(T=0), 1),
    (dict(T=65), 2), (dict(scale=-1.0), 1), (dict(window=-1), 1), (dict(page_size=0), 1), (dict(max_pages=1 << 28), 2), (dict(num_seqs=70000), 2),
    (dict(q_stride=4), 1), (dict(q_stride=516), 1), (dict(k_new_stride=252), 1), (dict(v_new_stride=260), 1), (dict(k_token_stride=4), 1),
    (dict(v_page_stride=-4096), 1), (dict(table_stride=2), 1), (dict(num_pages=-1), 1),
])
def test_tree_refusals(L, kw, code):
    got, size, _ = tree(L, **kw)
    assert got == code and size == code


STRIDES = [f"{c}_{n}_stride" for c in "kv" for n in ("page", "token", "head")]


@pytest.mark.parametrize("cache_dtype", [0, 2])
@pytest.mark.parametrize("name", STRIDES)
def test_tree_refuses_caches_without_a_stride(L, name, cache_dtype):
    """An expanded cache: a tensor map does not have strides of 0.  In a dimension of one the stride is not used."""
    got, size, _ = tree(L, cache_dtype=cache_dtype, **{name: 0})
    assert got == 1 and size == 1 and b"strides of 0" in L.lib().gdn_last_error()
    n = ctypes.c_size_t(0)
    one = dict(num_seqs=2, T=4, Hq=4, Hkv=1, D=128, cache_dtype=cache_dtype, scale=0.1, page_size=1, max_pages=8, num_pages=1)
    assert L.lib().gdn_paged_attn_tree_workspace_size(ctypes.byref(L.GdnTreeProblem(**one)), ctypes.byref(n)) == 0


@pytest.mark.parametrize("name", STRIDES)
def test_tree_over_an_expanded_fp32_cache(L, name):
    assert tree(L, dtype=1, cache_dtype=1, **{name: 0})[1] == 0


@pytest.mark.parametrize("ptrs", [dict(q=None), dict(q=ODD), dict(k_new=None), dict(v_new=ODD), dict(k=ODD), dict(v=None), dict(table=None), dict(lens=None),
                                  dict(parents=None), dict(parents=FAKE + 1), dict(o=ODD), dict(ks=ODD), dict(lse=ODD)])
def test_tree_pointer_refusals(L, ptrs):
    assert tree(L, ptrs=ptrs)[0] == 1


def test_tree_workspace(L):
    assert tree(L, num_seqs=0)[1:] == (0, 0)
    need = tree(L)[2]
    assert need > 0 and tree(L, ws=(None, 0))[0] == 3 and tree(L, ws=(FAKE, need - 1))[0] == 3 and tree(L, ws=(ODD, need))[0] == 1


def write(L, ptrs=None, **kw):
    f = dict(count=4, num_rows=4, Hkv=2, D=64, dtype=0, cache_dtype=0, page_size=16, num_pages=20, k_page_stride=2048, k_token_stride=128, k_head_stride=64,
             v_page_stride=2048, v_token_stride=128, v_head_stride=64)
    f.update(kw)
    a = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, rows=None, ks=None, vs=None)
    a.update(ptrs or {})
    return L.lib().gdn_paged_cache_write(ctypes.byref(L.GdnCacheProblem(**f)), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(num_rows=-1), 1), (dict(num_pages=-1), 1), (dict(count=1 << 32), 2), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(D=72), 2),
    (dict(dtype=1), 1), (dict(cache_dtype=1), 1), (dict(page_size=0), 1), (dict(k_stride=64), 1), (dict(v_stride=130), 1), (dict(k_head_stride=4), 1),
    (dict(v_token_stride=-128), 1), (dict(Hkv=1 << 20), 2),
    (dict(k_page_stride=0), 1), (dict(v_page_stride=0), 1), (dict(k_token_stride=0), 1), (dict(v_token_stride=0), 1), (dict(k_head_stride=0), 1), (dict(v_head_stride=0), 1),
    (dict(ptrs=dict(k=None)), 1), (dict(ptrs=dict(v=ODD)), 1), (dict(ptrs=dict(kc=None)), 1), (dict(ptrs=dict(vc=ODD)), 1), (dict(ptrs=dict(slots=FAKE + 4)), 1),
    (dict(ptrs=dict(slots=None)), 1), (dict(ptrs=dict(rows=ODD)), 1), (dict(ptrs=dict(ks=ODD)), 1), (dict(ptrs=dict(vs=ODD)), 1),
])
def test_write_refusals(L, kw, code):
    assert write(L, **kw) == code and L.lib().gdn_last_error()


def test_write_to_caches_of_one_of_each_has_no_strides_to_check(L):
    assert write(L, num_pages=1, page_size=1, Hkv=1, count=0, k_stride=64, v_stride=64, k_page_stride=0, v_page_stride=0, k_token_stride=0, v_token_stride=0,
                 k_head_stride=0, v_head_stride=0) == 0


def test_write_of_nothing_is_fine(L):
    assert write(L, count=0, ptrs=dict(k=None, v=None, slots=None)) == 0


def table(L, which="extend", ptrs=None, **kw):
    f = dict(num_seqs=2, max_pages=4, page_size=16, stack_size=8, total=4)
    f.update(kw)
    a = dict(table=FAKE, lens=FAKE, change=FAKE, stack=FAKE, free=FAKE)
    if which == "extend":
        a.update(slots=FAKE, cu=FAKE)
    a.update({n: x for n, x in (ptrs or {}).items() if n in a})
    return getattr(L.lib(), "gdn_page_table_" + which)(ctypes.byref(L.GdnTableProblem(**f)), *a.values(), None)


@pytest.mark.parametrize("which", ["extend", "trim"])
@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=-1), 1), (dict(num_seqs=8193), 2), (dict(max_pages=-1), 1), (dict(page_size=0), 1), (dict(stack_size=-1), 1), (dict(total=-1), 1),
    (dict(total=1 << 32), 2), (dict(table_stride=3), 1), (dict(max_pages=1 << 28), 2),
    (dict(ptrs=dict(table=None)), 1), (dict(ptrs=dict(lens=ODD)), 1), (dict(ptrs=dict(change=None)), 1), (dict(ptrs=dict(stack=None)), 1), (dict(ptrs=dict(free=None)), 1),
])
def test_table_refusals(L, which, kw, code):
    assert table(L, which, **kw) == code and L.lib().gdn_last_error()


def test_table_output_refusals(L):
    assert table(L, ptrs=dict(slots=FAKE + 4)) == 1 and table(L, ptrs=dict(slots=None)) == 1 and table(L, ptrs=dict(cu=None)) == 1


def test_wait_timeout_refusals(L):
    for kernels, limit in ((-1, 100), (4, 100), (0, 0), (3, 1000001)):
        assert L.lib().gdn_debug_attn_wait_timeout(kernels, limit, None) == 1 and L.lib().gdn_last_error()


# ------------------------------------------------------------------------------ the Python side
def prompt_args(B=2, T=3, Tk=3, Hq=4, Hkv=2, D=64):
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return dict(q=z(B, T, Hq, D), k=z(B, Tk, Hkv, D), v=z(B, Tk, Hkv, D))


def tree_args(N=3, T=4, Hq=4, Hkv=2, D=64):
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return dict(q=z(N, T, Hq, D), k_new=z(N, T, Hkv, D), v_new=z(N, T, Hkv, D), k_cache=z(5, 16, Hkv, D), v_cache=z(5, 16, Hkv, D),
                page_table=torch.zeros(N, 2, dtype=I32), seq_lens=torch.ones(N, dtype=I32), parents=torch.full((N, T), -1, dtype=I32))


def write_args(n=6, Hkv=2, D=64):
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return dict(k=z(n, Hkv, D), v=z(n, Hkv, D), k_cache=z(5, 16, Hkv, D), v_cache=z(5, 16, Hkv, D), slots=torch.arange(n))


def table_args(N=3):
    z = lambda *s: torch.zeros(*s, dtype=I32)  # noqa: E731
    return dict(page_table=z(N, 4), seq_lens=z(N), free_pages=z(9), num_free=z(1), page_size=16)


def one_row(t, dims=1):
    return t[(slice(0, 1),) * dims].expand(t.shape)


def calls(gdn):
    return [(gdn.prompt_attention, prompt_args()), (gdn.paged_attention_tree, tree_args()), (gdn.paged_cache_write, write_args()),
            (gdn.page_table_extend, dict(table_args(), new_lens=torch.zeros(3, dtype=I32), total=0)),
            (gdn.page_table_trim, dict(table_args(), keep_lens=torch.zeros(3, dtype=I32)))]


def test_host_tensors_are_refused(L):
    for call, args in calls(L):
        with pytest.raises(ValueError, match="CUDA"):
            call(**args)


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_prompt_refuses_expanded_rows(L, name):
    a = prompt_args(1, 6, 6)
    a[name] = one_row(a[name], 2)
    with pytest.raises(ValueError, match=f"the rows of {name} lie at a stride of 0"):
        L.prompt_attention(**a)


@pytest.mark.parametrize("name", ["q", "k_new", "v_new", "page_table"])
def test_tree_refuses_expanded_rows(L, name):
    a = tree_args()
    a[name] = one_row(a[name], 1 if name == "page_table" else 2)
    with pytest.raises(ValueError, match=f"the rows of {name} lie at a stride of 0"):
        L.paged_attention_tree(**a)


def test_write_refuses_expanded_rows(L):
    for name in ("k", "v"):
        a = write_args()
        a[name] = one_row(a[name])
        with pytest.raises(ValueError, match=f"the rows of {name} lie at a stride of 0"):
            L.paged_cache_write(**a)


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(2, 3, 4, 128, dtype=BF)), dict(k=torch.zeros(2, 4, 2, 64, dtype=BF)), dict(v=torch.zeros(2, 3, 2, 64)), dict(q=torch.zeros(2, 3, 256, dtype=BF)),
    dict(cu_seqlens=torch.zeros(3, dtype=I32)), dict(cu_seqlens_k=torch.zeros(3, dtype=I32)), dict(window=-1), dict(k=torch.zeros(1, 3, 2, 64, dtype=BF)),
])
def test_prompt_refuses_shapes(L, kw):
    with pytest.raises(ValueError, match="must|needs|B == 1"):
        L.prompt_attention(**dict(prompt_args(), **kw))


def test_prompt_refuses_other_lengths_of_keys_without_their_own_lengths(L):
    with pytest.raises(ValueError, match="cu_seqlens_k"):
        L.prompt_attention(**prompt_args(1, 3, 5), cu_seqlens=torch.tensor([0, 3], dtype=I32))


@pytest.mark.parametrize("kw", [
    dict(parents=torch.zeros(3, 5, dtype=I32)), dict(parents=torch.zeros(3, 4)), dict(k_new=torch.zeros(3, 4, 4, 64, dtype=BF)), dict(v_new=torch.zeros(3, 4, 2, 64)),
    dict(v_cache=torch.zeros(5, 16, 2, 64)), dict(seq_lens=torch.zeros(4, dtype=I32)), dict(page_table=torch.zeros(2, 2, dtype=I32)), dict(k_scale=torch.ones(3)),
    dict(workspace=torch.zeros(64, dtype=torch.uint8)[::2]), dict(o=torch.zeros(3, 4, 4, 64)),
])
def test_tree_refuses_shapes(L, kw):
    with pytest.raises(ValueError, match="must"):
        L.paged_attention_tree(**dict(tree_args(), **kw))


@pytest.mark.parametrize("kw", [
    dict(slots=torch.zeros(6, dtype=I32)), dict(slots=torch.arange(7)), dict(rows=torch.zeros(5, dtype=I32)), dict(rows=torch.zeros(6)), dict(k=torch.zeros(6, 3, 64, dtype=BF)),
    dict(v=torch.zeros(6, 2, 64)), dict(v_scale=torch.ones(3)), dict(v_cache=torch.zeros(5, 16, 2, 64)),
])
def test_write_refuses_shapes(L, kw):
    with pytest.raises(ValueError, match="must|slots for"):
        L.paged_cache_write(**dict(write_args(), **kw))


@pytest.mark.parametrize("kw", [dict(new_lens=torch.zeros(2, dtype=I32)), dict(new_lens=torch.zeros(3)), dict(total=-1), dict(page_size=0), dict(num_free=torch.zeros(2, dtype=I32)),
                                dict(free_pages=torch.zeros(3)), dict(page_table=torch.zeros(3, 4)), dict(page_table=torch.zeros(3, 8, dtype=I32)[:, ::2]),
                                dict(seq_lens=torch.zeros(3, 1, dtype=I32))])
def test_table_refuses_shapes(L, kw):
    with pytest.raises(ValueError, match="must"):
        L.page_table_extend(**dict(dict(table_args(), new_lens=torch.zeros(3, dtype=I32), total=5), **kw))


@pytest.mark.parametrize("which,name", [(1, n) for n in ("q", "k_new", "v_new", "k_cache", "v_cache")] + [(2, n) for n in ("k", "v", "k_cache", "v_cache")])
def test_calls_for_inference_refuse_gradients(L, which, name):
    call, args = calls(L)[which]
    args[name].requires_grad_(True)
    with pytest.raises(RuntimeError, match="differentiable"):
        call(**args)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call(**args)


@pytest.mark.parametrize("which,name", [(0, "q"), (0, "v"), (1, "q"), (2, "k")])
def test_forward_mode_tangents_are_refused(L, which, name):
    call, args = calls(L)[which]
    with torch.autograd.forward_ad.dual_level():
        args[name] = torch.autograd.forward_ad.make_dual(args[name], torch.ones_like(args[name]))
        with pytest.raises(RuntimeError, match="tangent"):
            call(**args)


def test_a_second_derivative_of_attention_is_refused(L, monkeypatch):
    def fwd(q, k, v, scale, window, cu, cu_k, lse, rest):
        z = scale * torch.einsum("bqhd,bkhd->bhqk", q, k)
        return torch.einsum("bhqk,bkhd->bqhd", z.softmax(-1), v), z.logsumexp(-1).transpose(1, 2), None

    def bwd(q, k, v, o, lse, do, scale, window, cu, cu_k, dlse, rest):
        with torch.enable_grad():
            leaves = [x.detach().requires_grad_(True) for x in (q, k, v)]
            return torch.autograd.grad((fwd(*leaves, scale, 0, None, None, True, True)[0] * do.detach()).sum(), leaves)

    monkeypatch.setattr(L, "gdn_prompt_attn_fwd", fwd)
    monkeypatch.setattr(L, "gdn_prompt_attn_bwd", bwd)
    q = torch.randn(1, 3, 2, 8, generator=torch.Generator().manual_seed(0)).requires_grad_(True)
    o = L.prompt_attention(q, torch.ones(1, 3, 2, 8), torch.ones(1, 3, 2, 8))
    (g,) = torch.autograd.grad(o.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (o.sum() + g.square().sum()).backward()
