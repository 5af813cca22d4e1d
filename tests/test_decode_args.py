"""What the decoding calls' Python side refuses, on the CPU: the shapes, strides and gradients of the
arguments are looked at before their devices, so host tensors reach these checks."""
import pytest
import torch

from chunked_prefill_gb300 import build as gbuild

BF = torch.bfloat16


@pytest.fixture(scope="module")
def gdn():
    gbuild.build()
    from chunked_prefill_gb300 import gdn
    return gdn


def step_args(B=4, T=1, Hqk=1, Hv=2):
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return dict(q=z(B, T, Hqk, 128), k=z(B, T, Hqk, 128), v=z(B, T, Hv, 128), g=torch.zeros(B, T, Hv), beta=torch.zeros(B, T, Hv),
                state=torch.zeros(B, Hv, 128, 128))


def paged_args(N=3, Hq=4, Hkv=2, D=64):
    return dict(q=torch.zeros(N, Hq, D, dtype=BF), k_cache=torch.zeros(5, 16, Hkv, D, dtype=BF), v_cache=torch.zeros(5, 16, Hkv, D, dtype=BF),
                page_table=torch.zeros(N, 2, dtype=torch.int32), seq_lens=torch.ones(N, dtype=torch.int32))


def one_row(t, dims=1):
    """All rows the first one, as an expanded view."""
    return t[(slice(0, 1),) * dims].expand(t.shape)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("B,T", [(4, 1), (1, 4), (2, 3)])
def test_step_refuses_expanded_rows(gdn, name, B, T):
    """A stride of 0 means contiguous rows to the C ABI: an expanded view would be read past its end."""
    a = step_args(B, T)
    a[name] = one_row(a[name], 2)
    with pytest.raises(ValueError, match=f"the rows of {name} lie at a stride of 0"):
        gdn.gated_delta_rule_step(**a)


@pytest.mark.parametrize("name", ["q", "page_table"])
def test_attention_refuses_expanded_rows(gdn, name):
    a = paged_args()
    a[name] = one_row(a[name])
    with pytest.raises(ValueError, match=f"the rows of {name} lie at a stride of 0"):
        gdn.paged_attention_decode(**a)


def test_attention_refuses_an_expanded_new_token(gdn):
    a = paged_args()
    new = one_row(torch.zeros(3, 2, 64, dtype=BF))
    with pytest.raises(ValueError, match="the rows of k_new and v_new lie at a stride of 0"):
        gdn.paged_attention_decode(**a, k_new=new, v_new=new)


@pytest.mark.parametrize("dim", [1, 8, 64])
def test_norm_refuses_expanded_rows(gdn, dim):
    x, w = torch.zeros(5, dim), torch.ones(dim)
    one = one_row(torch.zeros(5, dim))
    for name, call in (("x", lambda: gdn.rms_norm(one, w)), ("residual", lambda: gdn.rms_norm(x, w, residual=one)),
                       ("residual", lambda: gdn.rms_norm_quant(x, w, residual=one)), ("s", lambda: gdn.gdn_rmsnorm_bwd(one, w, x)),
                       ("dy", lambda: gdn.gdn_rmsnorm_bwd(x, w, one)), ("dsum", lambda: gdn.gdn_rmsnorm_bwd(x, w, x, dsum=one))):
        with pytest.raises(ValueError, match=f"the rows of {name} lie at a stride of 0"):
            call()


def test_one_row_may_have_any_stride(gdn):
    """A single row, and no rows, have no distance between rows: these get as far as their device."""
    a = step_args(1, 1)
    a["beta"] = torch.zeros(1).expand(1, 1, 2).contiguous().as_strided((1, 1, 2), (0, 0, 1))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_delta_rule_step(**a)
    a = paged_args(N=1)
    a["q"], a["page_table"] = a["q"].as_strided((1, 4, 64), (0, 64, 1)), a["page_table"].as_strided((1, 2), (0, 1))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.paged_attention_decode(**a)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.rms_norm(torch.zeros(64).as_strided((1, 64), (0, 1)), torch.ones(64))


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 12, dtype=torch.uint8)[::2]])
def test_a_workspace_that_is_not_contiguous_is_refused(gdn, ws):
    """A view's values need not be bytes of its own: the kernels would write past them."""
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        gdn.paged_attention_decode(**paged_args(), workspace=ws)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        gdn.gdn_rmsnorm_bwd(torch.zeros(3, 8), torch.ones(8), torch.zeros(3, 8), workspace=ws)


@pytest.mark.parametrize("name", ["x", "weight", "residual"])
def test_the_8_bit_norm_refuses_gradients(gdn, name):
    """Its outputs carry no gradient: the residual stream would be cut without a word."""
    a = dict(x=torch.zeros(3, 8), weight=torch.ones(8), residual=torch.zeros(3, 8))
    a[name].requires_grad_(True)
    with pytest.raises(RuntimeError, match="differentiable"):
        gdn.rms_norm_quant(**a)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # as far as the device
        gdn.rms_norm_quant(**a)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "state", "state_out", "A_log", "dt_bias"])
def test_the_step_refuses_gradients(gdn, name):
    a = dict(step_args(), state_out=torch.zeros(4, 2, 128, 128), A_log=torch.zeros(2), dt_bias=torch.zeros(2))
    a[name].requires_grad_(True)
    with pytest.raises(RuntimeError, match="differentiable"):
        gdn.gated_delta_rule_step(**a)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        gdn.gated_delta_rule_step(**a)


@pytest.mark.parametrize("name", ["q", "k_cache", "v_cache", "k_new", "v_new", "k_scale", "v_scale"])
def test_attention_refuses_gradients(gdn, name):
    new = lambda: torch.zeros(3, 2, 64, dtype=BF)  # noqa: E731
    a = dict(paged_args(), k_new=new(), v_new=new(), k_scale=torch.ones(2), v_scale=torch.ones(2))
    a[name].requires_grad_(True)
    with pytest.raises(RuntimeError, match="differentiable"):
        gdn.paged_attention_decode(**a)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        gdn.paged_attention_decode(**a)


def test_a_second_derivative_of_the_norm_is_refused(gdn, monkeypatch):
    """The gradient kernel has no derivative: a penalty on the norm's gradient must not train on zeros."""
    def fwd(x, weight, residual, eps, offset):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * (weight + offset), None, None

    def bwd(s, weight, dy, dsum, eps, offset):
        with torch.enable_grad():
            at = s.detach().requires_grad_(True)
            return torch.autograd.grad((fwd(at, weight.detach(), None, eps, offset)[0] * dy.detach()).sum(), at)[0], torch.zeros(s.shape[-1])

    monkeypatch.setattr(gdn, "gdn_rmsnorm_fwd", fwd)
    monkeypatch.setattr(gdn, "gdn_rmsnorm_bwd", bwd)
    x = torch.randn(3, 8, generator=torch.Generator().manual_seed(0)).requires_grad_(True)
    y, _ = gdn.rms_norm(x, torch.ones(8))
    (gx,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (y.sum() + gx.square().sum()).backward()


@pytest.mark.parametrize("no_grad", [False, True])
def test_forward_mode_tangents_are_refused(gdn, no_grad):
    """No call has a forward-mode derivative: a tangent must not be dropped."""
    step, attn = step_args(), paged_args()
    x, w = torch.zeros(3, 8), torch.ones(8)
    with torch.autograd.forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
        dual = lambda t: torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: gdn.rms_norm(dual(x), w), lambda: gdn.rms_norm(x, dual(w)), lambda: gdn.rms_norm(x, w, residual=dual(x)),
                     lambda: gdn.rms_norm_quant(dual(x), w), lambda: gdn.gated_delta_rule_step(**dict(step, v=dual(step["v"]))),
                     lambda: gdn.paged_attention_decode(**dict(attn, q=dual(attn["q"])))):
            with pytest.raises(RuntimeError, match="tangent"):
                call()


def test_the_binding_is_built_again_for_another_torch_or_python(gdn, monkeypatch):
    assert not gbuild._binding_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", torch.__version__ + ".post1")
        assert gbuild._binding_stale()
    with monkeypatch.context() as m:
        m.setattr(gbuild.sys.implementation, "cache_tag", "cpython-300")
        assert gbuild._binding_stale()
    assert not gbuild._binding_stale()
