"""GPU parity of the RMS norm with the residual's addition, its 8-bit output and its backward pass
against the fp64 oracle.

Tolerances: the sum of squares is a sum of dim positive terms taken as sums over at most dim / 256
of them and a tree, so r is off by a factor of at most 1 +- (64 + dim / 128) 2^-24 =: 1 +- e.  fp32
results are off by 4 e of their terms' size; bf16 ones (8 significant bits) by 2^-8 of the result more; an 8-bit value
by 2^-4 of itself (half a unit of 3 mantissa bits), below 2^-6 by half the smallest step, 2^-10,
of its scale.  dweight sums rows terms: (64 + rows) 2^-24 of their absolute sum."""
import numpy as np
import pytest
import torch

from oracle import decode

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (3, 7), (40, 77), (33, 235), (9, 1001), (3, 5001), (2, 8190), (5, 64), (2, 1000), (17, 1024), (4, 2048), (3, 4100), (2, 5120), (1, 8192), (2, 16384), (1, 20000)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_gb300 import build
    build.build()


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def eps_of(dim):
    return (64 + dim / 128) * 2.0 ** -24


def make(rows, dim, dtype, residual, seed, wdtype=None):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=r(rows, dim).to(dtype), weight=(1 + 0.3 * r(dim)).to(wdtype or dtype), residual=r(rows, dim).mul(2).to(dtype) if residual else None,
                dy=r(rows, dim).to(dtype), dsum=r(rows, dim).to(dtype))


def cuda(d):
    return {n: None if t is None else t.cuda() for n, t in d.items()}


def close(got, ref, size, dtype, e):
    tol = 4 * e * size + (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) if dtype == BF else 0) + 1e-38
    assert (np.abs(np64(got) - ref) <= tol).all(), float((np.abs(np64(got) - ref) - tol).max())


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual,offset", [(False, 0.0), (True, 1.0)])
def test_forward(rows, dim, dtype, residual, offset):
    from chunked_prefill_gb300 import gdn
    d = make(rows, dim, dtype, residual, rows + dim)
    x = cuda(d)
    y, total = gdn.rms_norm(x["x"], x["weight"], residual=x["residual"], eps=1e-5, weight_offset=offset)
    ry, rs = decode.norm(np64(d["x"]), np64(d["weight"]), np64(d["residual"]), 1e-5, offset)
    close(y, ry, np.abs(ry), dtype, eps_of(dim))
    if residual:
        close(total, rs, np.abs(rs), dtype, 2.0 ** -24)
    else:
        assert total is None


@pytest.mark.parametrize("rows,dim,group", [(1, 1, 0), (3, 7, 0), (2, 1000, 8), (17, 1024, 128), (4, 2048, 0), (3, 4100, 4), (2, 5120, 128), (3, 8192, 64),
                                            (2, 16384, 0), (1, 20000, 0), (1, 20000, 32), (2, 384, 384), (2, 768, 256), (2, 640, 5), (33, 235, 0), (9, 1001, 0), (9, 1002, 6), (3, 5001, 0)])
@pytest.mark.parametrize("dtype,residual", [(BF, True), (BF, False), (F32, True)])
def test_8_bit_output(rows, dim, group, dtype, residual):
    from chunked_prefill_gb300 import gdn
    d = make(rows, dim, dtype, residual, rows + dim + group)
    x = cuda(d)
    y, scale, total = gdn.rms_norm_quant(x["x"], x["weight"], residual=x["residual"], group=group)
    ry, rs = decode.norm(np64(d["x"]), np64(d["weight"]), np64(d["residual"]))
    sc = decode.norm_scales(ry, group)
    assert y.dtype == torch.float8_e4m3fn and scale.shape == (rows, dim // group if group else 1)
    assert (np.abs(np64(scale) - sc) <= 4 * eps_of(dim) * sc).all()
    wide = np.repeat(sc, dim // sc.shape[1], 1)
    back = np64(y.float()) * wide
    # 2^-4 of the value, and the few values whose quotient lies at a rounding boundary stay within it
    assert (np.abs(back - ry) <= 2.0 ** -4 * np.abs(ry) * (1 + 1e-3) + 2.0 ** -10 * wide * (1 + 1e-3)).all()
    assert np.abs(np64(y.float())).max() <= 448
    if residual:
        close(total, rs, np.abs(rs), dtype, 2.0 ** -24)


@pytest.mark.parametrize("rows,dim", SHAPES + [(3001, 136), (0, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("with_sum,offset", [(False, 0.0), (True, 1.0)])
def test_backward(rows, dim, dtype, with_sum, offset):
    from chunked_prefill_gb300 import gdn
    d = make(rows, dim, dtype, False, rows + dim)
    x = cuda(d)
    dx, dw = gdn.gdn_rmsnorm_bwd(x["x"], x["weight"], x["dy"], dsum=x["dsum"] if with_sum else None, eps=1e-5, weight_offset=offset)
    rx, rw, sx, sw = decode.norm_bwd(np64(d["x"]), np64(d["weight"]), np64(d["dy"]), np64(d["dsum"]) if with_sum else None, 1e-5, offset)
    close(dx, rx, sx, dtype, eps_of(dim))
    assert (np.abs(np64(dw) - rw) <= ((64 + rows) * 2.0 ** -24 + 4 * eps_of(dim)) * sw + 1e-38).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_autograd(dtype):
    """Through the differentiable call, with rows in two leading dimensions: x and residual get
    the same gradient, the backward pass takes the sum as it was rounded."""
    from chunked_prefill_gb300 import gdn
    d = make(6, 256, dtype, True, 3, wdtype=F32)
    x = {n: t.cuda() for n, t in d.items()}
    leaf = {n: x[n].requires_grad_(True) for n in ("x", "weight", "residual")}
    y, total = gdn.rms_norm(leaf["x"].view(2, 3, 256), leaf["weight"], residual=leaf["residual"].view(2, 3, 256))
    ((y.float() * x["dy"].view(2, 3, 256).float()).sum() + (total.float() * x["dsum"].view(2, 3, 256).float()).sum()).backward()
    s = np64(total).reshape(6, 256)
    rx, rw, sx, sw = decode.norm_bwd(s, np64(d["weight"]), np64(d["dy"]), np64(d["dsum"]))
    close(leaf["x"].grad, rx, sx, dtype, eps_of(256))
    assert torch.equal(leaf["x"].grad, leaf["residual"].grad)
    assert (np.abs(np64(leaf["weight"].grad) - rw) <= (80 * 2.0 ** -24 + 4 * eps_of(256)) * sw).all()
    # one output unused
    for pick in (0, 1):
        x2 = d["x"].cuda().requires_grad_(True)
        out = gdn.rms_norm(x2, x["weight"].detach(), residual=x["residual"].detach())[pick]
        (out.float() * x["dy"].float()).sum().backward()
        want = decode.norm_bwd(s, np64(d["weight"]), np64(d["dy"]))[0] if pick == 0 else np64(d["dy"])
        assert np.abs(np64(x2.grad) - want).max() <= 2.0 ** -7 * np.abs(want).max()


@pytest.mark.parametrize("dim", [256, 250])
def test_strided_rows(dim):
    """Rows inside wider rows, on 16-byte boundaries and off them: the bits of contiguous rows."""
    from chunked_prefill_gb300 import gdn
    d = make(9, dim, BF, True, 5)
    x = cuda(d)
    want = gdn.rms_norm(x["x"], x["weight"], residual=x["residual"])
    gwant = gdn.gdn_rmsnorm_bwd(x["x"], x["weight"], x["dy"], dsum=x["dsum"])
    for lead, pad in ((8, 8), (1, 3)):
        wide = {n: torch.zeros(9, lead + dim + pad, dtype=BF, device="cuda") for n in ("x", "residual", "dy", "dsum")}
        v = {}
        for n, w in wide.items():
            v[n] = w[:, lead:lead + dim]
            v[n].copy_(x[n])
        tol = 2.0 ** -8
        got = gdn.rms_norm(v["x"], x["weight"], residual=v["residual"])
        for a, b in zip(got + gdn.gdn_rmsnorm_bwd(v["x"], x["weight"], v["dy"], dsum=v["dsum"]), want + gwant):
            assert ((a.float() - b.float()).abs() <= tol * b.float().abs() + 1e-6).all()


def test_degenerate_rows():
    """A zero row gives zeros with the smallest scale (no division by zero), rows with infinities
    and NaN give NaN in those rows alone, and large and tiny rows neither overflow nor vanish."""
    from chunked_prefill_gb300 import gdn
    x = torch.randn(6, 512, generator=torch.Generator().manual_seed(1)).cuda()
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] *= 1e15
    x[4] *= 1e-18
    w = torch.ones(512, device="cuda")
    y, _ = gdn.rms_norm(x, w, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 5])
    for i in (3, 5):
        ref = decode.norm(np64(x[i:i + 1]), np.ones(512), eps=0.0)[0]
        assert np.abs(np64(y[i:i + 1]) - ref).max() <= 1e-5 * np.abs(ref).max()
    y8, scale, _ = gdn.rms_norm_quant(x, w, eps=1e-6)
    assert (y8[0].float() == 0).all() and scale[0, 0] == 2.0 ** -126
    assert torch.isnan(scale[1]).all() and torch.isnan(y8[1].float()).all() and torch.isnan(scale[2]).all()
    assert torch.isfinite(y8[3:].float()).all() and torch.isfinite(scale[3:]).all()


def test_determinism_and_stream():
    from chunked_prefill_gb300 import gdn
    d = make(4000, 1000, BF, False, 2)
    x = cuda(d)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    a = gdn.gdn_rmsnorm_bwd(x["x"], x["weight"], x["dy"])
    with torch.cuda.stream(st):
        b = gdn.gdn_rmsnorm_bwd(x["x"], x["weight"], x["dy"])
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    from chunked_prefill_gb300 import gdn
    x, w = torch.zeros(4, 64, device="cuda", dtype=BF), torch.ones(64, device="cuda", dtype=BF)
    for bad in (lambda: gdn.rms_norm(x.cpu(), w), lambda: gdn.rms_norm(x, w[:32]), lambda: gdn.rms_norm(x, w, residual=x[:2]),
                lambda: gdn.rms_norm(x, w, residual=x.float()), lambda: gdn.rms_norm(x.t(), torch.ones(4, device="cuda", dtype=BF)),
                lambda: gdn.rms_norm_quant(x, w, group=48), lambda: gdn.gdn_rmsnorm_bwd(x, w, x.float())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gdn.GdnError):
        gdn.rms_norm(x, w, eps=-1.0)
    with pytest.raises(gdn.GdnError):
        gdn.rms_norm(x, w, weight_offset=float("inf"))
    with pytest.raises(TypeError):
        gdn.rms_norm(x.half(), w)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,dim", [(5, 1024), (7, 1001), (3, 235), (2, 20000)])
def test_in_place(dtype, rows, dim):
    """sum over the residual and y over x; dx over dy: the bits of the calls with outputs of their own."""
    import ctypes
    from chunked_prefill_gb300 import gdn
    d = make(rows, dim, dtype, True, 6)
    x = cuda(d)
    want = gdn.rms_norm(x["x"], x["weight"], residual=x["residual"])
    code = gdn._dtype_code(dtype)
    p = gdn.GdnNormProblem(rows, dim, code, code, code, 0, 1e-6, 0.0)
    xi, ri, dyi = x["x"].clone(), x["residual"].clone(), x["dy"].clone()
    L = gdn.lib()
    gdn._check(L.gdn_rmsnorm_fwd(ctypes.byref(p), xi.data_ptr(), ri.data_ptr(), x["weight"].data_ptr(), xi.data_ptr(), None, ri.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream))
    assert torch.equal(xi, want[0]) and torch.equal(ri, want[1])
    gwant = gdn.gdn_rmsnorm_bwd(x["x"], x["weight"], x["dy"])
    n = ctypes.c_size_t(0)
    gdn._check(L.gdn_rmsnorm_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    ws, dw = torch.empty(n.value, dtype=torch.uint8, device="cuda"), torch.empty(dim, device="cuda")
    gdn._check(L.gdn_rmsnorm_bwd(ctypes.byref(p), x["x"].data_ptr(), x["weight"].data_ptr(), dyi.data_ptr(), None, dyi.data_ptr(), dw.data_ptr(),
                                 ws.data_ptr(), n.value, torch.cuda.current_stream().cuda_stream))
    assert torch.equal(dyi, gwant[0]) and torch.equal(dw, gwant[1])


def test_shapes_alternate():
    """Calls of one kernel with more and less shared memory, in turn."""
    from chunked_prefill_gb300 import gdn
    for _ in range(2):
        for rows, dim, group in ((2, 16384, 1), (2, 12000, 3), (2, 14000, 1)):
            d = make(rows, dim, BF, True, dim)
            x = cuda(d)
            y, scale, _ = gdn.rms_norm_quant(x["x"], x["weight"], residual=x["residual"], group=group)
            ry = decode.norm(np64(d["x"]), np64(d["weight"]), np64(d["residual"]))[0]
            sc = decode.norm_scales(ry, group)
            assert (np.abs(np64(scale) - sc) <= 4 * eps_of(dim) * sc).all()
        for rows, dim in ((700, 8192), (700, 5000), (700, 7999)):
            d = make(rows, dim, BF, False, dim)
            x = cuda(d)
            dx, dw = gdn.gdn_rmsnorm_bwd(x["x"], x["weight"], x["dy"], dsum=x["dsum"])
            rx, rw, sx, sw = decode.norm_bwd(np64(d["x"]), np64(d["weight"]), np64(d["dy"]), np64(d["dsum"]))
            close(dx, rx, sx, BF, eps_of(dim))
            assert (np.abs(np64(dw) - rw) <= ((64 + rows) * 2.0 ** -24 + 4 * eps_of(dim)) * sw + 1e-38).all()


def test_rows_past_32_bit_offsets():
    """More than 2^31 values: the last rows are those of a call on them alone, in every direction."""
    from chunked_prefill_gb300 import gdn
    dim, rows, tail = 16384, 131080, 24
    assert rows * dim > 2 ** 31
    x = torch.randn(rows, dim, device="cuda", dtype=BF)
    w = torch.randn(dim, device="cuda", dtype=BF)
    y, _ = gdn.rms_norm(x, w)
    assert torch.equal(y[-tail:], gdn.rms_norm(x[-tail:].contiguous(), w)[0])
    y8, scale, _ = gdn.rms_norm_quant(x, w, group=128)
    z8, zscale, _ = gdn.rms_norm_quant(x[-tail:].contiguous(), w, group=128)
    assert torch.equal(y8[-tail:].view(torch.uint8), z8.view(torch.uint8)) and torch.equal(scale[-tail:], zscale)
    dx, _ = gdn.gdn_rmsnorm_bwd(x, w, y)
    assert torch.equal(dx[-tail:], gdn.gdn_rmsnorm_bwd(x[-tail:].contiguous(), w, y[-tail:].contiguous())[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 512, 1001, 2048, 20000])
def test_rows_of_every_size_match_the_oracle(dtype, dim):
    """Rows of 1e15, of 1 and of 1e-18 without eps, and down to subnormal ones beside it, where the 8-bit
    scale ends at 2^-126: values, scales and gradients against the oracle, none of them lost."""
    from chunked_prefill_gb300 import gdn
    gen = torch.Generator().manual_seed(dim)
    w = torch.ones(dim, dtype=dtype)
    sizes = torch.tensor([1e15, 1.0, 1e-18])[:, None]
    x, dy = (torch.randn(3, dim, generator=gen) * sizes).to(dtype), torch.randn(3, dim, generator=gen).to(dtype)
    y, _ = gdn.rms_norm(x.cuda(), w.cuda(), eps=0.0)
    ry = decode.norm(np64(x), np64(w), eps=0.0)[0]
    close(y, ry, np.abs(ry), dtype, eps_of(dim))
    assert (np.abs(np64(y)).max(1) > 1).all()
    dx, _ = gdn.gdn_rmsnorm_bwd(x.cuda(), w.cuda(), dy.cuda(), eps=0.0)
    rx, _, sx, _ = decode.norm_bwd(np64(x), np64(w), np64(dy), eps=0.0)
    close(dx, rx, sx, dtype, eps_of(dim))
    tiny = (torch.randn(4, dim, generator=gen) * torch.tensor([1e15, 1e-18, 1e-30, 1e-39])[:, None]).to(dtype)
    for rows, eps in ((x, 0.0), (tiny, 1e-6)):
        y8, scale, _ = gdn.rms_norm_quant(rows.cuda(), w.cuda(), eps=eps)
        ry = decode.norm(np64(rows), np64(w), eps=eps)[0]
        sc = decode.norm_scales(ry)
        assert (np.abs(np64(scale) - sc) <= 4 * eps_of(dim) * sc).all()
        assert (np.abs(np64(y8.float()) * sc - ry) <= 2.0 ** -4 * np.abs(ry) * (1 + 1e-3) + 2.0 ** -10 * sc * (1 + 1e-3)).all()
        assert (np.abs(np64(y8.float())).max(1) >= 32).all()
