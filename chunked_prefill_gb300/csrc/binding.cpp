// Native argument marshalling of the decoding operators for Python: checks tensors, fills the C
// ABI's problem structures and calls libgdn.so.  A decoding step is made of many calls that take a
// few microseconds on the GPU, and the same checks written in Python cost 20 to 30 us a call.
// Nothing is computed here.  The library's functions are handed over by address (bind), so that this
// module and the ctypes binding use one and the same loaded library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/gdn.h"

namespace {

struct Bad {
    PyObject* type;  // NULL: the Python error is set already
    std::string msg;
};
void need(bool ok, const char* msg) {
    if (!ok) throw Bad{PyExc_ValueError, msg};
}
void need(bool ok, const std::string& msg) {
    if (!ok) throw Bad{PyExc_ValueError, msg};
}

decltype(&gdn_recurrent_step) f_step;
decltype(&gdn_paged_attn_workspace_size) f_paged_size;
decltype(&gdn_paged_attn_decode) f_paged;
decltype(&gdn_rmsnorm_fwd) f_norm_fwd;
decltype(&gdn_rmsnorm_bwd_workspace_size) f_norm_bwd_size;
decltype(&gdn_rmsnorm_bwd) f_norm_bwd;
PyObject* on_error;  // called with a status that is not GDN_OK; raises

void check(gdn_status st) {
    if (st == GDN_OK) return;
    PyObject* r = PyObject_CallFunction(on_error, "i", int(st));
    Py_XDECREF(r);
    throw Bad{nullptr, ""};
}

// ---- arguments
struct Args {
    PyObject* const* a;
    Py_ssize_t n, at = 0;
    PyObject* next() {
        if (at >= n) throw Bad{PyExc_TypeError, "too few arguments"};
        return a[at++];
    }
    const at::Tensor& tensor(const char* name) {
        PyObject* o = next();
        if (!THPVariable_Check(o)) throw Bad{PyExc_TypeError, std::string(name) + " must be a tensor"};
        return THPVariable_Unpack(o);
    }
    const at::Tensor* maybe(const char* name) {
        PyObject* o = next();
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) throw Bad{PyExc_TypeError, std::string(name) + " must be a tensor or None"};
        return &THPVariable_Unpack(o);
    }
    double number() {
        const double x = PyFloat_AsDouble(next());
        if (x == -1.0 && PyErr_Occurred()) throw Bad{nullptr, ""};
        return x;
    }
    int64_t integer() {
        const int64_t x = PyLong_AsLongLong(next());
        if (x == -1 && PyErr_Occurred()) throw Bad{nullptr, ""};
        return x;
    }
    bool flag() {
        const int x = PyObject_IsTrue(next());
        if (x < 0) throw Bad{nullptr, ""};
        return x != 0;
    }
};

// The device and stream of a call: a torch.cuda.Stream (the last argument), or None for the device's
// current one.  What the call allocates belongs to that stream.
struct On {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard guard;
    void* stream;
    On(const at::Tensor& t, Args& a) : device(t.device()) {
        PyObject* o = a.next();
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
            return;
        }
        PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw Bad{nullptr, ""};
        stream = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!stream && PyErr_Occurred()) throw Bad{nullptr, ""};
        guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), t.device().index()));
    }
};

void need_cuda(const at::Tensor& like, const char* name, const at::Tensor& t) {
    need(t.is_cuda() && t.device() == like.device(), std::string(name) + " must be a CUDA tensor on the device of the others");
}
void need_cuda(const at::Tensor& like, const char* name, const at::Tensor* t) {
    if (t) need_cuda(like, name, *t);
}
int code(const at::Tensor& t, const char* what) {
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_FP32;
    throw Bad{PyExc_TypeError, std::string(what) + " must be bfloat16 or float32, got " + c10::toString(t.scalar_type())};
}
template <typename T = float> T* ptr(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
template <typename T = float> T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}
// The caller's scratch: its bytes are counted from its values, which a strided or expanded view has not all of.
void need_scratch(const at::Tensor* t) {
    if (t) need(t->is_contiguous(), "workspace must be contiguous");
}
// device scratch of n bytes: the caller's where it is large enough
at::Tensor scratch(size_t n, const at::Tensor* given, const at::Tensor& like) {
    if (n == 0) return like;  // not used
    if (given && size_t(given->numel()) * given->element_size() >= n) return *given;
    return empty({int64_t(n < 16 ? 16 : n)}, at::kByte, like);
}
void need_vector(const char* name, const at::Tensor* t, at::ScalarType type, int64_t n, const char* what) {
    if (t) need(t->scalar_type() == type && t->dim() == 1 && t->size(0) == n && t->is_contiguous(), std::string(name) + " must be a contiguous " + what);
}

// The stride of rows of which there is more than one.  The C ABI's 0 stands for contiguous rows, so an
// expanded view (every row the same one) would be read past its end.
int64_t apart(const char* name, int64_t stride) {
    if (stride == 0) throw Bad{PyExc_ValueError, std::string("the rows of ") + name + " lie at a stride of 0 (an expanded view): pass a contiguous copy"};
    return stride;
}

// Elements from one token to the next of a [B, T, ...] tensor whose last dimensions are contiguous
// (`inner` values) and whose tokens lie at one stride.
int64_t token_stride(const char* name, const at::Tensor& t, int64_t inner) {
    int64_t want = 1;
    for (int64_t d = t.dim() - 1; d > 1; --d) {
        need(t.size(d) == 1 || t.stride(d) == want, std::string("the heads and features of ") + name + " must be contiguous");
        want *= t.size(d);
    }
    const int64_t B = t.size(0), T = t.size(1);
    if (B * T <= 1) return inner;
    if (T == 1) return apart(name, t.stride(0));
    need(B == 1 || t.stride(0) == T * t.stride(1), std::string("the tokens of ") + name + " must lie at one stride");
    return apart(name, t.stride(1));
}

PyObject* step(Args& a) {
    const at::Tensor &q = a.tensor("q"), &k = a.tensor("k"), &v = a.tensor("v"), &g = a.tensor("g"), &beta = a.tensor("beta");
    const double scale = a.number();
    const at::Tensor *in = a.maybe("state_in"), *out = a.maybe("state_out"), *slots = a.maybe("slots"), *cu = a.maybe("cu_seqlens"),
                     *A_log = a.maybe("A_log"), *bias = a.maybe("dt_bias"), *given = a.maybe("o");
    need(q.dim() == 4 && k.sizes() == q.sizes() && v.dim() == 4 && v.size(0) == q.size(0) && v.size(1) == q.size(1) && v.size(2) > 0 && q.size(2) > 0,
         "q and k must be [B,T,Hqk,K] and v [B,T,Hv,V]");
    need(k.scalar_type() == q.scalar_type() && v.scalar_type() == q.scalar_type(), "q, k and v must match in dtype");
    const int64_t B = q.size(0), T = q.size(1), Hqk = q.size(2), K = q.size(3), Hv = v.size(2), V = v.size(3);
    need(g.dim() == 3 && g.size(0) == B && g.size(1) == T && g.size(2) == Hv && beta.sizes() == g.sizes(), "g and beta must be [B,T,Hv]");
    need(g.scalar_type() == at::kFloat && beta.scalar_type() == at::kFloat, "g and beta must be float32");
    need(B * T < (int64_t(1) << 31) && Hqk < (1 << 30) && Hv < (1 << 30) && K < (1 << 30) && V < (1 << 30), "too many tokens or heads");
    gdn_step_problem p{};
    int64_t n = B;
    if (cu) {
        need(B == 1, "cu_seqlens needs B == 1");
        need(cu->scalar_type() == at::kInt && cu->dim() == 1 && cu->numel() >= 1 && cu->is_contiguous(), "cu_seqlens must be a contiguous int32 [num_seqs+1]");
        n = cu->numel() - 1;
        p.cu_seqlens = ptr<int32_t>(cu);
    }
    need_vector("slots", slots, at::kInt, n, "int32 [num_seqs]");
    int64_t num_slots = n;
    for (const auto& [name, pool] : {std::pair{"state_in", in}, std::pair{"state_out", out}}) {
        if (!pool) continue;
        need(pool->scalar_type() == at::kFloat && pool->dim() == 4 && pool->size(1) == Hv && pool->size(2) == K && pool->size(3) == V && pool->is_contiguous(),
             std::string(name) + " must be a contiguous float32 [num_slots,Hv,K,V]");
        num_slots = pool->size(0);
    }
    if (in && out) need(in->size(0) == out->size(0), "state_in and state_out must have the same slots");
    need(slots || num_slots >= n, std::to_string(num_slots) + " slots for " + std::to_string(n) + " sequences");
    need_vector("A_log", A_log, at::kFloat, Hv, "float32 [Hv]");
    need_vector("dt_bias", bias, at::kFloat, Hv, "float32 [Hv]");
    if (given) need(given->sizes() == v.sizes() && given->scalar_type() == v.scalar_type() && given->is_contiguous(), "o must be contiguous and match v");
    p.num_seqs = int32_t(n);
    p.total_tokens = int32_t(B * T);
    p.Hqk = int32_t(Hqk);
    p.Hv = int32_t(Hv);
    p.K = int32_t(K);
    p.V = int32_t(V);
    p.dtype = code(q, "q, k and v");
    p.scale = float(scale);
    p.slots = ptr<int32_t>(slots);
    p.num_slots = num_slots;
    p.q_stride = token_stride("q", q, Hqk * K);
    p.k_stride = token_stride("k", k, Hqk * K);
    p.v_stride = token_stride("v", v, Hv * V);
    p.g_stride = token_stride("g", g, Hv);
    p.beta_stride = token_stride("beta", beta, Hv);
    need_cuda(q, "q", q);
    need_cuda(q, "k", k);
    need_cuda(q, "v", v);
    need_cuda(q, "g", g);
    need_cuda(q, "beta", beta);
    need_cuda(q, "state_in", in);
    need_cuda(q, "state_out", out);
    need_cuda(q, "slots", slots);
    need_cuda(q, "cu_seqlens", cu);
    need_cuda(q, "A_log", A_log);
    need_cuda(q, "dt_bias", bias);
    need_cuda(q, "o", given);
    On on(q, a);
    const at::Tensor o = given ? *given : empty(v.sizes(), v.scalar_type(), v);
    p.clear_rest = !given;  // what the allocator hands out is not a result
    check(f_step(&p, q.data_ptr(), k.data_ptr(), v.data_ptr(), ptr(g), ptr(beta), ptr(A_log), ptr(bias), ptr(in), ptr(out), o.data_ptr(), on.stream));
    return THPVariable_Wrap(o);
}

int cache_code(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_FP32;
    need(t.scalar_type() == at::kFloat8_e4m3fn, "k_cache and v_cache must both be bfloat16, float32 or float8_e4m3fn");
    return GDN_E4M3;
}
int32_t small(int64_t x, const char* what) {
    need(x < (int64_t(1) << 31), std::string("too many ") + what);
    return int32_t(x);
}

PyObject* paged(Args& a) {
    const at::Tensor &q = a.tensor("q"), &kc = a.tensor("k_cache"), &vc = a.tensor("v_cache"), &table = a.tensor("page_table"), &lens = a.tensor("seq_lens");
    const double scale = a.number();
    const at::Tensor *kn = a.maybe("k_new"), *vn = a.maybe("v_new"), *ks = a.maybe("k_scale"), *vs = a.maybe("v_scale");
    const int64_t window = a.integer();
    const at::Tensor* given = a.maybe("o");
    const bool make_lse = a.at < a.n && a.a[a.at] == Py_True;  // lse: a tensor, None, or True for a new one
    const at::Tensor* lse = nullptr;
    if (make_lse)
        ++a.at;
    else
        lse = a.maybe("lse");
    const at::Tensor* ws = a.maybe("workspace");
    need(q.dim() == 3 && kc.dim() == 4 && vc.sizes() == kc.sizes(), "q must be [N,Hq,D], k_cache and v_cache [num_pages,page_size,Hkv,D]");
    const int64_t N = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = kc.size(2);
    need(kc.size(3) == D, "q and the caches must match in D");
    need(vc.scalar_type() == kc.scalar_type(), "k_cache and v_cache must both be bfloat16, float32 or float8_e4m3fn");
    need(table.scalar_type() == at::kInt && table.dim() == 2 && table.size(0) == N && (table.size(1) <= 1 || table.stride(1) == 1),
         "page_table must be int32 [N,max_pages] with contiguous rows");
    need(lens.scalar_type() == at::kInt && lens.dim() == 1 && lens.size(0) == N && lens.is_contiguous(), "seq_lens must be a contiguous int32 [N]");
    need((kn == nullptr) == (vn == nullptr), "k_new and v_new go together");
    auto rows = [&](const char* name, const at::Tensor& t, int64_t heads) {
        need(t.dim() == 3 && t.size(0) == N && t.size(1) == heads && t.size(2) == D && t.scalar_type() == q.scalar_type(),
             std::string(name) + " must be [N," + std::to_string(heads) + ",D] of q's dtype");
        need(t.stride(2) == 1 && (heads == 1 || t.stride(1) == D), std::string("the heads and features of ") + name + " must be contiguous");
    };
    rows("q", q, Hq);
    gdn_paged_problem p{};
    if (kn) {
        rows("k_new", *kn, Hkv);
        rows("v_new", *vn, Hkv);
        if (N > 1) {
            need(kn->stride(0) == vn->stride(0), "k_new and v_new must have the same row stride");
            p.new_stride = apart("k_new and v_new", kn->stride(0));
        }
    }
    need_vector("k_scale", ks, at::kFloat, Hkv, "float32 [Hkv]");
    need_vector("v_scale", vs, at::kFloat, Hkv, "float32 [Hkv]");
    need(kc.stride(3) == 1 && vc.stride(3) == 1, "the features of the caches must be contiguous");
    if (given) need(given->sizes() == q.sizes() && given->scalar_type() == q.scalar_type() && given->is_contiguous(), "o must be contiguous and match q");
    if (lse) need(lse->dim() == 2 && lse->size(0) == N && lse->size(1) == Hq && lse->scalar_type() == at::kFloat && lse->is_contiguous(), "lse must be a contiguous float32 [N,Hq]");
    need(window < (int64_t(1) << 31), "window too large");
    p.num_seqs = small(N, "sequences");
    p.Hq = small(Hq, "heads");
    p.Hkv = small(Hkv, "heads");
    p.D = small(D, "features");
    p.dtype = code(q, "q");
    p.cache_dtype = cache_code(kc);
    p.scale = float(scale);
    p.window = int32_t(window < 0 ? -1 : window);
    p.page_size = small(kc.size(1), "tokens to a page");
    p.max_pages = small(table.size(1), "pages");
    p.num_pages = kc.size(0);
    p.q_stride = N > 1 ? apart("q", q.stride(0)) : 0;
    p.table_stride = N > 1 && table.size(1) > 0 ? apart("page_table", table.stride(0)) : 0;
    p.k_page_stride = kc.stride(0);
    p.k_token_stride = kc.stride(1);
    p.k_head_stride = kc.stride(2);
    p.v_page_stride = vc.stride(0);
    p.v_token_stride = vc.stride(1);
    p.v_head_stride = vc.stride(2);
    need_scratch(ws);
    need_cuda(q, "q", q);
    need_cuda(q, "k_cache", kc);
    need_cuda(q, "v_cache", vc);
    need_cuda(q, "page_table", table);
    need_cuda(q, "seq_lens", lens);
    need_cuda(q, "k_new", kn);
    need_cuda(q, "v_new", vn);
    need_cuda(q, "k_scale", ks);
    need_cuda(q, "v_scale", vs);
    need_cuda(q, "o", given);
    need_cuda(q, "lse", lse);
    need_cuda(q, "workspace", ws);
    On on(q, a);
    size_t bytes = 0;
    check(f_paged_size(&p, &bytes));
    const at::Tensor work = scratch(bytes, ws, q), o = given ? *given : empty(q.sizes(), q.scalar_type(), q);
    at::Tensor new_lse;
    if (make_lse) {
        new_lse = empty({N, Hq}, at::kFloat, q);
        lse = &new_lse;
    }
    check(f_paged(&p, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ptr<int32_t>(table), ptr<int32_t>(lens), ptr<void>(kn), ptr<void>(vn), ptr(ks), ptr(vs),
                  o.data_ptr(), ptr(lse), bytes ? work.data_ptr() : nullptr, bytes ? size_t(work.numel()) * work.element_size() : 0, on.stream));
    if (!make_lse) return THPVariable_Wrap(o);
    PyObject* r = PyTuple_New(2);
    if (!r) throw Bad{nullptr, ""};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(o));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(new_lse));
    return r;
}

// The elements between the rows of a [..., dim] tensor (0: contiguous).
int64_t row_stride(const char* name, const at::Tensor& t) {
    if (t.is_contiguous()) return 0;
    need(t.dim() == 2 && t.stride(1) == 1, std::string(name) + " must be contiguous, or two-dimensional with contiguous rows");
    return t.size(0) > 1 ? apart(name, t.stride(0)) : 0;
}
void like_rows(const char* name, const at::Tensor& t, const at::Tensor& x) {
    need(t.sizes() == x.sizes() && t.scalar_type() == x.scalar_type(), std::string(name) + " must match the rows in shape and dtype");
}
gdn_norm_problem norm_problem(const at::Tensor& x, const at::Tensor& w, double eps, double offset) {
    need(x.dim() >= 1 && x.size(-1) > 0, "rows must be [..., dim]");
    gdn_norm_problem p{};
    p.dim = small(x.size(-1), "values to a row");
    need(w.dim() == 1 && w.size(0) == p.dim && w.is_contiguous(), "weight must be a contiguous [dim]");
    p.rows = x.numel() / p.dim;
    p.dtype = p.out_dtype = code(x, "the rows");
    p.weight_dtype = code(w, "weight");
    p.eps = float(eps);
    p.weight_offset = float(offset);
    return p;
}
PyObject* tuple_of(const at::Tensor& a, const at::Tensor* b, const at::Tensor* c) {
    PyObject* none = Py_None;
    PyObject* r = PyTuple_New(3);
    if (!r) throw Bad{nullptr, ""};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
    const at::Tensor* rest[2] = {b, c};
    for (int i = 0; i < 2; ++i) {
        if (!rest[i]) Py_INCREF(none);
        PyTuple_SET_ITEM(r, i + 1, rest[i] ? THPVariable_Wrap(*rest[i]) : none);
    }
    return r;
}

PyObject* norm_fwd(Args& a) {
    const at::Tensor &x = a.tensor("x"), &w = a.tensor("weight");
    const at::Tensor* res = a.maybe("residual");
    const double eps = a.number(), offset = a.number();
    const bool quant = a.flag();
    const int64_t group = a.integer();
    const bool want_sum = a.flag();
    gdn_norm_problem p = norm_problem(x, w, eps, offset);
    p.x_stride = row_stride("x", x);
    if (res) {
        like_rows("residual", *res, x);
        p.residual_stride = row_stride("residual", *res);
    }
    need_cuda(x, "x", x);
    need_cuda(x, "weight", w);
    need_cuda(x, "residual", res);
    On on(x, a);
    at::Tensor total, scale;
    if (res && want_sum) total = empty(x.sizes(), x.scalar_type(), x);
    if (quant) {
        need(group >= 0 && (group == 0 || p.dim % group == 0), "group must be 0 or divide dim");
        p.out_dtype = GDN_E4M3;
        p.group = int32_t(group);
        c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
        shape.back() = group ? p.dim / group : 1;
        scale = empty(shape, at::kFloat, x);
    }
    const at::Tensor y = empty(x.sizes(), quant ? at::kFloat8_e4m3fn : x.scalar_type(), x);
    check(f_norm_fwd(&p, x.data_ptr(), ptr<void>(res), w.data_ptr(), y.data_ptr(), quant ? ptr(scale) : nullptr, total.defined() ? total.data_ptr() : nullptr, on.stream));
    return tuple_of(y, quant ? &scale : nullptr, total.defined() ? &total : nullptr);
}

PyObject* norm_bwd(Args& a) {
    const at::Tensor &s = a.tensor("s"), &w = a.tensor("weight"), &dy = a.tensor("dy");
    const at::Tensor* dsum = a.maybe("dsum");
    const double eps = a.number(), offset = a.number();
    const at::Tensor* ws = a.maybe("workspace");
    gdn_norm_problem p = norm_problem(s, w, eps, offset);
    p.x_stride = row_stride("s", s);
    like_rows("dy", dy, s);
    p.dy_stride = row_stride("dy", dy);
    if (dsum) {
        like_rows("dsum", *dsum, s);
        p.dsum_stride = row_stride("dsum", *dsum);
    }
    need_scratch(ws);
    need_cuda(s, "s", s);
    need_cuda(s, "weight", w);
    need_cuda(s, "dy", dy);
    need_cuda(s, "dsum", dsum);
    need_cuda(s, "workspace", ws);
    On on(s, a);
    size_t bytes = 0;
    check(f_norm_bwd_size(&p, &bytes));
    const at::Tensor work = scratch(bytes, ws, s), dx = empty(s.sizes(), s.scalar_type(), s), dw = empty({p.dim}, at::kFloat, s);
    check(f_norm_bwd(&p, s.data_ptr(), w.data_ptr(), dy.data_ptr(), ptr<void>(dsum), dx.data_ptr(), ptr(dw), work.data_ptr(),
                     size_t(work.numel()) * work.element_size(), on.stream));
    PyObject* r = PyTuple_New(2);
    if (!r) throw Bad{nullptr, ""};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(dx));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(dw));
    return r;
}

// True when gradients are on and one of the arguments (tensors or None) requires one.  A forward-mode tangent
// (level 0 is the only level there is) would be dropped, whether gradients are on or not: refused.
PyObject* wants_grad(Args& a) {
    const bool on = c10::GradMode::is_enabled(), forward = torch::autograd::ForwardADLevel::try_get_by_idx(0) != nullptr;
    if (!on && !forward) Py_RETURN_FALSE;
    bool wants = false;
    while (a.at < a.n) {
        const at::Tensor* t = a.maybe("argument");
        if (!t) continue;
        if (forward && t->_fw_grad(0).defined()) throw Bad{PyExc_RuntimeError, "forward-mode differentiation is not implemented here, but an argument carries a tangent"};
        wants |= on && t->requires_grad();
    }
    if (wants) Py_RETURN_TRUE;
    Py_RETURN_FALSE;
}

PyObject* bind(Args& a) {
    void* at[6];
    for (void*& p : at) {
        p = PyLong_AsVoidPtr(a.next());
        if (!p) throw Bad{PyExc_ValueError, "a function's address is missing"};
    }
    f_step = reinterpret_cast<decltype(f_step)>(at[0]);
    f_paged_size = reinterpret_cast<decltype(f_paged_size)>(at[1]);
    f_paged = reinterpret_cast<decltype(f_paged)>(at[2]);
    f_norm_fwd = reinterpret_cast<decltype(f_norm_fwd)>(at[3]);
    f_norm_bwd_size = reinterpret_cast<decltype(f_norm_bwd_size)>(at[4]);
    f_norm_bwd = reinterpret_cast<decltype(f_norm_bwd)>(at[5]);
    PyObject* f = a.next();
    Py_INCREF(f);
    Py_XDECREF(on_error);
    on_error = f;
    Py_RETURN_NONE;
}

template <PyObject* (*F)(Args&)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        if (!on_error && F != &bind) throw Bad{PyExc_RuntimeError, "the library is not bound"};
        Args a{args, n};
        return F(a);
    } catch (const Bad& b) {
        if (b.type) PyErr_SetString(b.type, b.msg.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<&name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(step), METHOD(paged), METHOD(norm_fwd), METHOD(norm_bwd), METHOD(wants_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
