// C ABI of the decoding operators: argument checks, defaults of the strides and the launches.
// Nothing here allocates, frees or synchronises.
#include <atomic>

#include "gdn_checks.h"
#include "gdn_decode.h"
#include "gdn_internal.h"

namespace gdn {
int sm_count_cached() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sm_count();
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        n = sm_count();
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}
}  // namespace gdn

namespace {

gdn_status check_step(gdn_step_problem& p) {
    if (p.K <= 0 || p.V <= 0) return fail(GDN_ERR_INVALID_ARG, "K and V must be positive");
    if (p.K != 128 || p.V != 128) return fail(GDN_ERR_UNSUPPORTED, "only K = V = 128 is implemented (got K=%d V=%d)", p.K, p.V);
    if (p.Hqk <= 0 || p.Hv <= 0) return fail(GDN_ERR_INVALID_ARG, "Hqk and Hv must be positive");
    if (p.Hv % p.Hqk) return fail(GDN_ERR_INVALID_ARG, "Hv (%d) must be a multiple of Hqk (%d)", p.Hv, p.Hqk);
    if (p.dtype != GDN_BF16 && p.dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "dtype must be GDN_BF16 or GDN_FP32");
    TRY(check_scale(p.scale));
    if (p.num_seqs < 0 || p.total_tokens < 0 || p.num_slots < 0)
        return fail(GDN_ERR_INVALID_ARG, "num_seqs, total_tokens and num_slots must be >= 0");
    if (!p.cu_seqlens && p.num_seqs > 0 && p.total_tokens % p.num_seqs)
        return fail(GDN_ERR_INVALID_ARG, "without cu_seqlens total_tokens (%d) must be a multiple of num_seqs (%d)", p.total_tokens, p.num_seqs);
    if (int64_t(p.num_seqs) * p.Hv > (int64_t(1) << 28))
        return fail(GDN_ERR_UNSUPPORTED, "more than 2^28 (sequence, v-head) pairs");
    const int64_t unit = p.dtype == GDN_BF16 ? 8 : 4;
    TRY(check_stride("q_stride", p.q_stride, int64_t(p.Hqk) * p.K, unit));
    TRY(check_stride("k_stride", p.k_stride, int64_t(p.Hqk) * p.K, unit));
    TRY(check_stride("v_stride", p.v_stride, int64_t(p.Hv) * p.V, unit));
    TRY(check_stride("g_stride", p.g_stride, p.Hv, 1));
    TRY(check_stride("beta_stride", p.beta_stride, p.Hv, 1));
    TRY(check_ptr("cu_seqlens", p.cu_seqlens, 4, true));
    TRY(check_ptr("slots", p.slots, 4, true));
    return GDN_OK;
}

gdn_status check_paged(gdn_paged_problem& p) {
    if (p.Hq <= 0 || p.Hkv <= 0) return fail(GDN_ERR_INVALID_ARG, "Hq and Hkv must be positive");
    if (p.Hq % p.Hkv) return fail(GDN_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", p.Hq, p.Hkv);
    if (p.D <= 0) return fail(GDN_ERR_INVALID_ARG, "D must be positive");
    if (p.D != 64 && p.D != 128 && p.D != 256) return fail(GDN_ERR_UNSUPPORTED, "only D = 64, 128, 256 are implemented (got %d)", p.D);
    const bool ok = p.dtype == GDN_BF16 ? (p.cache_dtype == GDN_BF16 || p.cache_dtype == GDN_E4M3)
                                        : (p.dtype == GDN_FP32 && p.cache_dtype == GDN_FP32);
    if (!ok) return fail(GDN_ERR_INVALID_ARG, "dtype, cache_dtype must be bf16 with bf16 or e4m3, or fp32 with fp32");
    TRY(check_scale(p.scale));
    if (p.num_seqs < 0 || p.max_pages < 0 || p.num_pages < 0 || p.window < 0)
        return fail(GDN_ERR_INVALID_ARG, "num_seqs, max_pages, num_pages and window must be >= 0");
    if (p.page_size <= 0) return fail(GDN_ERR_INVALID_ARG, "page_size must be positive");
    if (int64_t(p.max_pages) * p.page_size > 0x7fff0000)
        return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_size above 2^31 tokens");
    if (p.num_seqs > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 sequences in one call");
    if (p.Hq > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 query heads");
    const int64_t act = 16 / int64_t(elem(p.dtype)), unit = 16 / int64_t(elem(p.cache_dtype));
    TRY(check_stride("q_stride", p.q_stride, int64_t(p.Hq) * p.D, act));
    TRY(check_stride("new_stride", p.new_stride, int64_t(p.Hkv) * p.D, act));
    TRY(check_stride("table_stride", p.table_stride, p.max_pages, 1));
    const int64_t strides[6] = {p.k_page_stride, p.k_token_stride, p.k_head_stride, p.v_page_stride, p.v_token_stride, p.v_head_stride};
    for (int64_t s : strides)
        if (s < 0 || s % unit) return fail(GDN_ERR_INVALID_ARG, "cache strides must be >= 0 and multiples of %lld elements (16 bytes), got %lld", (long long)unit, (long long)s);
    return GDN_OK;
}

gdn_status check_norm(gdn_norm_problem& p, bool backward) {
    if (p.rows < 0) return fail(GDN_ERR_INVALID_ARG, "rows must be >= 0");
    if (p.rows > 0x7fffffff) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
    if (p.dim <= 0) return fail(GDN_ERR_INVALID_ARG, "dim must be positive (got %d)", p.dim);
    if (p.dtype != GDN_BF16 && p.dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "dtype must be GDN_BF16 or GDN_FP32");
    if (p.weight_dtype != GDN_BF16 && p.weight_dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "weight_dtype must be GDN_BF16 or GDN_FP32");
    if (!backward && p.out_dtype != p.dtype && p.out_dtype != GDN_E4M3) return fail(GDN_ERR_INVALID_ARG, "out_dtype must be dtype or GDN_E4M3");
    if (!isfinite(p.eps) || p.eps < 0.f) return fail(GDN_ERR_INVALID_ARG, "eps must be finite and >= 0 (got %g)", double(p.eps));
    if (!isfinite(p.weight_offset)) return fail(GDN_ERR_INVALID_ARG, "weight_offset must be finite");
    if (p.group < 0 || (p.group > 0 && p.dim % p.group)) return fail(GDN_ERR_INVALID_ARG, "group (%d) must be 0 or divide dim (%d)", p.group, p.dim);
    TRY(check_stride("x_stride", p.x_stride, p.dim, 1));
    TRY(check_stride("residual_stride", p.residual_stride, p.dim, 1));
    TRY(check_stride("dy_stride", p.dy_stride, p.dim, 1));
    TRY(check_stride("dsum_stride", p.dsum_stride, p.dim, 1));
    for (int64_t s : {p.x_stride, p.residual_stride, p.dy_stride, p.dsum_stride})
        if (s > 0x7fffffff) return fail(GDN_ERR_UNSUPPORTED, "row strides of more than 2^31 - 1 values");
    return GDN_OK;
}

// An output may lie in an input's place where its rows do: contiguous, and of the same type.
gdn_status check_in_place(const gdn_norm_problem& p, const char* out, const void* o, int out_dtype, const char* in, const void* i, int64_t stride) {
    if (!o || o != i || p.rows == 0) return GDN_OK;
    if (out_dtype != p.dtype) return fail(GDN_ERR_INVALID_ARG, "%s may be %s only in the same type", out, in);
    if (p.rows > 1 && stride != p.dim) return fail(GDN_ERR_INVALID_ARG, "%s may be %s only where its rows are contiguous", out, in);
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_recurrent_step(const gdn_step_problem* problem, const void* q, const void* k,
                              const void* v, const float* g, const float* beta, const float* A_log,
                              const float* dt_bias, const float* state_in, float* state_out,
                              void* o, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::StepArgs A{*problem, q, k, v, g, beta, A_log, dt_bias, state_in, state_out, o, 0};
    gdn_step_problem& p = A.p;
    TRY(check_step(p));
    const bool none = p.total_tokens == 0;
    TRY(check_ptr("q", q, 16, none));
    TRY(check_ptr("k", k, 16, none));
    TRY(check_ptr("v", v, 16, none));
    TRY(check_ptr("o", o, 16, none));
    TRY(check_ptr("g", g, 4, none));
    TRY(check_ptr("beta", beta, 4, none));
    TRY(check_ptr("state_in", state_in, 16, true));
    TRY(check_ptr("state_out", state_out, 16, true));
    TRY(check_ptr("A_log", A_log, 4, true));
    TRY(check_ptr("dt_bias", dt_bias, 4, true));
    if ((A_log == nullptr) != (dt_bias == nullptr)) return fail(GDN_ERR_INVALID_ARG, "A_log and dt_bias go together");
    if (p.num_seqs == 0) {
        const size_t bytes = size_t(p.total_tokens) * p.Hv * p.V * elem(p.dtype);
        return done(p.clear_rest && bytes ? cudaMemsetAsync(o, 0, bytes, static_cast<cudaStream_t>(stream)) : cudaSuccess);
    }
    return done(gdn::launch_step(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_paged_attn_workspace_size(const gdn_paged_problem* problem, size_t* bytes) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
    gdn_paged_problem p = *problem;
    TRY(check_paged(p));
    *bytes = p.num_seqs > 0 ? gdn::paged_plan(p).bytes : 0;
    return done(cudaSuccess);
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_paged_attn_decode(const gdn_paged_problem* problem, const void* q, void* k_cache,
                                 void* v_cache, const int32_t* page_table, const int32_t* seq_lens,
                                 const void* k_new, const void* v_new, const float* k_scale,
                                 const float* v_scale, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::PagedArgs A{};
    A.p = *problem;
    gdn_paged_problem& p = A.p;
    TRY(check_paged(p));
    if (p.num_seqs == 0) return done(cudaSuccess);
    const bool none = p.max_pages == 0 || p.num_pages == 0;  // every length is then 0
    TRY(check_ptr("q", q, 16));
    TRY(check_ptr("o", o, 16));
    TRY(check_ptr("k_cache", k_cache, 16, none));
    TRY(check_ptr("v_cache", v_cache, 16, none));
    TRY(check_ptr("page_table", page_table, 4, p.max_pages == 0));
    TRY(check_ptr("seq_lens", seq_lens, 4));
    TRY(check_ptr("k_new", k_new, 16, true));
    TRY(check_ptr("v_new", v_new, 16, true));
    TRY(check_ptr("k_scale", k_scale, 4, true));
    TRY(check_ptr("v_scale", v_scale, 4, true));
    TRY(check_ptr("lse", lse, 4, true));
    if ((k_new == nullptr) != (v_new == nullptr)) return fail(GDN_ERR_INVALID_ARG, "k_new and v_new go together");
    const gdn::PagedPlan plan = gdn::paged_plan(p);
    if (plan.bytes && (!workspace || workspace_bytes < plan.bytes))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", plan.bytes, workspace ? workspace_bytes : size_t(0));
    if (plan.bytes) TRY(check_ptr("workspace", workspace, 16));
    A.page_div.set(uint32_t(p.page_size));
    A.q = q;
    A.k_cache = k_cache;
    A.v_cache = v_cache;
    A.table = page_table;
    A.lens = seq_lens;
    A.k_new = k_new;
    A.v_new = v_new;
    A.k_scale = k_scale;
    A.v_scale = v_scale;
    A.o = o;
    A.lse = lse;
    char* ws = static_cast<char*>(workspace);
    A.cluster = plan.cluster;
    A.groups = plan.groups;
    A.heads = plan.heads;
    A.before = reinterpret_cast<int64_t*>(ws);
    A.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
    A.part = reinterpret_cast<float*>(ws + plan.off_part);
    return done(gdn::launch_paged(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_rmsnorm_fwd(const gdn_norm_problem* problem, const void* x, const void* residual,
                           const void* weight, void* y, float* y_scale, void* sum, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::NormArgs A{};
    A.p = *problem;
    gdn_norm_problem& p = A.p;
    TRY(check_norm(p, false));
    const size_t e = elem(p.dtype);
    const bool none = p.rows == 0;
    TRY(check_ptr("x", x, e, none));
    TRY(check_ptr("residual", residual, e, true));
    TRY(check_ptr("weight", weight, elem(p.weight_dtype)));
    TRY(check_ptr("y", y, elem(p.out_dtype), none));
    TRY(check_ptr("y_scale", y_scale, 4, none || p.out_dtype != GDN_E4M3));
    TRY(check_ptr("sum", sum, e, true));
    TRY(check_in_place(p, "sum", sum, p.dtype, "x", x, p.x_stride));
    TRY(check_in_place(p, "sum", sum, p.dtype, "residual", residual, p.residual_stride));
    TRY(check_in_place(p, "y", y, p.out_dtype, "x", x, p.x_stride));
    TRY(check_in_place(p, "y", y, p.out_dtype, "residual", residual, p.residual_stride));
    if (none) return done(cudaSuccess);
    A.inv_dim = 1.f / float(p.dim);
    A.x = x;
    A.residual = residual;
    A.weight = weight;
    A.y = y;
    A.y_scale = y_scale;
    A.sum = sum;
    return done(gdn::launch_norm_fwd(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_rmsnorm_bwd_workspace_size(const gdn_norm_problem* problem, size_t* bytes) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
    gdn_norm_problem p = *problem;
    TRY(check_norm(p, true));
    *bytes = size_t(gdn::norm_bwd_parts(p)) * p.dim * sizeof(float);
    return done(cudaSuccess);
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_rmsnorm_bwd(const gdn_norm_problem* problem, const void* s, const void* weight,
                           const void* dy, const void* dsum, void* dx, float* dweight,
                           void* workspace, size_t workspace_bytes, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::NormArgs A{};
    A.p = *problem;
    gdn_norm_problem& p = A.p;
    TRY(check_norm(p, true));
    const size_t e = elem(p.dtype);
    const bool none = p.rows == 0;
    TRY(check_ptr("s", s, e, none));
    TRY(check_ptr("weight", weight, elem(p.weight_dtype)));
    TRY(check_ptr("dy", dy, e, none));
    TRY(check_ptr("dsum", dsum, e, true));
    TRY(check_ptr("dx", dx, e, none));
    TRY(check_ptr("dweight", dweight, 4));
    TRY(check_in_place(p, "dx", dx, p.dtype, "s", s, p.x_stride));
    TRY(check_in_place(p, "dx", dx, p.dtype, "dy", dy, p.dy_stride));
    TRY(check_in_place(p, "dx", dx, p.dtype, "dsum", dsum, p.dsum_stride));
    const size_t need = size_t(gdn::norm_bwd_parts(p)) * p.dim * sizeof(float);
    if (!workspace || workspace_bytes < need)
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : size_t(0));
    TRY(check_ptr("workspace", workspace, 16));
    A.inv_dim = 1.f / float(p.dim);
    A.x = s;
    A.weight = weight;
    A.dy = dy;
    A.dsum = dsum;
    A.dx = dx;
    A.dweight = dweight;
    A.part = static_cast<float*>(workspace);
    return done(gdn::launch_norm_bwd(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

}  // extern "C"
