// C ABI of attention over prompts, of drafted trees over a paged cache, and of the cache's own operators:
// argument checks, defaults of the strides and the launches.  Nothing here allocates, frees or synchronises, but
// that gdn_attn_device_status waits for its stream and copies from the device.
#include "gdn_attn.h"
#include "gdn_checks.h"
#include "gdn_internal.h"

namespace {

gdn_status check_heads(int Hq, int Hkv, int D) {
    if (Hq <= 0 || Hkv <= 0) return fail(GDN_ERR_INVALID_ARG, "Hq and Hkv must be positive");
    if (Hq % Hkv) return fail(GDN_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
    if (D <= 0) return fail(GDN_ERR_INVALID_ARG, "D must be positive");
    if (D != 64 && D != 128 && D != 256) return fail(GDN_ERR_UNSUPPORTED, "only D = 64, 128, 256 are implemented (got %d)", D);
    if (Hq > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 query heads");
    return GDN_OK;
}
gdn_status check_types(int dtype, int cache) {
    const bool ok = dtype == GDN_BF16 ? (cache == GDN_BF16 || cache == GDN_E4M3) : (dtype == GDN_FP32 && cache == GDN_FP32);
    if (!ok) return fail(GDN_ERR_INVALID_ARG, "dtype, cache_dtype must be bf16 with bf16 or e4m3, or fp32 with fp32");
    return GDN_OK;
}
gdn_status check_cache_strides(int64_t unit, int64_t a, int64_t b, int64_t c, int64_t d, int64_t e, int64_t f) {
    for (int64_t s : {a, b, c, d, e, f})
        if (s < 0 || s % unit) return fail(GDN_ERR_INVALID_ARG, "cache strides must be >= 0 and multiples of %lld elements (16 bytes), got %lld", (long long)unit, (long long)s);
    return GDN_OK;
}

// Whether a page, token or head of the caches stands for several.
template <typename P> bool no_stride(const P& p) {
    return (p.num_pages > 1 && !(p.k_page_stride && p.v_page_stride)) || (p.page_size > 1 && !(p.k_token_stride && p.v_token_stride)) || (p.Hkv > 1 && !(p.k_head_stride && p.v_head_stride));
}

gdn_status check_prompt(gdn_prompt_problem& p) {
    TRY(check_heads(p.Hq, p.Hkv, p.D));
    if (p.dtype != GDN_BF16 && p.dtype != GDN_FP32) return fail(GDN_ERR_INVALID_ARG, "dtype must be GDN_BF16 or GDN_FP32");
    TRY(check_scale(p.scale));
    if (p.num_seqs < 0 || p.total_q < 0 || p.total_k < 0 || p.window < 0)
        return fail(GDN_ERR_INVALID_ARG, "num_seqs, total_q, total_k and window must be >= 0");
    if (p.num_seqs > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 sequences in one call");
    if (p.total_q > 0x7fff0000 || p.total_k > 0x7fff0000) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 2^16 rows");
    if (!p.cu_seqlens) {
        if (p.cu_seqlens_k) return fail(GDN_ERR_INVALID_ARG, "cu_seqlens_k without cu_seqlens");
        if (p.num_seqs > 0 ? p.total_q % p.num_seqs || p.total_k % p.num_seqs : p.total_q || p.total_k)
            return fail(GDN_ERR_INVALID_ARG, "without cu_seqlens total_q (%d) and total_k (%d) must be multiples of num_seqs (%d)", p.total_q, p.total_k, p.num_seqs);
    } else if (!p.cu_seqlens_k && p.total_k != p.total_q) {
        return fail(GDN_ERR_INVALID_ARG, "total_k (%d) must be total_q (%d) without cu_seqlens_k", p.total_k, p.total_q);
    }
    if (int64_t(p.total_q) * p.Hq > (int64_t(1) << 33)) return fail(GDN_ERR_UNSUPPORTED, "more than 2^33 (row, query head) pairs");
    const int64_t unit = 16 / int64_t(elem(p.dtype));
    TRY(check_stride("q_stride", p.q_stride, int64_t(p.Hq) * p.D, unit));
    TRY(check_stride("k_stride", p.k_stride, int64_t(p.Hkv) * p.D, unit));
    TRY(check_stride("v_stride", p.v_stride, int64_t(p.Hkv) * p.D, unit));
    for (int64_t s : {p.q_stride, p.k_stride, p.v_stride})
        if (s >= (int64_t(1) << 37)) return fail(GDN_ERR_UNSUPPORTED, "token strides of 2^37 elements or more");
    TRY(check_ptr("cu_seqlens", p.cu_seqlens, 4, true));
    TRY(check_ptr("cu_seqlens_k", p.cu_seqlens_k, 4, true));
    return GDN_OK;
}

gdn_status check_tree(gdn_tree_problem& p) {
    TRY(check_heads(p.Hq, p.Hkv, p.D));
    TRY(check_types(p.dtype, p.cache_dtype));
    TRY(check_scale(p.scale));
    if (p.num_seqs < 0 || p.max_pages < 0 || p.num_pages < 0 || p.window < 0)
        return fail(GDN_ERR_INVALID_ARG, "num_seqs, max_pages, num_pages and window must be >= 0");
    if (p.T < 1) return fail(GDN_ERR_INVALID_ARG, "T must be positive (got %d)", p.T);
    if (p.T > 64) return fail(GDN_ERR_UNSUPPORTED, "more than 64 drafted tokens (got %d)", p.T);
    if (p.page_size <= 0) return fail(GDN_ERR_INVALID_ARG, "page_size must be positive");
    if (int64_t(p.max_pages) * p.page_size > 0x7ffe0000) return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_size above 2^31 tokens");
    if (p.num_seqs > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 sequences in one call");
    if (p.num_pages > 0x7ffffffe) return fail(GDN_ERR_UNSUPPORTED, "2^31 - 1 pages or more");
    const int64_t act = 16 / int64_t(elem(p.dtype));
    TRY(check_stride("q_stride", p.q_stride, int64_t(p.Hq) * p.D, act));
    TRY(check_stride("k_new_stride", p.k_new_stride, int64_t(p.Hkv) * p.D, act));
    TRY(check_stride("v_new_stride", p.v_new_stride, int64_t(p.Hkv) * p.D, act));
    TRY(check_stride("table_stride", p.table_stride, p.max_pages, 1));
    TRY(check_cache_strides(16 / int64_t(elem(p.cache_dtype)), p.k_page_stride, p.k_token_stride, p.k_head_stride, p.v_page_stride, p.v_token_stride, p.v_head_stride));
    // the tensor cores' kernels read pages through tensor maps, whose strides are not to be 0
    if (p.dtype == GDN_BF16 && no_stride(p)) return fail(GDN_ERR_INVALID_ARG, "a bf16 or 8-bit cache must not have strides of 0 (an expanded view)");
    return GDN_OK;
}

gdn_status check_cache(gdn_cache_problem& p) {
    if (p.count < 0 || p.num_rows < 0 || p.num_pages < 0) return fail(GDN_ERR_INVALID_ARG, "count, num_rows and num_pages must be >= 0");
    if (p.count > 0x7fffffff) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 1 rows in one call");
    if (p.Hkv <= 0 || p.D <= 0) return fail(GDN_ERR_INVALID_ARG, "Hkv and D must be positive");
    if (p.D % 16) return fail(GDN_ERR_UNSUPPORTED, "D (%d) must be a multiple of 16", p.D);
    if (int64_t(p.Hkv) * p.D > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "rows of more than 2^20 values");
    TRY(check_types(p.dtype, p.cache_dtype));
    if (p.page_size <= 0) return fail(GDN_ERR_INVALID_ARG, "page_size must be positive");
    const int64_t act = 16 / int64_t(elem(p.dtype));
    TRY(check_stride("k_stride", p.k_stride, int64_t(p.Hkv) * p.D, act));
    TRY(check_stride("v_stride", p.v_stride, int64_t(p.Hkv) * p.D, act));
    TRY(check_cache_strides(16 / int64_t(elem(p.cache_dtype)), p.k_page_stride, p.k_token_stride, p.k_head_stride, p.v_page_stride, p.v_token_stride, p.v_head_stride));
    // a head, token or page that stands for several would be written by each
    if (no_stride(p)) return fail(GDN_ERR_INVALID_ARG, "a cache that is written to must not have strides of 0");
    return GDN_OK;
}

gdn_status check_table(gdn_table_problem& p) {
    if (p.num_seqs < 0 || p.max_pages < 0 || p.stack_size < 0 || p.total < 0)
        return fail(GDN_ERR_INVALID_ARG, "num_seqs, max_pages, stack_size and total must be >= 0");
    if (p.page_size <= 0) return fail(GDN_ERR_INVALID_ARG, "page_size must be positive");
    if (p.num_seqs > gdn::TABLE_SEQS) return fail(GDN_ERR_UNSUPPORTED, "more than %d sequences in one call", gdn::TABLE_SEQS);
    if (int64_t(p.max_pages) * p.page_size + p.page_size > 0x7fff0000) return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_size above 2^31 tokens");
    if (p.total > 0x7fffffff) return fail(GDN_ERR_UNSUPPORTED, "more than 2^31 - 1 new tokens");
    return check_stride("table_stride", p.table_stride, p.max_pages, 1);
}
gdn_status check_table_ptrs(const gdn::TableArgs& A, const char* change) {
    const bool none = A.p.num_seqs == 0;
    TRY(check_ptr("page_table", A.table, 4, none || A.p.max_pages == 0));
    TRY(check_ptr("seq_lens", A.lens, 4, none));
    TRY(check_ptr(change, A.change, 4, none));
    TRY(check_ptr("free_pages", A.stack, 4, A.p.stack_size == 0));
    return check_ptr("num_free", A.free, 4);
}

gdn_status prompt_ptrs(const gdn_prompt_problem& p, const void* q, const void* k, const void* v) {
    TRY(check_ptr("q", q, 16, p.total_q == 0));
    TRY(check_ptr("k", k, 16, p.total_k == 0));
    return check_ptr("v", v, 16, p.total_k == 0);
}

}  // namespace

extern "C" {

gdn_status gdn_prompt_attn_fwd(const gdn_prompt_problem* problem, const void* q, const void* k, const void* v,
                               void* o, float* lse, void* o_rest, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::PromptArgs A{};
    A.p = *problem;
    TRY(check_prompt(A.p));
    TRY(prompt_ptrs(A.p, q, k, v));
    TRY(check_ptr("o", o, 16, A.p.total_q == 0));
    TRY(check_ptr("lse", lse, 4, true));
    TRY(check_ptr("o_rest", o_rest, 16, true));
    if (o_rest && A.p.dtype != GDN_BF16) return fail(GDN_ERR_INVALID_ARG, "o_rest is of bf16 outputs alone");
    if (A.p.total_q == 0) return done(cudaSuccess);
    A.q = q;
    A.k = k;
    A.v = v;
    A.o = o;
    A.lse = lse;
    A.o_rest = o_rest;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return done(A.p.dtype == GDN_FP32 ? gdn::launch_prompt_fwd_simt(A, st) : gdn::launch_prompt_fwd_tc(A, st));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_prompt_attn_bwd_workspace_size(const gdn_prompt_problem* problem, size_t* bytes) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
    gdn_prompt_problem p = *problem;
    TRY(check_prompt(p));
    *bytes = gdn::prompt_bwd_workspace(p);
    return done(cudaSuccess);
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_prompt_attn_bwd(const gdn_prompt_problem* problem, const void* q, const void* k, const void* v,
                               const void* o, const float* lse, const void* o_rest, const void* dO,
                               const float* dlse, void* dq, void* dk, void* dv, void* workspace,
                               size_t workspace_bytes, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::PromptArgs A{};
    A.p = *problem;
    TRY(check_prompt(A.p));
    const bool no_q = A.p.total_q == 0, no_k = A.p.total_k == 0;
    TRY(prompt_ptrs(A.p, q, k, v));
    TRY(check_ptr("o", o, 16, no_q));
    TRY(check_ptr("lse", lse, 4, no_q));
    TRY(check_ptr("o_rest", o_rest, 16, true));
    if (o_rest && A.p.dtype != GDN_BF16) return fail(GDN_ERR_INVALID_ARG, "o_rest is of bf16 outputs alone");
    TRY(check_ptr("dO", dO, 16, no_q));
    TRY(check_ptr("dlse", dlse, 4, true));
    TRY(check_ptr("dq", dq, 16, no_q));
    TRY(check_ptr("dk", dk, 16, no_k));
    TRY(check_ptr("dv", dv, 16, no_k));
    const size_t need = gdn::prompt_bwd_workspace(A.p);
    if (need && (!workspace || workspace_bytes < need))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : size_t(0));
    if (need) TRY(check_ptr("workspace", workspace, 16));
    if (no_q && no_k) return done(cudaSuccess);
    A.q = q;
    A.k = k;
    A.v = v;
    A.o_in = o;
    A.rest_in = o_rest;
    A.lse_in = lse;
    A.dO = dO;
    A.dlse = dlse;
    A.dq = dq;
    A.dk = dk;
    A.dv = dv;
    A.stat_rows = (int64_t(A.p.total_q) + 127) / 128 * 128;
    A.stat = static_cast<float2*>(workspace);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = gdn::launch_prompt_stat(A, st);
    if (e != cudaSuccess) return done(e);
    return done(A.p.dtype == GDN_FP32 ? gdn::launch_prompt_bwd_simt(A, st) : gdn::launch_prompt_bwd_tc(A, st));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_attn_device_status(void* stream) try {
    const cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return done(e);
    const int fwd = gdn::prompt_fwd_status(), bwd = gdn::prompt_bwd_status(), t16 = gdn::tree_status_bf16(), t8 = gdn::tree_status_f8();
    if (fwd < 0 || bwd < 0 || t16 < 0 || t8 < 0) return done(cudaGetLastError());
    if (fwd || bwd || t16 || t8)
        return fail(GDN_ERR_TIMEOUT, "a device-side wait gave up (prompt%s%s, tree%s%s)", fwd ? " forward" : "", bwd ? " backward" : "", t16 ? " bf16" : "", t8 ? " 8 bits" : "");
    return done(cudaSuccess);
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_debug_attn_wait_timeout(int32_t kernels, int32_t limit_us, void* stream) try {
    if (kernels < 0 || kernels > 3) return fail(GDN_ERR_INVALID_ARG, "kernels must be in [0, 3]");
    if (limit_us < 1 || limit_us > 1000000) return fail(GDN_ERR_INVALID_ARG, "limit_us must be in [1, 1000000]");
    const auto wait_out = kernels == 0 ? gdn::prompt_fwd_wait_out : kernels == 1 ? gdn::prompt_bwd_wait_out : kernels == 2 ? gdn::tree_wait_out_bf16 : gdn::tree_wait_out_f8;
    return done(wait_out(limit_us, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_paged_attn_tree_workspace_size(const gdn_tree_problem* problem, size_t* bytes) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
    gdn_tree_problem p = *problem;
    TRY(check_tree(p));
    *bytes = p.num_seqs > 0 ? gdn::tree_plan(p).bytes : 0;
    return done(cudaSuccess);
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_paged_attn_tree(const gdn_tree_problem* problem, const void* q, const void* k_new, const void* v_new,
                               const void* k_cache, const void* v_cache, const int32_t* page_table,
                               const int32_t* seq_lens, const int32_t* parents, const float* k_scale,
                               const float* v_scale, void* o, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::TreeArgs A{};
    A.p = *problem;
    gdn_tree_problem& p = A.p;
    TRY(check_tree(p));
    if (p.num_seqs == 0) return done(cudaSuccess);
    const bool none = p.max_pages == 0 || p.num_pages == 0;  // every length is then 0
    TRY(check_ptr("q", q, 16));
    TRY(check_ptr("k_new", k_new, 16));
    TRY(check_ptr("v_new", v_new, 16));
    TRY(check_ptr("k_cache", k_cache, 16, none));
    TRY(check_ptr("v_cache", v_cache, 16, none));
    TRY(check_ptr("page_table", page_table, 4, p.max_pages == 0));
    TRY(check_ptr("seq_lens", seq_lens, 4));
    TRY(check_ptr("parents", parents, 4));
    TRY(check_ptr("k_scale", k_scale, 4, true));
    TRY(check_ptr("v_scale", v_scale, 4, true));
    TRY(check_ptr("o", o, 16));
    TRY(check_ptr("lse", lse, 4, true));
    const gdn::TreePlan plan = gdn::tree_plan(p);
    if (plan.bytes && (!workspace || workspace_bytes < plan.bytes))
        return fail(GDN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", plan.bytes, workspace ? workspace_bytes : size_t(0));
    if (plan.bytes) TRY(check_ptr("workspace", workspace, 16));
    A.page_div.set(uint32_t(p.page_size));
    A.q = q;
    A.k_new = k_new;
    A.v_new = v_new;
    A.k_cache = k_cache;
    A.v_cache = v_cache;
    A.table = page_table;
    A.lens = seq_lens;
    A.parents = parents;
    A.k_scale = k_scale;
    A.v_scale = v_scale;
    A.o = o;
    A.lse = lse;
    char* ws = static_cast<char*>(workspace);
    A.groups = plan.groups;
    A.heads = plan.heads;
    A.before = reinterpret_cast<int64_t*>(ws);
    A.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
    A.part = reinterpret_cast<float*>(ws + plan.off_part);
    return done(gdn::launch_tree(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_paged_cache_write(const gdn_cache_problem* problem, const void* k, const void* v, void* k_cache,
                                 void* v_cache, const int64_t* slots, const int32_t* rows, const float* k_scale,
                                 const float* v_scale, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::CacheArgs A{*problem, k, v, k_cache, v_cache, slots, rows, k_scale, v_scale};
    TRY(check_cache(A.p));
    if (A.p.count == 0 || A.p.num_rows == 0 || A.p.num_pages == 0) return done(cudaSuccess);  // nothing has a place
    TRY(check_ptr("k", k, 16));
    TRY(check_ptr("v", v, 16));
    TRY(check_ptr("k_cache", k_cache, 16));
    TRY(check_ptr("v_cache", v_cache, 16));
    TRY(check_ptr("slots", slots, 8));
    TRY(check_ptr("rows", rows, 4, true));
    TRY(check_ptr("k_scale", k_scale, 4, true));
    TRY(check_ptr("v_scale", v_scale, 4, true));
    return done(gdn::launch_cache_write(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_page_table_extend(const gdn_table_problem* problem, int32_t* page_table, int32_t* seq_lens,
                                 const int32_t* new_lens, int32_t* free_pages, int32_t* num_free, int64_t* slots,
                                 int32_t* cu_seqlens, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::TableArgs A{*problem, page_table, seq_lens, new_lens, free_pages, num_free, slots, cu_seqlens};
    TRY(check_table(A.p));
    TRY(check_table_ptrs(A, "new_lens"));
    TRY(check_ptr("slots", slots, 8, A.p.total == 0));
    TRY(check_ptr("cu_seqlens", cu_seqlens, 4));
    return done(gdn::launch_table_extend(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

gdn_status gdn_page_table_trim(const gdn_table_problem* problem, const int32_t* page_table, int32_t* seq_lens,
                               const int32_t* keep_lens, int32_t* free_pages, int32_t* num_free, void* stream) try {
    if (!problem) return fail(GDN_ERR_INVALID_ARG, "problem is NULL");
    gdn::TableArgs A{*problem, const_cast<int32_t*>(page_table), seq_lens, keep_lens, free_pages, num_free, nullptr, nullptr};
    TRY(check_table(A.p));
    TRY(check_table_ptrs(A, "keep_lens"));
    return done(gdn::launch_table_trim(A, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return no_host_memory();
}

}  // extern "C"
