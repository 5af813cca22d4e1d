// A paged key-value cache's own operators (include/gdn.h): keys and values written to slots, and the page
// tables kept on the device from the requests' lengths.
//
// gdn_paged_cache_write moves every value once: bound by HBM for a prompt, by the launch for a few tokens.
// Up to 32 lanes have a token, whose slot and row they look up once, and two 16-byte pieces of the output each.
// 32767 tokens of 8 heads of 128 from bf16 into 8 bits: 44 us, 4.6 TB/s; the conversion's instructions beside the
// bytes.  96 accepted tokens: 5 us a call.
//
// gdn_page_table_extend and _trim are latency: one launch, in which every CTA sums the requests' needs for
// itself (a scan over up to 8 requests a thread) and keeps the sums in shared memory, so that the tokens and
// pages can be dealt out evenly, each finding its request by bisection.  Only lengths and the count of free
// pages are both read and written: a cluster barrier lies between (8 CTAs from 4096 tokens on, one below), or, from
// 32768 tokens on, where slots are the most of it, another launch, which writes them when the first's CTAs have all ended.
#include "gdn_attn.h"
#include "gdn_paged.cuh"

namespace gdn {
namespace {

// ---- writing the cache
// Pieces to a thread: more hold registers, fewer look slots up again (32767 tokens of 8 heads of 128 into 8 bits, 128 threads: 1 49 us,
// 2 46, 3 49, 4 47, 8 68; 256 threads, 4 51).
constexpr int WT = 128, WU = 2;

struct WriteShape {
    int lanes;          // of a token
    int pieces, half;   // of a token; of its keys
    FastDiv by_row, by_page;
};

// x / s to the nearest: the quotient's estimate x r with r = 1 / s to the nearest, corrected by its exact remainder (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990); for s within 2^+-60, where nothing of a quotient
// that counts in 8 bits (2^-10 to 448) over- or underflows on the way.  A quotient past that range stays past it, infinite or not.
__device__ __forceinline__ float quotient_by(float x, float s, float r) {
    const float q = x * r, y = fmaf(fmaf(-q, s, x), r, q);
    return fabsf(q) < 1e30f ? y : q;
}

// A: the rows' type, C: the cache's.  PV values make 16 bytes of the cache.
template <typename A, typename C>
__global__ void __launch_bounds__(WT) k_cache_write(const CacheArgs G, const WriteShape S) {
    constexpr int PV = 16 / int(sizeof(C)), LV = PV * int(sizeof(A)) / 16;  // 16-byte loads of a piece
    const gdn_cache_problem& p = G.p;
    const int per = WT / S.lanes, lane = threadIdx.x & (S.lanes - 1);
    const int64_t n = int64_t(blockIdx.x) * per + threadIdx.x / S.lanes;
    if (n >= p.count) return;
    const int64_t row = G.rows ? G.rows[n] : n, slot = G.slots[n];
    if (slot < 0 || slot >= p.num_pages * p.page_size || row < 0 || row >= p.num_rows) return;
    const int64_t page = slot >> 31 ? slot / p.page_size : S.by_page.of(int(slot)), in = slot - page * p.page_size;
    {
        const A *k = static_cast<const A*>(G.k) + row * p.k_stride, *v = static_cast<const A*>(G.v) + row * p.v_stride;
        C *kc = static_cast<C*>(G.k_cache) + page * p.k_page_stride + in * p.k_token_stride, *vc = static_cast<C*>(G.v_cache) + page * p.v_page_stride + in * p.v_token_stride;
        uint4 raw[WU][LV];
        C* to[WU];
        float scale[WU];
#pragma unroll
        for (int u = 0; u < WU; ++u) {
            const int r = (int(blockIdx.y) * WU + u) * S.lanes + lane;
            to[u] = nullptr;
            scale[u] = 1.f;
            if (r >= S.pieces) continue;
            const bool second = r >= S.half;
            const int at = second ? r - S.half : r, head = S.by_row.of(at), d = (at - head * (p.D / PV)) * PV;
            const A* from = (second ? v : k) + head * p.D + d;
            to[u] = (second ? vc + head * p.v_head_stride : kc + head * p.k_head_stride) + d;
            const float* s = second ? G.v_scale : G.k_scale;
            if (s) scale[u] = s[head];
#pragma unroll
            for (int l = 0; l < LV; ++l) raw[u][l] = reinterpret_cast<const uint4*>(from)[l];
        }
#pragma unroll
        for (int u = 0; u < WU; ++u) {
            if (!to[u]) continue;
            alignas(16) C out[PV];
            // with divisions 32767 tokens of 8 heads of 128 took 70 us instead of 49
            const bool quick = sizeof(C) == 1 && scale[u] >= 8.673617e-19f && scale[u] <= 1.1529215e18f;
            const float r = 1.f / scale[u];
#pragma unroll
            for (int l = 0; l < LV; ++l) {
                const A* x = reinterpret_cast<const A*>(&raw[u][l]);
#pragma unroll
                for (int e = 0; e < PV / LV; e += 2) {
                    const float a = to_f(x[e]), b = to_f(x[e + 1]);
                    if constexpr (sizeof(C) == 1) {
                        const float2 y = quick ? make_float2(quotient_by(a, scale[u], r), quotient_by(b, scale[u], r)) : make_float2(a / scale[u], b / scale[u]);
                        // saturating at 448, NaN kept
                        *reinterpret_cast<__nv_fp8x2_storage_t*>(&out[l * (PV / LV) + e]) = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                    } else {
                        out[l * (PV / LV) + e] = to_cache<C>(a, scale[u]);
                        out[l * (PV / LV) + e + 1] = to_cache<C>(b, scale[u]);
                    }
                }
            }
            *reinterpret_cast<uint4*>(to[u]) = *reinterpret_cast<const uint4*>(out);
        }
    }
}

template <typename A, typename C>
cudaError_t write_as(const CacheArgs& G, cudaStream_t st) {
    constexpr int PV = 16 / int(sizeof(C));
    WriteShape S;
    S.half = G.p.Hkv * (G.p.D / PV);
    S.pieces = 2 * S.half;
    S.lanes = 32;
    while (S.lanes > 2 && S.lanes / 2 >= S.pieces) S.lanes /= 2;
    S.by_row.set(uint32_t(G.p.D / PV));
    S.by_page.set(uint32_t(G.p.page_size));
    const int per = WT / S.lanes;
    const dim3 grid(unsigned((G.p.count + per - 1) / per), unsigned((S.pieces + WU * S.lanes - 1) / (WU * S.lanes)));
    timing_begin("paged_cache_write", st);
    k_cache_write<A, C><<<grid, WT, 0, st>>>(G, S);
    timing_end(st);
    return cudaGetLastError();
}

// ---- page tables
constexpr int TT_ = 1024;

// What a CTA keeps of a request: extend: its first new token, its length before, the place on the stack of
// its first new page (downwards), the pages that it takes (-1: refused); trim: pages given by the requests
// after it, -, its columns before, and kept.
struct Request {
    int first, len, place, pages;
};

__device__ __forceinline__ int64_t warp_sum_upto(int64_t x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
// The sum of x over the threads before this one; total: over all.
__device__ __forceinline__ int64_t sum_before(int64_t x, int64_t* wsum, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t upto = warp_sum_upto(x);
    if (lane == 31) wsum[warp] = upto;
    __syncthreads();
    const int64_t w = warp_sum_upto(wsum[lane]);
    total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    __syncthreads();
    return (warp ? before : 0) + upto - x;
}
__device__ __forceinline__ int stack_top(const TableArgs& A) {
    const int f = *A.free;
    return f < 0 ? 0 : f < A.p.stack_size ? f : A.p.stack_size;
}
__device__ __forceinline__ int64_t length_of(const TableArgs& A, int n) {
    const int64_t len = A.lens[n], cap = int64_t(A.p.max_pages) * A.p.page_size;
    return len < 0 ? 0 : len < cap ? len : cap;
}
__device__ __forceinline__ void cluster_barrier(bool several) {
    if (several)
        cluster_sync();
    else
        __syncthreads();
}

// FILL: slots and pages; UPDATE: lengths, count and sums
template <bool FILL, bool UPDATE>
__global__ void __launch_bounds__(TT_) k_table_extend(const TableArgs A, const FastDiv by_page) {
    extern __shared__ Request req[];
    __shared__ int64_t wsum[32];
    const gdn_table_problem& p = A.p;
    if (!UPDATE) tc::pdl_launch_dependents();  // the other launch sums alongside: what it reads is written by itself alone
    const int tid = threadIdx.x, N = p.num_seqs, per = (N + TT_ - 1) / TT_, n0 = min(N, tid * per), n1 = min(N, n0 + per);
    const int ps = p.page_size, top = stack_top(A);
    const int64_t cap = int64_t(p.max_pages) * ps;
    auto pages_of = [&](int64_t len) { return by_page.of(int(len + ps - 1)); };  // of at most cap tokens
    int64_t tokens = 0, pages = 0;
    for (int n = n0; n < n1; ++n) {
        const int64_t len = length_of(A, n), more = max(A.change[n], 0);
        tokens += more;
        if (len + more <= cap) pages += pages_of(len + more) - pages_of(len);
    }
    int64_t all, all_pages;
    int64_t at = sum_before(tokens, wsum, all), taken = sum_before(pages, wsum, all_pages);
    int64_t mine = 0;  // pages that this thread's requests get
    for (int n = n0; n < n1; ++n) {
        const int64_t len = length_of(A, n), more = max(A.change[n], 0);
        const bool fits = len + more <= cap;
        const int64_t need = fits ? pages_of(len + more) - pages_of(len) : 0;
        const bool granted = fits && (need == 0 || taken + need <= top);
        req[n] = {int(min(at, int64_t(0x7fffffff))), int(len), granted ? int(top - 1 - taken) : 0, granted ? int(need) : -1};
        if (granted) mine += need;
        at += more;
        taken += need;
    }
    int64_t given;
    sum_before(mine, wsum, given);
    const int ctas = int(gridDim.x), cta = int(blockIdx.x);  // one cluster where one launch does both
    cluster_barrier(FILL && UPDATE && ctas > 1);  // the requests are in shared memory; every CTA has read lengths and count
    if (!FILL) tc::pdl_wait();  // all CTAs of the launch before have ended
    if (UPDATE && cta == 0) {
        for (int n = tid; n < N; n += TT_) {
            const Request r = req[n];
            A.cu[n] = r.first;
            if (r.pages >= 0) A.lens[n] = r.len + max(A.change[n], 0);
        }
        if (tid == 0) {
            A.cu[N] = int(min(all, int64_t(0x7fffffff)));
            *A.free = int(top - given);
        }
    }
    if constexpr (!FILL) return;
    // pages, a warp to a request
    for (int n = cta * (TT_ / 32) + (tid >> 5); n < N; n += ctas * (TT_ / 32)) {
        const Request r = req[n];
        const int had = pages_of(r.len);
        for (int i = tid & 31; i < r.pages; i += 32) A.table[n * p.table_stride + had + i] = A.stack[r.place - i];
    }
    // slots
    const int64_t tokens_all = min(all, p.total);
    for (int64_t t = int64_t(cta) * TT_ + tid; t < p.total; t += int64_t(ctas) * TT_) {
        int64_t slot = -1;
        if (t < tokens_all) {
            int lo = 0, hi = N;  // the last request that begins at or before t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (req[mid].first <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            const Request r = req[lo];
            if (r.pages >= 0) {
                const int pos = r.len + int(t - r.first), column = by_page.of(pos), had = pages_of(r.len);
                const int page = column < had ? A.table[lo * p.table_stride + column] : A.stack[r.place - (column - had)];
                slot = int64_t(page) * ps + (pos - column * ps);
            }
        }
        A.slots[t] = slot;
    }
}

__global__ void __launch_bounds__(TT_) k_table_trim(const TableArgs A, const FastDiv by_page) {
    extern __shared__ Request req[];
    __shared__ int64_t wsum[32];
    const gdn_table_problem& p = A.p;
    const int tid = threadIdx.x, N = p.num_seqs, per = (N + TT_ - 1) / TT_, n0 = min(N, tid * per), n1 = min(N, n0 + per);
    const int top = stack_top(A);
    auto pages_of = [&](int64_t len) { return by_page.of(int(len + p.page_size - 1)); };
    int64_t pages = 0;
    for (int n = n0; n < n1; ++n) {
        const int64_t len = length_of(A, n), keep = min(len, int64_t(max(A.change[n], 0)));
        pages += pages_of(len) - pages_of(keep);
    }
    int64_t all, before = sum_before(pages, wsum, all);
    for (int n = n0; n < n1; ++n) {
        const int64_t len = length_of(A, n), keep = min(len, int64_t(max(A.change[n], 0)));
        const int has = pages_of(len), kept = pages_of(keep);
        before += has - kept;
        // 8192 rows can have more pages than 31 bits count; such places are past every stack's end
        req[n] = {int(min(all - before, int64_t(0x7fffffff))), int(keep), has, kept};
    }
    const int ctas = int(gridDim.x), cta = int(blockIdx.x);
    cluster_barrier(ctas > 1);
    if (cta == 0) {
        for (int n = tid; n < N; n += TT_) A.lens[n] = req[n].len;
        if (tid == 0) *A.free = int(min(top + all, int64_t(p.stack_size)));
    }
    for (int n = cta * (TT_ / 32) + (tid >> 5); n < N; n += ctas * (TT_ / 32)) {
        const Request r = req[n];
        for (int c = r.pages + (tid & 31); c < r.place; c += 32) {
            const int64_t to = int64_t(top) + r.first + (r.place - 1 - c);
            if (to < p.stack_size) A.stack[to] = A.table[n * p.table_stride + c];
        }
    }
}

// after: begins while the launch before, of the same kernel's other half, is at work
cudaError_t launch_table(void (*kern)(const TableArgs, const FastDiv), const char* name, const TableArgs& A, unsigned ctas, bool cluster, cudaStream_t st, bool after = false) {
    const int smem = A.p.num_seqs * int(sizeof(Request));
    cudaError_t e = smem_attr(kern, TABLE_SEQS * int(sizeof(Request)));
    if (e != cudaSuccess) return e;
    FastDiv by_page;
    by_page.set(uint32_t(A.p.page_size));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(TT_);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    if (after) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = after || (cluster && ctas > 1) ? 1 : 0;
    timing_begin(name, st);
    e = cudaLaunchKernelEx(&cfg, kern, A, by_page);
    timing_end(st);
    return e;
}

}  // namespace

cudaError_t launch_cache_write(const CacheArgs& A, cudaStream_t st) {
    if (A.p.dtype == GDN_FP32) return write_as<float, float>(A, st);
    return A.p.cache_dtype == GDN_BF16 ? write_as<__nv_bfloat16, __nv_bfloat16>(A, st) : write_as<__nv_bfloat16, __nv_fp8_e4m3>(A, st);
}
cudaError_t launch_table_extend(const TableArgs& A, cudaStream_t st) {
    // 500 prompts of up to 2000 tokens: a cluster of 8 CTAs takes 60 us, the two launches, the second summing beside the first, 15
    if (A.p.total > 32768) {
        const cudaError_t e = launch_table(k_table_extend<true, false>, "page_table_extend", A, unsigned(sm_count_cached()), false, st);
        return e != cudaSuccess ? e : launch_table(k_table_extend<false, true>, "page_table_update", A, 1, false, st, true);
    }
    return launch_table(k_table_extend<true, true>, "page_table_extend", A, A.p.total > 4096 ? 8 : 1, true, st);
}
cudaError_t launch_table_trim(const TableArgs& A, cudaStream_t st) {
    return launch_table(k_table_trim, "page_table_trim", A, A.p.num_seqs > 512 ? 8 : 1, true, st);
}

}  // namespace gdn
