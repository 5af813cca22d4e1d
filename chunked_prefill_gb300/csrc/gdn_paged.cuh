// What the kernels of attention over a paged cache share: the division of the work, the joins and the
// launches (see gdn_paged.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_decode.h"
#include "gdn_internal.h"
#include "tc05.cuh"

namespace gdn {
namespace {

constexpr float F8_MAX = 448.f;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Sequence n's tokens: those attended to are [first, len); its tiles of `tok` tokens start at base,
// which is first down to a multiple of 16 (a tile's rows then share a page of 16 k tokens).
struct Range {
    int len, first, base;
    bool fits;  // in the table: a new token has a place
    __device__ __forceinline__ int tiles(int tok) const {  // one at least: an empty row is written too
        const int64_t n = (int64_t(len) - base + tok - 1) / tok;
        return n > 1 ? int(n) : 1;
    }
};
__device__ __forceinline__ Range range_of(const PagedArgs& A, int n) {
    const int64_t cap = int64_t(A.p.max_pages) * A.p.page_size;
    Range R;
    const int64_t len = A.lens[n];
    R.len = int(len < 0 ? 0 : len < cap ? len : cap);
    R.fits = len > 0 && len <= cap;
    R.first = A.p.window > 0 && R.len > A.p.window ? R.len - A.p.window : 0;
    R.base = R.first & ~15;
    return R;
}

// A CTA's part [lo, hi) of the list of all tiles, and where it begins: tile `at` of block of heads
// `head` (of the group's A.heads) of sequence n.
struct Part {
    int64_t lo, hi;
    int n, group, head, at;
};
// a / b for a >= 0, b > 0; 64-bit division costs half a microsecond that small problems feel
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}
__device__ __forceinline__ int64_t share_of(int64_t total, int parts, int warps) {
    // a multiple of the warps (a power of two), so that none is left out
    return (quotient(total + parts - 1, parts) + warps - 1) & ~int64_t(warps - 1);
}
// CTA 0 also leaves the number of tiles before each sequence (per block of heads) in A.before.
template <int T, typename Args>
__device__ Part find_part(const Args& A, int tok, int warps) {
    if constexpr (std::is_same_v<Args, PagedArgs>) {
        if (A.cluster) {  // a cluster of CTAs per (sequence, block of heads), equal parts of its tiles
            const int pair = blockIdx.x / A.cluster, r = blockIdx.x % A.cluster, blocks = A.groups * A.heads, n = pair / blocks, b = pair % blocks;
            const int tiles = range_of(A, n).tiles(tok), share = ((tiles + A.cluster - 1) / A.cluster + warps - 1) / warps * warps;
            const int at = min(r * share, tiles);
            return {0, min(share, tiles - at), n, b % A.groups, b / A.groups, at};
        }
    }
    __shared__ int64_t wsum[T / 32];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 31, N = A.p.num_seqs;
    const int per = (N + T - 1) / T, n0 = min(N, tid * per), n1 = min(N, n0 + per);
    int64_t mine = 0;
    for (int n = n0; n < n1; ++n) mine += range_of(A, n).tiles(tok);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) wsum[tid >> 5] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
        if (w < tid >> 5) upto += wsum[w];
        total += wsum[w];
    }
    int64_t run = upto - mine;
    const int64_t share = share_of(total * A.heads, gridDim.x / A.groups, warps);
    Part P;
    P.lo = blockIdx.x / A.groups * share;
    P.hi = min(P.lo + share, total * A.heads);
    if (blockIdx.x == 0) {
        int64_t r = run;
        for (int n = n0; n < n1; ++n) {
            A.before[n] = r;
            r += range_of(A, n).tiles(tok);
        }
        if (tid == T - 1) A.before[N] = total;
    }
    if (P.lo < P.hi && run * A.heads <= P.lo && P.lo < upto * A.heads) {
        int n = n0, t = range_of(A, n).tiles(tok);
        while ((run + t) * A.heads <= P.lo) {
            run += t;
            t = range_of(A, ++n).tiles(tok);
        }
        const int64_t rest = P.lo - run * A.heads, head = quotient(rest, t);
        found[0] = n;
        found[1] = int(head);
        found[2] = int(rest - head * t);
    }
    __syncthreads();
    P.n = found[0], P.group = blockIdx.x % A.groups, P.head = found[1], P.at = found[2];
    return P;
}
// Where a CTA leaves rows [0, ROWS) of a pair that it has a part of: in its first place where the
// pair began before its part, in its second where the pair goes on after it.
__device__ __forceinline__ int64_t place_of(int cta, bool first, int rows) { return (int64_t(cta) * 2 + (first ? 0 : 1)) * rows; }

// ---- clusters: the join through distributed shared memory
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Joins the cluster's CTAs' results -- rows of D at `res`, (max, sum) pairs at `ml`, at the same places of
// every CTA's shared memory -- in rank order, each CTA a slice of the values, and writes them out.
template <typename Act, int D, int T>
__device__ void join_cluster(const PagedArgs& A, uint32_t res, uint32_t ml, int n, int hk, int hb, int rows) {
    const gdn_paged_problem& p = A.p;
    const int r = blockIdx.x % A.cluster, total = rows * (D / 4), each = (total + A.cluster - 1) / A.cluster;
    const float vs = A.v_scale ? A.v_scale[hk] : 1.f;
    cluster_sync();
    for (int i = r * each + threadIdx.x; i < min(total, (r + 1) * each); i += T) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        float2 m[8];
        float4 x[8];
        float M = -INFINITY;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (c >= A.cluster) continue;
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];\n" : "=f"(m[c].x), "=f"(m[c].y) : "r"(in_cta(ml + h * 8, c)) : "memory");
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                         : "=f"(x[c].x), "=f"(x[c].y), "=f"(x[c].z), "=f"(x[c].w)
                         : "r"(in_cta(res + (h * D + d) * 4, c))
                         : "memory");
            M = fmaxf(M, m[c].x);
        }
        float S = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (c >= A.cluster || m[c].y == 0.f) continue;  // an empty part has no rows
            const float w = m[c].x == -INFINITY ? 0.f : exp2f(m[c].x - M);
            S = fmaf(m[c].y, w, S);
            a.x = fmaf(x[c].x, w, a.x);
            a.y = fmaf(x[c].y, w, a.y);
            a.z = fmaf(x[c].z, w, a.z);
            a.w = fmaf(x[c].w, w, a.w);
        }
        const int64_t row = int64_t(n) * p.Hq + hk * (p.Hq / p.Hkv) + hb + h;
        const bool some = S > 0.f || S != S;
        const float f = some ? vs / S : 0.f;
        Act* o = static_cast<Act*>(A.o) + row * D + d;
        st2(o, a.x * f, a.y * f);
        st2(o + 2, a.z * f, a.w * f);
        if (A.lse && d == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
    }
    cluster_sync();  // the others have read this CTA's results
}

// a value of the new token's row in the cache's type
template <typename C> __device__ __forceinline__ C to_cache(float x, float scale);
template <> __device__ __forceinline__ float to_cache<float>(float x, float scale) { return x / scale; }
template <> __device__ __forceinline__ __nv_bfloat16 to_cache<__nv_bfloat16>(float x, float scale) {
    return __float2bfloat16_rn(x / scale);
}
template <> __device__ __forceinline__ __nv_fp8_e4m3 to_cache<__nv_fp8_e4m3>(float x, float scale) {
    const float y = x / scale;
    return __nv_fp8_e4m3(y != y ? y : fminf(fmaxf(y, -F8_MAX), F8_MAX));
}

// 2^x to 2^-22 of itself; -inf gives 0
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// copy of 16 bytes to shared memory, zeros where !in (the address is not read then)
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// Joins the parts of the rows that several CTAs have parts of, in the list's order.  A block of 8
// warps takes RPB rows: a warp each (8), or all 8 warps one row's parts (1: few rows, many parts).
constexpr int JW = 8;
template <typename Act, int D, int RPB>
__global__ void __launch_bounds__(32 * JW) k_paged_join(const PagedArgs A, int rows, int ctas, int warps) {
    constexpr int E = D / 32;
    __shared__ float acc_s[RPB == 1 ? JW : 1][D], ml_s[RPB == 1 ? JW : 1][2];
    tc::pdl_wait();
    const gdn_paged_problem& p = A.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = RPB == 1 ? blockIdx.x : int64_t(blockIdx.x) * JW + warp;
    if (row >= int64_t(p.num_seqs) * p.Hq) return;  // with RPB == 1 never
    const int n = int(quotient(row, p.Hq)), h = int(row - int64_t(n) * p.Hq), G = p.Hq / p.Hkv, nb = (G + rows - 1) / rows;
    const int block = (h / G) * nb + (h % G) / rows, in = (h % G) % rows;
    const int head = block / A.groups, group = block % A.groups;
    const int64_t before = A.before[n], tiles = A.before[n + 1] - before;
    const int64_t share = share_of(A.before[p.num_seqs] * A.heads, ctas / A.groups, warps);
    const int64_t at0 = before * A.heads + head * tiles, at1 = at0 + tiles;
    const int c0 = int(quotient(at0, share)), c1 = int(quotient(at1 - 1, share));
    if (c0 == c1) return;  // that CTA wrote it out
    // parts c0 .. c1; this warp's: c0 + first, first + step, ...
    const int parts = c1 - c0 + 1, first = RPB == 1 ? warp : 0, step = RPB == 1 ? JW : 1;
    auto place = [&](int i) { return place_of((c0 + i) * A.groups + group, i > 0, rows) + in; };  // the pair begins in c0's part
    float M = -INFINITY, S = 0.f, acc[E] = {};
    // batches of parts, everything of a batch requested at once
    constexpr int NB = (D == 256 ? 4 : 8) * (RPB == 1 ? 2 : 1);
    for (int i0 = first; i0 < parts; i0 += step * NB) {
        float2 ml[NB];
        float x[NB][E];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int i = i0 + step * b;
            ml[b] = make_float2(-INFINITY, 0.f);
            if (i < parts) {
                const int64_t at = place(i);
                ml[b] = A.part_ml[at];
#pragma unroll
                for (int e = 0; e < E; ++e) x[b][e] = A.part[at * D + 32 * e + lane];
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) x[b][e] = 0.f;
            }
        }
        float top = M;
#pragma unroll
        for (int b = 0; b < NB; ++b) top = fmaxf(top, ml[b].x);
        const float c = M == -INFINITY ? 0.f : ex2(M - top);
        M = top;
        S *= c;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= c;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float w = ml[b].x == -INFINITY ? 0.f : ex2(ml[b].x - M);
            S = fmaf(ml[b].y, w, S);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(x[b][e], w, acc[e]);
        }
    }
    if constexpr (RPB == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc_s[warp][32 * e + lane] = acc[e];
        if (lane == 0) {
            ml_s[warp][0] = M;
            ml_s[warp][1] = S;
        }
        __syncthreads();
        if (warp > 0) return;
        S = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < JW; ++w) M = fmaxf(M, ml_s[w][0]);
#pragma unroll
        for (int w = 0; w < JW; ++w) {
            const float c = ml_s[w][0] == -INFINITY ? 0.f : ex2(ml_s[w][0] - M);
            S = fmaf(ml_s[w][1], c, S);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(acc_s[w][32 * e + lane], c, acc[e]);
        }
    }
    const bool some = S > 0.f || S != S;
    const float f = some ? (A.v_scale ? A.v_scale[h / G] : 1.f) / S : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) static_cast<Act*>(A.o)[row * D + 32 * e + lane] = from_f<Act>(acc[e] * f);
    if (A.lse && lane == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
}

template <typename... K>
cudaError_t launch_clusters(void (*kern)(K...), const PagedArgs& A, int ctas, int threads, size_t smem, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = A.cluster > 1 ? A.cluster : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = A.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, A);
}

template <typename Act, int D>
cudaError_t launch_join(const PagedArgs& A, const PagedPlan& plan, const PagedShape& s, cudaStream_t st) {
    if (plan.cluster) return cudaGetLastError();
    const int64_t rows = int64_t(A.p.num_seqs) * A.p.Hq;
    // a block to a row where a row has more than 4 parts on average (one sequence of 131071 tokens: 46.7 us
    // instead of 47.8 with the parts in batches half as long; 30 of up to 6000 tokens, 8 kv-heads, 256 features, two parts
    // to a row: 102 us with a warp to a row instead of 106)
    const bool many = plan.ctas > int64_t(4) * A.p.num_seqs * plan.groups * plan.heads;
    timing_begin("paged_attn_join", st);
    const cudaError_t e =
        many ? launch_pdl(k_paged_join<Act, D, 1>, dim3(unsigned(rows)), dim3(32 * JW), 0, st, A, s.rows, plan.ctas, s.warps)
             : launch_pdl(k_paged_join<Act, D, JW>, dim3(unsigned((rows + JW - 1) / JW)), dim3(32 * JW), 0, st, A, s.rows, plan.ctas, s.warps);
    timing_end(st);
    return e;
}

}  // namespace
}  // namespace gdn
