// Attention of one new token per sequence over a paged key-value cache (include/gdn.h,
// gdn_paged_attn_decode): o_h = sum_t softmax(scale <q_h, k_t>)_t v_t, lse_h = log sum_t e^{z_t}.
//
// A sequence's tokens are cut into ranges of split_len tokens; a CTA takes one range of one
// kv-head (and a block of its query heads), keeping a running maximum m, sum l of e^{z - m} and
// accumulator of e^{z - m} v: one pass over keys and values.  Ranges are joined by a second
// kernel from (accumulator, m, l) triples in range order; a sequence of one range is written out
// directly.  Bound: HBM, 2 D bytes-per-value per token and kv-head.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_common.cuh"
#include "gdn_decode.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr float F8_MAX = 448.f;

// What a CTA has to do for sequence n.
struct Range {
    int len, first, count;  // tokens, the first one attended to, ranges
};
__device__ __forceinline__ Range range_of(const PagedArgs& A, int n) {
    const int64_t cap = int64_t(A.p.max_pages) * A.p.page_size;
    Range R;
    const int64_t len = A.lens[n];
    R.len = int(len < 0 ? 0 : len < cap ? len : cap);
    R.first = A.p.window > 0 && R.len > A.p.window ? R.len - A.p.window : 0;
    R.count = (R.len - R.first + A.split_len - 1) / A.split_len;
    if (R.count < 1) R.count = 1;
    return R;
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
__device__ __forceinline__ float from_cache(float x) { return x; }
__device__ __forceinline__ float from_cache(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float from_cache(__nv_fp8_e4m3 x) { return float(x); }

constexpr int PT = 128;  // threads
constexpr int GB = 4;    // query heads per CTA

template <typename C, int D> struct Lanes {
    static constexpr int E = (16 / int(sizeof(C)) > D / 32) ? 16 / int(sizeof(C)) : D / 32;  // values per lane
    static constexpr int LP = D / E;                                                         // lanes per token
    static constexpr int GROUPS = PT / LP;
};

template <typename C, int E>
__device__ __forceinline__ void load_row(const C* p, float (&x)[E]) {
    constexpr int W = 16 / int(sizeof(C));
#pragma unroll
    for (int b = 0; b < E / W; ++b) {
        C v[W];
        *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p + b * W);
#pragma unroll
        for (int e = 0; e < W; ++e) x[b * W + e] = from_cache(v[e]);
    }
}

template <typename Act, typename C, int D>
__global__ void __launch_bounds__(PT) k_paged(const PagedArgs A) {
    using L = Lanes<C, D>;
    constexpr int E = L::E, LP = L::LP, GROUPS = L::GROUPS;
    __shared__ __align__(16) float acc_s[GROUPS][GB][D];
    __shared__ float ml_s[GROUPS][GB][2];
    __shared__ __align__(16) C new_s[2][D];
    const gdn_paged_problem& p = A.p;
    const int tid = threadIdx.x, lane = tid % LP, grp = tid / LP;
    const int G = p.Hq / p.Hkv, nb = (G + GB - 1) / GB;
    const int split = blockIdx.x, hk = blockIdx.y / nb, hb = (blockIdx.y % nb) * GB, n = blockIdx.z;
    const Range R = range_of(A, n);
    if (split >= R.count) return;
    const int t0 = R.first + split * A.split_len, t1 = min(R.len, t0 + A.split_len);
    const float ks = A.k_scale ? A.k_scale[hk] : 1.f, vs = A.v_scale ? A.v_scale[hk] : 1.f;
    const int32_t* table = A.table + n * p.table_stride;
    const C* kc = static_cast<const C*>(A.k_cache) + hk * p.k_head_stride;
    const C* vc = static_cast<const C*>(A.v_cache) + hk * p.v_head_stride;

    int t_new = -1;  // the position whose row comes from k_new, v_new
    if (A.k_new && R.len > 0 && R.len == t1) {
        t_new = R.len - 1;
        const int page = table[t_new / p.page_size], slot = t_new % p.page_size;
        const bool in = page >= 0 && page < p.num_pages;
        for (int i = tid; i < D; i += PT) {
            const int64_t at = n * p.new_stride + hk * D + i;
            new_s[0][i] = to_cache<C>(to_f(static_cast<const Act*>(A.k_new)[at]), ks);
            new_s[1][i] = to_cache<C>(to_f(static_cast<const Act*>(A.v_new)[at]), vs);
            if (in && hb == 0) {
                const_cast<C*>(kc)[page * p.k_page_stride + slot * p.k_token_stride + i] = new_s[0][i];
                const_cast<C*>(vc)[page * p.v_page_stride + slot * p.v_token_stride + i] = new_s[1][i];
            }
        }
        __syncthreads();
    }

    float q[GB][E], acc[GB][E], m[GB], l[GB];
#pragma unroll
    for (int h = 0; h < GB; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[h][e] = 0.f;
            q[h][e] = hb + h < G ? to_f(static_cast<const Act*>(A.q)[n * p.q_stride + (hk * G + hb + h) * D + lane * E + e]) : 0.f;
        }
    }
    const float zs = p.scale * ks;
    for (int t = t0 + grp; t - grp < t1; t += GROUPS) {
        bool live = t < t1;
        float kx[E] = {}, vx[E] = {};
        if (live) {
            if (t == t_new) {
                load_row<C, E>(&new_s[0][lane * E], kx);
                load_row<C, E>(&new_s[1][lane * E], vx);
                const int page = table[t / p.page_size];
                live = page >= 0 && page < p.num_pages;
            } else {
                const int page = table[t / p.page_size], slot = t % p.page_size;
                live = page >= 0 && page < p.num_pages;
                if (live) {
                    load_row<C, E>(kc + page * p.k_page_stride + slot * p.k_token_stride + lane * E, kx);
                    load_row<C, E>(vc + page * p.v_page_stride + slot * p.v_token_stride + lane * E, vx);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) z = fmaf(q[h][e], kx[e], z);
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            if (live) {
                z *= zs;
                const float mn = fmaxf(m[h], z), c = m[h] == -INFINITY ? 0.f : expf(m[h] - mn);
                const float e0 = mn == -INFINITY ? 0.f : expf(z - mn);
                l[h] = fmaf(l[h], c, e0);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[h][e] = fmaf(acc[h][e], c, e0 * vx[e]);
                m[h] = mn;
            }
        }
    }
#pragma unroll
    for (int h = 0; h < GB; ++h) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc_s[grp][h][lane * E + e] = acc[h][e];
        if (lane == 0) {
            ml_s[grp][h][0] = m[h];
            ml_s[grp][h][1] = l[h];
        }
    }
    __syncthreads();
    for (int i = tid; i < GB * D; i += PT) {
        const int h = i / D, d = i % D;
        if (hb + h >= G) break;
        float M = -INFINITY, S = 0.f, a = 0.f;
        for (int g = 0; g < GROUPS; ++g) M = fmaxf(M, ml_s[g][h][0]);
        for (int g = 0; g < GROUPS; ++g) {
            const float c = ml_s[g][h][0] == -INFINITY ? 0.f : expf(ml_s[g][h][0] - M);
            S = fmaf(ml_s[g][h][1], c, S);
            a = fmaf(acc_s[g][h][d], c, a);
        }
        const int64_t row = int64_t(n) * p.Hq + hk * G + hb + h;
        if (R.count == 1) {
            static_cast<Act*>(A.o)[row * D + d] = from_f<Act>(S > 0.f || S != S ? a / S * vs : 0.f);
            if (A.lse && d == 0) A.lse[row] = M + logf(S);
        } else {
            A.part[(row * A.splits + split) * D + d] = a;
            if (d == 0) {
                float* ml = A.part + int64_t(p.num_seqs) * p.Hq * A.splits * D + (row * A.splits + split) * 2;
                ml[0] = M;
                ml[1] = S;
            }
        }
    }
}

template <typename Act>
__global__ void k_paged_join(const PagedArgs A) {
    const gdn_paged_problem& p = A.p;
    const int64_t row = blockIdx.x;
    const int n = int(row / p.Hq), h = int(row % p.Hq), d = threadIdx.x, D = p.D;
    const Range R = range_of(A, n);
    if (R.count == 1) return;
    const float* ml = A.part + int64_t(p.num_seqs) * p.Hq * A.splits * D + row * A.splits * 2;
    float M = -INFINITY, S = 0.f, a = 0.f;
    for (int i = 0; i < R.count; ++i) M = fmaxf(M, ml[2 * i]);
    for (int i = 0; i < R.count; ++i) {
        const float c = ml[2 * i] == -INFINITY ? 0.f : expf(ml[2 * i] - M);
        S = fmaf(ml[2 * i + 1], c, S);
        a = fmaf(A.part[(row * A.splits + i) * D + d], c, a);
    }
    const float vs = A.v_scale ? A.v_scale[h / (p.Hq / p.Hkv)] : 1.f;
    static_cast<Act*>(A.o)[row * D + d] = from_f<Act>(S > 0.f || S != S ? a / S * vs : 0.f);
    if (A.lse && d == 0) A.lse[row] = M + logf(S);
}

template <typename Act, typename C, int D>
cudaError_t launch_d(const PagedArgs& A, cudaStream_t st) {
    const int G = A.p.Hq / A.p.Hkv;
    dim3 grid(A.splits, A.p.Hkv * ((G + GB - 1) / GB), A.p.num_seqs);
    timing_begin("paged_attn", st);
    k_paged<Act, C, D><<<grid, PT, 0, st>>>(A);
    timing_end(st);
    if (A.splits > 1) {
        timing_begin("paged_attn_join", st);
        k_paged_join<Act><<<unsigned(int64_t(A.p.num_seqs) * A.p.Hq), D, 0, st>>>(A);
        timing_end(st);
    }
    return cudaGetLastError();
}

template <typename Act, typename C>
cudaError_t launch_c(const PagedArgs& A, cudaStream_t st) {
    return A.p.D == 64 ? launch_d<Act, C, 64>(A, st) : A.p.D == 128 ? launch_d<Act, C, 128>(A, st) : launch_d<Act, C, 256>(A, st);
}

}  // namespace

void paged_plan(const gdn_paged_problem& p, int* splits, int* split_len) {
    const int64_t cap = int64_t(p.max_pages) * p.page_size;
    const int64_t most = p.window > 0 && p.window < cap ? p.window : cap;
    *split_len = 1024;
    *splits = int((most + *split_len - 1) / *split_len);
    if (*splits < 1) *splits = 1;
}

cudaError_t launch_paged(const PagedArgs& A, cudaStream_t st) {
    if (A.p.dtype == GDN_FP32) return launch_c<float, float>(A, st);
    if (A.p.cache_dtype == GDN_BF16) return launch_c<__nv_bfloat16, __nv_bfloat16>(A, st);
    return launch_c<__nv_bfloat16, __nv_fp8_e4m3>(A, st);
}

}  // namespace gdn
