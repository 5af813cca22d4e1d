// Tile products of attention on the CUDA cores (fp32): 256 threads as 16 x 16, thread (ty, tx) holding rows
// ty + 16 i; tiles in shared memory with 4 floats between rows, so that 16-byte reads of 8 rows fall on
// distinct banks.
#pragma once
#include "gdn_attn.cuh"

namespace gdn {
namespace {

constexpr int ST = 256;

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// rows [0, R) of D values at `stride` into dst, zeros from `valid` on
template <int R, int D>
__device__ __forceinline__ void load_rows(float* dst, const float* src, int64_t stride, int valid) {
#pragma unroll 4
    for (int i = threadIdx.x; i < R * (D / 4); i += ST) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        *reinterpret_cast<float4*>(dst + r * (D + 4) + d) = r < valid ? ld4(src + r * stride + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// c[i][j] = sum_k A[ty + 16 i][k] B[tx + 16 j][k]
template <int MI, int NJ, int K>
__device__ __forceinline__ void mul_nt(float (&c)[MI][NJ], const float* A, const float* B) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) c[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float4 a[MI], b[NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = ld4(A + (ty + 16 * i) * (K + 4) + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = ld4(B + (tx + 16 * j) * (K + 4) + k);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                c[i][j] = fmaf(a[i].x, b[j].x, c[i][j]);
                c[i][j] = fmaf(a[i].y, b[j].y, c[i][j]);
                c[i][j] = fmaf(a[i].z, b[j].z, c[i][j]);
                c[i][j] = fmaf(a[i].w, b[j].w, c[i][j]);
            }
    }
}

// c[i][4 v + e] += sum_n P(ty + 16 i, n) V[n][64 v + 4 tx + e] over n < count, with P(r, n) = P[r ld + n], or
// P[n ld + r] where TRANS.  counts(i, n): of a masked tile, whether row i's product with n counts at all
// (a weight of 0 would make NaN of an infinite value).
template <int MI, int D, bool TRANS, bool MASKED, typename F>
__device__ __forceinline__ void mul_add(float (&c)[MI][D / 16], int count, const float* P, int ld, const float* V, F counts) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int n = 0; n < count; ++n) {
        float p[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) p[i] = TRANS ? P[n * ld + ty + 16 * i] : P[(ty + 16 * i) * ld + n];
#pragma unroll
        for (int v = 0; v < D / 64; ++v) {
            const float4 x = ld4(V + n * (D + 4) + 64 * v + 4 * tx);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if (MASKED && !counts(i, n)) continue;
                c[i][4 * v] = fmaf(p[i], x.x, c[i][4 * v]);
                c[i][4 * v + 1] = fmaf(p[i], x.y, c[i][4 * v + 1]);
                c[i][4 * v + 2] = fmaf(p[i], x.z, c[i][4 * v + 2]);
                c[i][4 * v + 3] = fmaf(p[i], x.w, c[i][4 * v + 3]);
            }
        }
    }
}

// over the 16 threads that share rows
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void st4(float* p, float a, float b, float c, float d) { *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d); }
// One step of a running softmax over a tile of BN keys: z scores in units of log 2 (-inf where masked), in
// place of which the weights are left at P [BM][BN + 4]; statistics and accumulators follow.
template <int MI, int NJ, int DV>
__device__ __forceinline__ void softmax_step(float (&z)[MI][NJ], float (&m)[MI], float (&l)[MI], float (&acc)[MI][DV], float* P) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        float top = z[i][0];
#pragma unroll
        for (int j = 1; j < NJ; ++j) top = fmaxf(top, z[i][j]);
        top = fmaxf(m[i], row_max(top));
        const float sub = top == -INFINITY ? 0.f : top, c = ex2(m[i] - sub);
        m[i] = top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float w = ex2(z[i][j] - sub);
            sum += w;
            P[(ty + 16 * i) * (16 * NJ + 4) + tx + 16 * j] = w;
        }
        l[i] = fmaf(l[i], c, sum);  // of this thread's keys; summed over the row at the end
#pragma unroll
        for (int d = 0; d < DV; ++d) acc[i][d] *= c;
    }
}

}  // namespace
}  // namespace gdn
