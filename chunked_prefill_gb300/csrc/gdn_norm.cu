// Root-mean-square norm with the residual's addition, with an optional 8-bit output, and its
// backward pass (include/gdn.h, gdn_rmsnorm_fwd and gdn_rmsnorm_bwd).
//   s = x + residual,  r = rsqrt(mean s^2 + eps),  y = r s w,  w = weight + offset
//   dx = r (w dy - n mean(w dy n)) + dsum,  dweight = sum_rows dy n,  n = r s
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_common.cuh"
#include "gdn_decode.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int NT = 256;               // threads per row
constexpr float F8_MAX = 448.f;
constexpr float F8_TINY = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// max that keeps a NaN
__device__ __forceinline__ float nan_max(float a, float b) { return (a > b || a != a) ? a : b; }
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = nan_max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <bool MAX>
__device__ float block_red(float v, float* red) {
    v = MAX ? warp_max(v) : warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = red[0];
    for (int w = 1; w < NT / 32; ++w) t = MAX ? nan_max(t, red[w]) : t + red[w];
    return t;
}

__device__ __forceinline__ float weight_at(const void* w, int dt, int i) {
    return dt == GDN_BF16 ? to_f(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

template <typename Op>
__global__ void __launch_bounds__(NT) k_norm_fwd(const NormArgs A) {
    const gdn_norm_problem& p = A.p;
    __shared__ float red[NT / 32];
    const Op* xr = static_cast<const Op*>(A.x);
    const Op* rr = static_cast<const Op*>(A.residual);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const Op* x = xr + row * p.x_stride;
        const Op* res = rr ? rr + row * p.residual_stride : nullptr;
        auto at = [&](int i) { return res ? to_f(x[i]) + to_f(res[i]) : to_f(x[i]); };
        float ss = 0.f;
        for (int i = threadIdx.x; i < p.dim; i += NT) {
            const float v = at(i);
            ss = fmaf(v, v, ss);
        }
        const float r = rsqrtf(block_red<false>(ss, red) / float(p.dim) + p.eps);
        auto y_at = [&](int i) { return at(i) * r * (weight_at(A.weight, p.weight_dtype, i) + p.weight_offset); };
        if (p.out_dtype == GDN_E4M3) {
            const int group = p.group ? p.group : p.dim;
            for (int g = 0; g < p.dim / group; ++g) {
                float m = 0.f;
                for (int i = threadIdx.x; i < group; i += NT) m = nan_max(m, fabsf(y_at(g * group + i)));
                m = block_red<true>(m, red);
                const float sc = nan_max(m / F8_MAX, F8_TINY);
                if (threadIdx.x == 0) A.y_scale[row * (p.dim / group) + g] = sc;
                for (int i = threadIdx.x; i < group; i += NT)
                    static_cast<__nv_fp8_e4m3*>(A.y)[row * p.dim + g * group + i] = __nv_fp8_e4m3(y_at(g * group + i) / sc);
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < p.dim; i += NT) {
            const float v = at(i), y = y_at(i);
            if (A.sum) static_cast<Op*>(A.sum)[row * p.dim + i] = from_f<Op>(v);
            if (p.out_dtype != GDN_E4M3) static_cast<Op*>(A.y)[row * p.dim + i] = from_f<Op>(y);
        }
    }
}

template <typename Op>
__global__ void __launch_bounds__(NT) k_norm_bwd(const NormArgs A) {
    const gdn_norm_problem& p = A.p;
    __shared__ float red[NT / 32];
    float* part = A.part + int64_t(blockIdx.x) * p.dim;
    for (int i = threadIdx.x; i < p.dim; i += NT) part[i] = 0.f;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const Op* x = static_cast<const Op*>(A.x) + row * p.x_stride;
        const Op* dy = static_cast<const Op*>(A.dy) + row * p.dy_stride;
        const Op* ds = A.dsum ? static_cast<const Op*>(A.dsum) + row * p.dsum_stride : nullptr;
        float ss = 0.f, c = 0.f;
        for (int i = threadIdx.x; i < p.dim; i += NT) {
            const float v = to_f(x[i]), w = weight_at(A.weight, p.weight_dtype, i) + p.weight_offset;
            ss = fmaf(v, v, ss);
            c = fmaf(w * to_f(dy[i]), v, c);
        }
        const float r = rsqrtf(block_red<false>(ss, red) / float(p.dim) + p.eps);
        c = block_red<false>(c, red) * r / float(p.dim);
        for (int i = threadIdx.x; i < p.dim; i += NT) {
            const float n = to_f(x[i]) * r, d = to_f(dy[i]);
            const float w = weight_at(A.weight, p.weight_dtype, i) + p.weight_offset;
            const float add = ds ? to_f(ds[i]) : 0.f;
            part[i] = fmaf(d, n, part[i]);
            static_cast<Op*>(A.dx)[row * p.dim + i] = from_f<Op>(fmaf(r, w * d - n * c, add));
        }
    }
}

__global__ void __launch_bounds__(NT) k_norm_dw(const float* part, int parts, int dim, float* dw) {
    const int i = blockIdx.x * NT + threadIdx.x;
    if (i >= dim) return;
    float t = 0.f;
    for (int b = 0; b < parts; ++b) t += part[int64_t(b) * dim + i];
    dw[i] = t;
}

}  // namespace

int norm_bwd_parts(const gdn_norm_problem& p) {
    const int64_t most = 8 * int64_t(sm_count_cached());
    return int(p.rows < most ? (p.rows > 0 ? p.rows : 1) : most);
}

cudaError_t launch_norm_fwd(const NormArgs& A, cudaStream_t st) {
    const int64_t most = 1 << 20;
    const unsigned nb = unsigned(A.p.rows < most ? A.p.rows : most);
    timing_begin("rmsnorm_fwd", st);
    if (A.p.dtype == GDN_BF16)
        k_norm_fwd<__nv_bfloat16><<<nb, NT, 0, st>>>(A);
    else
        k_norm_fwd<float><<<nb, NT, 0, st>>>(A);
    timing_end(st);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormArgs& A, cudaStream_t st) {
    const int parts = norm_bwd_parts(A.p);
    timing_begin("rmsnorm_bwd", st);
    if (A.p.dtype == GDN_BF16)
        k_norm_bwd<__nv_bfloat16><<<parts, NT, 0, st>>>(A);
    else
        k_norm_bwd<float><<<parts, NT, 0, st>>>(A);
    k_norm_dw<<<(A.p.dim + NT - 1) / NT, NT, 0, st>>>(A.part, parts, A.p.dim, A.dweight);
    timing_end(st);
    return cudaGetLastError();
}

}  // namespace gdn
