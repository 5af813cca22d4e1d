// Root-mean-square norm with the residual's addition, with an optional 8-bit output, and its
// backward pass (include/gdn.h, gdn_rmsnorm_fwd and gdn_rmsnorm_bwd).
//   s = x + residual,  r = rsqrt(mean s^2 + eps),  y = r s w,  w = weight + offset
//   dx = r (w dy - n mean(w dy n)) + dsum,  dweight = sum_rows dy n,  n = r s
//
// Bound: HBM (forward: x, residual in, sum, y out; backward: s, dy, dsum in, dx out).  A row is
// read once into registers, NV vectors of VEC values a thread, and everything after its reductions
// comes from there.  A row belongs to LPR lanes of a warp (8, 16 or 32: short rows, several to a
// warp, no barrier) or, LPR = 0, to a whole CTA.  VEC is 16 bytes' worth of values where pointers,
// strides and dim allow it.  Contiguous rows of any other dim are taken in the 16-byte pieces of memory that
// they lie in (SHIFT: piece j of a row starts a0 = row dim mod VEC values before the row's value j VEC),
// value by value only in a row's first and last piece; other rows value by value (VEC = 1); rows past the registers' reach (max_threads x NV x
// VEC values) take the looping kernels at the end.
//
// The backward keeps a CTA on a fixed sequence of rows (row = CTA, CTA + grid, ...) with its share
// of dweight in registers; the CTAs' shares are then added in CTA order by a second launch, so
// dweight has the same bits in every run.
//
// Measured, bf16 (of the copy bandwidth measured on the same GPUs): 32768 x 4096 with the residual 154 us (7.0
// TB/s, 1.04); 8191 x 5120 with the residual to 8 bits in groups of 128, 48 us (6.1 TB/s, 0.92: issue slots 75 %
// busy); gradient of 32768 x 2048 with dsum 90.5 us (5.9 TB/s, 0.89: 86 us and the sum of 608 shares).
#include "gdn_norm.cuh"

namespace gdn {
namespace {

// dweight from the CTAs' shares: 16 columns by 64 runs of consecutive shares, the runs then added in a
// tree of fixed shape.
constexpr int DW_C = 16, DW_R = 64;
__global__ void __launch_bounds__(DW_C * DW_R) k_norm_dw(const float* part, int parts, int dim, float* dw) {
    __shared__ float run[DW_R][DW_C];
    const int c = threadIdx.x % DW_C, y = threadIdx.x / DW_C, i = blockIdx.x * DW_C + c;
    const int per = (parts + DW_R - 1) / DW_R, b1 = min(parts, (y + 1) * per);
    float t = 0.f;
    tc::pdl_wait();
    if (i < dim)
#pragma unroll 8
        for (int b = y * per; b < b1; ++b) t += part[int64_t(b) * dim + i];
    run[y][c] = t;
#pragma unroll
    for (int o = DW_R / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (y < o) run[y][c] += run[y + o][c];
    }
    if (y == 0 && i < dim) dw[i] = run[0][c];
}

}  // namespace

cudaError_t norm_fwd_bf16(const NormArgs& A, cudaStream_t st) { return fwd_type<__nv_bfloat16>(A, st); }
cudaError_t norm_bwd_bf16(const NormArgs& A, int& parts, cudaStream_t st) { return bwd_type<__nv_bfloat16>(A, parts, st); }

// CTAs of the backward at most, whatever the pointers' alignment turns out to be.
int norm_bwd_parts(const gdn_norm_problem& p) {
    const int full = full_vec(p.dtype);
    int most = 8;
    for (int i = 0; i < 3; ++i) {
        if (i == 1 && p.dim % full) continue;
        const int n = parts_of(p, layout_of(p.rows, p.dim, i ? full : 1, i == 2, true));
        if (n > most) most = n;
    }
    return most;
}

cudaError_t launch_norm_fwd(const NormArgs& A, cudaStream_t st) {
    timing_begin("rmsnorm_fwd", st);
    const cudaError_t e = A.p.dtype == GDN_BF16 ? norm_fwd_bf16(A, st) : norm_fwd_fp32(A, st);
    timing_end(st);
    return e;
}

cudaError_t launch_norm_bwd(const NormArgs& A, cudaStream_t st) {
    const gdn_norm_problem& p = A.p;
    int parts = 0;
    timing_begin("rmsnorm_bwd", st);
    const cudaError_t e = p.dtype == GDN_BF16 ? norm_bwd_bf16(A, parts, st) : norm_bwd_fp32(A, parts, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
    timing_begin("rmsnorm_dweight", st);
    const cudaError_t e2 = launch_pdl(k_norm_dw, dim3((p.dim + DW_C - 1) / DW_C), dim3(DW_C * DW_R), 0, st, static_cast<const float*>(A.part), parts, int(p.dim), A.dweight);
    timing_end(st);
    return e2;
}

}  // namespace gdn
