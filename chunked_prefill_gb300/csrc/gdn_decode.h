// Internal launch interface of the decoding operators: the recurrent step, attention of one
// new token over a paged cache, and the RMS norm with the residual's addition.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

// Multiprocessors of the current device (looked up once per device).
int sm_count_cached();

struct StepArgs {
    gdn_step_problem p;  // strides filled in
    const void *q, *k, *v;
    const float *g, *beta, *A_log, *dt_bias, *state_in;
    float* state_out;
    void* o;
    int ahead;  // items from one whose state is in use to the one asked into L2 (set by the launch)
};
cudaError_t launch_step(const StepArgs& A, cudaStream_t st);

// Division of 0 <= x < 2^31 by a constant 1 <= d < 2^31: x / d = (x * mul) >> (32 + shift), with
// 2^shift the power of two that d lies above (2^shift < d <= 2^(shift+1)) and mul = ceil(2^(32+shift) / d)
// < 2^32: the error x (mul d - 2^(32+shift)) / (d 2^(32+shift)) < x / 2^(32+shift) < 1 / d for x < 2^31.
struct FastDiv {
    uint32_t mul, shift;
    void set(uint32_t d) {
        shift = 0;
        while ((2ull << shift) < d) ++shift;
        mul = d == 1 ? 0u : uint32_t(((1ull << (32 + shift)) + d - 1) / d);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int of(int x) const {
        return mul ? int(__umulhi(uint32_t(x), mul) >> shift) : x;
    }
#endif
};

struct PagedArgs {
    gdn_paged_problem p;  // strides filled in
    const void* q;
    void *k_cache, *v_cache;
    const int32_t *table, *lens;
    const void *k_new, *v_new;
    const float *k_scale, *v_scale;
    void* o;
    float* lse;
    int cluster;      // CTAs per (sequence, block of heads), joined in the kernel; 0: parts of a list
    int groups;       // of blocks of query heads (a block shares a kv-head)
    int heads;        // blocks in a group
    int64_t* before;  // [num_seqs + 1] tiles before each sequence, per block of heads
    float* part;      // partial results: two places per CTA, of a block's rows by D ...
    float2* part_ml;  // ... and their (max, sum) pairs
    FastDiv page_div;
};
// The launch for a problem (a function of the problem and the device alone): CTAs (a multiple of the
// groups of heads), rows to a block of query heads, and the bytes of the workspace (before, part_ml, part, in this order).
struct PagedPlan {
    int ctas, rows, groups, heads;
    int cluster;
    bool solo;  // CTAs of one warp
    size_t off_ml, off_part, bytes;
};
PagedPlan paged_plan(const gdn_paged_problem& p);
// What a launch needs to know of a kernel: tokens of a tile, rows of a block of heads, warps that share
// tiles, CTAs per multiprocessor.
struct PagedShape {
    int tok, rows, warps, ctas;
};
PagedShape paged_shape_bf16(int D);
PagedShape paged_shape_f8(int D);
PagedShape paged_shape_fp32(int D, int G);
cudaError_t launch_paged_bf16(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st);
cudaError_t launch_paged_f8(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st);
cudaError_t launch_paged_fp32(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st);
cudaError_t launch_paged(const PagedArgs& A, cudaStream_t st);

struct NormArgs {
    gdn_norm_problem p;  // strides filled in
    const void *x, *residual, *weight;
    void* y;
    float* y_scale;
    void* sum;
    const void *dy, *dsum;  // backward
    void* dx;
    float *dweight, *part;
    float inv_dim;  // 1 / dim
};
int norm_bwd_parts(const gdn_norm_problem& p);
// By the type of the rows; parts: the CTAs' shares of dweight that were written.
cudaError_t norm_fwd_bf16(const NormArgs& A, cudaStream_t st);
cudaError_t norm_fwd_fp32(const NormArgs& A, cudaStream_t st);
cudaError_t norm_bwd_bf16(const NormArgs& A, int& parts, cudaStream_t st);
cudaError_t norm_bwd_fp32(const NormArgs& A, int& parts, cudaStream_t st);
cudaError_t launch_norm_fwd(const NormArgs& A, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs& A, cudaStream_t st);

}  // namespace gdn
