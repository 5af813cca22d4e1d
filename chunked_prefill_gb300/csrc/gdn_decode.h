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
};
cudaError_t launch_step(const StepArgs& A, cudaStream_t st);

struct PagedArgs {
    gdn_paged_problem p;  // strides filled in
    const void* q;
    void *k_cache, *v_cache;
    const int32_t *table, *lens;
    const void *k_new, *v_new;
    const float *k_scale, *v_scale;
    void* o;
    float* lse;
    float* part;     // partial outputs [rows][split][D], then their (max, sum) pairs
    int splits;      // ranges of the cache per sequence at most
    int split_len;   // tokens per range
};
// Ranges that the cache is split into (a function of the problem and the device alone).
void paged_plan(const gdn_paged_problem& p, int* splits, int* split_len);
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
};
int norm_bwd_parts(const gdn_norm_problem& p);
cudaError_t launch_norm_fwd(const NormArgs& A, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs& A, cudaStream_t st);

}  // namespace gdn
