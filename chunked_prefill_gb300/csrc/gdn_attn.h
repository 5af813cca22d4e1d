// Internal launch interface of attention over prompts, of drafted trees over a paged cache, and of the
// cache's own operators (writing it, its page tables).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdn.h"
#include "gdn_decode.h"

namespace gdn {

struct PromptArgs {
    gdn_prompt_problem p;  // strides filled in
    const void *q, *k, *v;
    void* o;
    float* lse;
    void* o_rest;
    // backward
    const void *o_in, *rest_in, *dO;
    const float *lse_in, *dlse;
    void *dq, *dk, *dv;
    // [Hq][rows] pairs of (lse in units of log 2, <dO, o> - dlse) of every query, rows = total_q up to a multiple of 128
    float2* stat;
    int64_t stat_rows;
};
size_t prompt_bwd_workspace(const gdn_prompt_problem& p);
cudaError_t launch_prompt_fwd_simt(const PromptArgs& A, cudaStream_t st);
cudaError_t launch_prompt_bwd_simt(const PromptArgs& A, cudaStream_t st);
// bf16, on the tensor cores
cudaError_t launch_prompt_fwd_tc(const PromptArgs& A, cudaStream_t st);
int prompt_fwd_status();  // not 0 where a wait of an earlier launch gave up (reads and clears it; synchronises)
cudaError_t prompt_fwd_wait_out(int32_t limit_us, cudaStream_t st);  // of its test: a wait that gives up
cudaError_t launch_prompt_bwd_tc(const PromptArgs& A, cudaStream_t st);
int prompt_bwd_parts(const gdn_prompt_problem& p);
int prompt_bwd_status();
cudaError_t prompt_bwd_wait_out(int32_t limit_us, cudaStream_t st);
cudaError_t launch_prompt_stat(const PromptArgs& A, cudaStream_t st);

struct TreeArgs {
    gdn_tree_problem p;  // strides filled in
    const void *q, *k_new, *v_new, *k_cache, *v_cache;
    const int32_t *table, *lens, *parents;
    const float *k_scale, *v_scale;
    void* o;
    float* lse;
    // Blocks of rows (drafted token by drafted token, the query heads of a kv-head), kv-head by kv-head, dealt
    // to `groups` groups of `heads` blocks: as PagedArgs.
    int groups, heads;
    int64_t* before;  // [num_seqs + 1] tiles before each sequence, per block
    float* part;      // partial results, two places per CTA
    float2* part_ml;
    FastDiv page_div;
};
struct TreePlan {
    int ctas, rows, tok;  // CTAs, rows of a block, cached tokens of a tile
    int groups, heads;
    size_t off_ml, off_part, bytes;
};
TreePlan tree_plan(const gdn_tree_problem& p);
// What a launch needs to know of a kernel: rows of a block, tokens of a tile, CTAs per multiprocessor.
struct TreeShape {
    int rows, tok, ctas;
};
cudaError_t launch_tree_bf16(const TreeArgs& A, const TreePlan& plan, cudaStream_t st);
cudaError_t launch_tree_f8(const TreeArgs& A, const TreePlan& plan, cudaStream_t st);
int tree_status_bf16();
int tree_status_f8();
cudaError_t tree_wait_out_bf16(int32_t limit_us, cudaStream_t st);
cudaError_t tree_wait_out_f8(int32_t limit_us, cudaStream_t st);
cudaError_t launch_tree(const TreeArgs& A, cudaStream_t st);

struct CacheArgs {
    gdn_cache_problem p;
    const void *k, *v;
    void *k_cache, *v_cache;
    const int64_t* slots;
    const int32_t* rows;
    const float *k_scale, *v_scale;
};
cudaError_t launch_cache_write(const CacheArgs& A, cudaStream_t st);

struct TableArgs {
    gdn_table_problem p;
    int32_t *table, *lens;
    const int32_t* change;  // new_lens or keep_lens
    int32_t *stack, *free;
    int64_t* slots;
    int32_t* cu;
};
constexpr int TABLE_SEQS = 8192;
cudaError_t launch_table_extend(const TableArgs& A, cudaStream_t st);
cudaError_t launch_table_trim(const TableArgs& A, cudaStream_t st);

}  // namespace gdn
