// What the kernels of attention of drafted trees over a paged cache share (see gdn_tree.cu).
#pragma once
#include "gdn_attn.cuh"

namespace gdn {

// Sequence n's cached tokens: those that a drafted token may attend to are [first, len).  Its tiles are those
// of `tok` cached tokens from base on, and one more: the drafted tokens.
struct TreeRange {
    int len, first, base;
    __device__ __forceinline__ int cached(int tok) const { return (len - base + tok - 1) / tok; }
    __device__ __forceinline__ int tiles(int tok) const { return cached(tok) + 1; }
};
static __device__ __forceinline__ TreeRange range_of(const TreeArgs& A, int n) {
    const int64_t cap = int64_t(A.p.max_pages) * A.p.page_size, len = A.lens[n];
    TreeRange R;
    R.len = int(len < 0 ? 0 : len < cap ? len : cap);
    R.first = A.p.window > 0 && R.len >= A.p.window ? R.len - A.p.window + 1 : 0;
    R.base = min(R.first & ~15, R.len);
    return R;
}

namespace {

// Which drafted tokens (bits) a drafted token attends to, and its number of ancestors; none and -1 where
// there is no such token.
struct Tree {
    uint64_t sees[64];
    int depth[64];
};
__device__ __forceinline__ void read_token(const TreeArgs& A, int n, int t, uint64_t& sees, int& depth) {
    const int32_t* parents = A.parents + int64_t(n) * A.p.T;
    sees = 0, depth = -1;
    for (int at = t; at >= 0;) {
        ++depth;
        if (A.p.window == 0 || depth < A.p.window) sees |= uint64_t(1) << at;
        const int up = parents[at];
        if (up < -1 || up >= at) {
            sees = 0, depth = -1;
            break;
        }
        at = up;
    }
}
// By the first 64 threads of the CTA; the caller synchronises.
__device__ __forceinline__ void read_tree(const TreeArgs& A, int n, Tree& tree) {
    const int t = threadIdx.x;
    if (t >= 64) return;
    uint64_t sees = 0;
    int depth = -1;
    if (t < A.p.T) read_token(A, n, t, sees, depth);
    tree.sees[t] = sees;
    tree.depth[t] = depth;
}
// The first cached token that a drafted token `depth` deep attends to.
__device__ __forceinline__ int first_cached(const TreeArgs& A, const TreeRange& R, int depth) {
    const int64_t f = int64_t(R.len) + depth - A.p.window + 1;
    return A.p.window > 0 && f > 0 ? int(min(f, int64_t(R.len))) : 0;
}

// Joins the parts of the rows that several CTAs have parts of, in the list's order: a warp to a row.  A (sequence, block)
// that several have is found at the border between the first and the second of them: blocks (CTA, 8 rows at a
// time of its first block), of which those whose CTA is a second one work.  (A warp to every row of the output: 66 us for
// 64 sequences of 31 drafted tokens and 64 heads, with 150 borders among 512 blocks.)
template <typename Act, int D>
__global__ void __launch_bounds__(256) k_tree_join(const TreeArgs A, int rows, int ctas) {
    constexpr int E = D / 32, NB = D == 256 ? 4 : 8;
    tc::pdl_wait();
    const gdn_tree_problem& p = A.p;
    const int lane = threadIdx.x & 31, cta = blockIdx.x, group = cta % A.groups, c = cta / A.groups;
    const int64_t share = share_of(A.before[p.num_seqs] * A.heads, ctas / A.groups, 1), lo = c * share;
    if (c == 0 || lo >= A.before[p.num_seqs] * A.heads) return;
    int n = 0, end = p.num_seqs;  // the last sequence that begins at or before lo: 32 candidates a round
    while (end - n > 1) {
        const int step = (end - n + 31) / 32, x = n + lane * step;
        const uint32_t votes = __ballot_sync(0xffffffffu, x < end && A.before[x] * A.heads <= lo);
        n += (31 - __clz(votes)) * step;
        end = min(end, n + step);
    }
    const int64_t before = A.before[n], tiles = A.before[n + 1] - before, rest = lo - before * A.heads;
    const int head = int(quotient(rest, tiles));
    const int64_t at0 = before * A.heads + head * tiles, at1 = at0 + tiles;
    const int c0 = int(quotient(at0, share)), c1 = int(quotient(at1 - 1, share));
    const int G = p.Hq / p.Hkv, all_rows = p.T * G, nb = (all_rows + rows - 1) / rows, block = head * A.groups + group, hk = block / nb;
    if (at0 == lo || c0 != c - 1) return;  // begins here, or joined at an earlier border
    const int parts = c1 - c0 + 1;
#pragma unroll 1
    for (int in = blockIdx.y * 8 + (threadIdx.x >> 5); in < rows; in += gridDim.y * 8) {
        const int r = (block - hk * nb) * rows + in, t = r / G;
        if (r >= all_rows) return;
        const int64_t row = (int64_t(n) * p.T + t) * p.Hq + hk * G + (r - t * G);
        float M = -INFINITY, S = 0.f, acc[E] = {};
        for (int i0 = 0; i0 < parts; i0 += NB) {  // batches of parts, everything of a batch requested at once
            float2 ml[NB];
            float x[NB][E];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int i = i0 + b;
                ml[b] = make_float2(-INFINITY, 0.f);
                if (i < parts) {
                    const int64_t at = place_of((c0 + i) * A.groups + group, i > 0, rows) + in;
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
                if (ml[b].x == -INFINITY && ml[b].y == 0.f) continue;  // that part has none of this row's keys
                const float w = ml[b].x == -INFINITY ? 1.f : ex2(ml[b].x - M);
                S = fmaf(ml[b].y, w, S);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(x[b][e], w, acc[e]);
            }
        }
        const bool some = S > 0.f || S != S;
        const float f = some ? 1.f / S : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) static_cast<Act*>(A.o)[row * D + 32 * e + lane] = from_f<Act>(acc[e] * f);
        if (A.lse && lane == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
    }
}

template <typename Act, int D>
cudaError_t launch_tree_join(const TreeArgs& A, const TreePlan& plan, cudaStream_t st) {
    const int rows = A.p.T * (A.p.Hq / A.p.Hkv) < plan.rows ? A.p.T * (A.p.Hq / A.p.Hkv) : plan.rows;
    // Up to 64 rows each warp has one; above, four in turn, for most CTAs find no work: 248 rows to a kv-head 37 and 26 us.
    const int blocks = rows <= 64 ? (rows + 7) / 8 : (rows + 31) / 32;
    timing_begin("tree_attn_join", st);
    const cudaError_t e = launch_pdl(k_tree_join<Act, D>, dim3(unsigned(plan.ctas), unsigned(blocks)), dim3(256), 0, st, A, plan.rows, plan.ctas);
    timing_end(st);
    return e;
}

}  // namespace
}  // namespace gdn
