// What the kernels of attention over prompts share: the sequences and the numbering of their tiles.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_attn.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_paged.cuh"
#include "tc05.cuh"

namespace gdn {
namespace {

// A sequence's rows: queries [q0, q0 + lq), keys [k0, k0 + lk).  rest: no sequence, rows that none covers.
struct Seq {
    int q0, lq, k0, lk;
    bool rest;
};
__device__ __forceinline__ int cut(int x, int lo, int hi) { return x < lo ? lo : x < hi ? x : hi; }

// Tiles of BM rows.  Packed rows are numbered so that a tile's sequence is found by bisection: with the rows
// in front of the first sequence as number 0, the sequences as 1 .. N and the rows behind the last as N + 1,
// those of number m begin at floor(start_m / BM) + m.  That leaves each ceil(rows / BM) numbers at least, and
// floor(total / BM) + N + 2 in all; some stand for no tile.
__host__ __device__ inline int64_t tile_numbers(const gdn_prompt_problem& p, bool keys, int BM) {
    const int64_t total = keys ? p.total_k : p.total_q;
    if (p.cu_seqlens) return total / BM + p.num_seqs + 2;
    return p.num_seqs ? (total / p.num_seqs + BM - 1) / BM * p.num_seqs : 0;
}

// The sequence of tile number t and the tile's first row in it; false where it stands for none.  To be called
// by whole warps.
template <int BM>
__device__ __forceinline__ bool find_tile(const gdn_prompt_problem& p, bool keys, int t, Seq& s, int& row) {
    const int N = p.num_seqs;
    if (!p.cu_seqlens) {
        const int lq = p.total_q / N, lk = p.total_k / N, per = ((keys ? lk : lq) + BM - 1) / BM, n = t / per;
        s = {n * lq, lq, n * lk, lk, false};
        row = (t - n * per) * BM;
        return true;
    }
    const int32_t *cq = p.cu_seqlens, *ck = p.cu_seqlens_k ? p.cu_seqlens_k : cq, *cu = keys ? ck : cq;
    const int total = keys ? p.total_k : p.total_q, lane = threadIdx.x & 31;
    auto start = [&](int m) { return m == 0 ? 0 : cut(cu[m - 1], 0, total); };
    int lo = 0, hi = N + 2;  // the last number that begins at or before t: 32 candidates a round
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, m = lo + lane * step;
        const bool le = m < hi && start(m) / BM + m <= t;
        const uint32_t votes = __ballot_sync(0xffffffffu, le);
        const int last = votes ? 31 - __clz(votes) : 0;
        lo += last * step;
        hi = min(hi, lo + step);
    }
    const int from = start(lo), to = lo <= N ? cut(cu[lo], from, total) : total;
    row = (t - (from / BM + lo)) * BM;
    if (row < 0 || row >= to - from) return false;
    s.rest = lo == 0 || lo == N + 1;
    if (s.rest) {
        s.q0 = s.k0 = from;
        s.lq = keys ? 0 : to - from;
        s.lk = keys ? to - from : 0;
        return p.clear_rest != 0;
    }
    s.q0 = cut(cq[lo - 1], 0, p.total_q);
    s.lq = cut(cq[lo], s.q0, p.total_q) - s.q0;
    s.k0 = cut(ck[lo - 1], 0, p.total_k);
    s.lk = cut(ck[lo], s.k0, p.total_k) - s.k0;
    return true;
}

// Query i (of its sequence) attends to keys [first_key, last_key]; none where last_key < first_key.
__device__ __forceinline__ int last_key(const Seq& s, int i) { return i + s.lk - s.lq; }
__device__ __forceinline__ int first_key(const gdn_prompt_problem& p, const Seq& s, int i) {
    const int64_t f = int64_t(last_key(s, i)) - p.window + 1;
    return p.window > 0 && f > 0 ? int(f) : 0;
}
// Key t is attended to by queries [first_query, last_query].
__device__ __forceinline__ int first_query(const Seq& s, int t) { return max(0, t - (s.lk - s.lq)); }
__device__ __forceinline__ int last_query(const gdn_prompt_problem& p, const Seq& s, int t) {
    const int64_t l = int64_t(t) - (s.lk - s.lq) + p.window - 1;
    return p.window > 0 && l < s.lq - 1 ? int(l) : s.lq - 1;
}

}  // namespace
}  // namespace gdn
