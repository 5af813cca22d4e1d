// Attention of one new token per sequence over a paged key-value cache (include/gdn.h,
// gdn_paged_attn_decode): o_h = sum_t softmax(scale <q_h, k_t>)_t v_t, lse_h = log sum_t e^{z_t}.
//
// Long caches.  The blocks of up to 16 query heads that share a kv-head are dealt to `groups` groups
// (block b to group b % groups).  A group's work is a list of tiles of tokens: sequence by sequence,
// its blocks of heads one after another, tile by tile.  The grid fills the GPU once, with the same
// number of CTAs to each group, each taking an equal, contiguous part of its group's list, so that
// uneven lengths neither leave a tail nor ask the host for the lengths.  On each (sequence, block of
// heads) in its part a CTA keeps a running maximum m, sum l of e^{z - m} and accumulator of e^{z - m} v:
// one pass over keys and values.  A pair that lies in one CTA's part is written out by it; of others
// every CTA leaves (accumulator, m, l) -- at most two per CTA, its first pair's and its last one's --
// and a second kernel joins them in the list's order.
// Short caches.  A cluster of 1 to 8 CTAs, or a CTA of one warp where there are very many, has each
// (sequence, block of heads); a cluster joins its parts through distributed shared memory.
// Bound: HBM, 2 D bytes-per-value per token and kv-head.
//
// bf16 and 8-bit caches: k_paged_mma.  A warp takes tiles of 16 (or 32) tokens through shared memory of
// its own, STAGES tiles deep (cp.async, whole rows by consecutive lanes), so that the loop has no barrier
// of the CTA, whatever the page size.  Both products run on m16n8k16 tensor-core fragments, the block's
// query heads being the 16 rows: S = Q K^T, and O = P V with P as S's accumulator lies.  Rows are kept
// with their 16-byte pieces exchanged (piece ^ row % 8), which makes the copies and the fragments' reads
// (ldmatrix; transposed for V) free of bank conflicts.  With 16 query rows a tcgen05 tile would be mostly
// padding, and the time goes into loading: the first layout here, in which a thread copied the very pieces
// its fragments need (a warp's lanes spread over 4 to 8 rows), ended at 68 % of the copy bandwidth with the
// arithmetic taken out.
// 8-bit caches: S is a product of 8-bit operands, each query value the sum of two; values are converted to
// fp16 (exactly; ldmatrix hands out pairs of bytes, so a value row's bytes are read as 16-byte pieces of 4
// tokens and paired by byte permutes).  The weights are rounded to bf16 (fp16 for 8-bit caches) for the second
// product, 2^-9 (2^-12) of each on average, while their sum l adds them unrounded in fp32.
//
// fp32: k_paged_fp32 (gdn_paged_fp32.cu), on the CUDA cores.
//
// Measured (of the copy bandwidth measured on the same GPUs): 64 sequences of up to 8192 tokens, 32 / 8 heads,
// 128 features, bf16, 162 us (6.7 TB/s, 1.00); 128 of up to 16384, 64 / 8, 8 bits, 322 us (6.6 TB/s, 0.98); one
// of 131071, 32 / 4, bf16, 46.7 us (5.7 TB/s, 0.86: finding the parts and the join take 5 us); 4 of up to 700,
// 16 / 2, 256 features, the new token written, 9.1 us (latency).
#include "gdn_paged.cuh"

namespace gdn {
namespace {

constexpr int CLUSTER_WORK = 4096;  // features times tokens per warp that are not worth splitting

PagedShape shape_of(const gdn_paged_problem& p) {
    if (p.dtype == GDN_FP32) return paged_shape_fp32(p.D, p.Hq / p.Hkv);
    return p.cache_dtype == GDN_BF16 ? paged_shape_bf16(p.D) : paged_shape_f8(p.D);
}

}  // namespace

PagedPlan paged_plan(const gdn_paged_problem& p) {
    const PagedShape s = shape_of(p);
    const int G = p.Hq / p.Hkv;
    PagedPlan r;
    r.rows = s.rows;
    const int blocks = p.Hkv * ((G + s.rows - 1) / s.rows);
    // Groups of heads: with as many as there are blocks of heads, CTAs next to one another read the same
    // tokens for different heads at about the same time (a token's heads lie side by side in a page);
    // fewer where the CTAs could not be dealt out evenly otherwise.
    const int full = s.ctas * sm_count_cached();
    r.groups = 1;
    for (int g = 1; g <= blocks && g <= full; ++g)
        if (blocks % g == 0 && (full / g * g >= full / r.groups * r.groups || full / g * g * 50 >= full * 49)) r.groups = g;
    r.heads = blocks / r.groups;
    // no more CTAs than the problem can have shares of one tile per warp
    const int64_t cap = int64_t(p.max_pages) * p.page_size, most = p.window > 0 && p.window < cap - 16 ? p.window + 16 : cap;
    const int64_t tiles = (most / s.tok + 1) * r.heads * p.num_seqs, want = (tiles + s.warps - 1) / s.warps;
    const int parts = full / r.groups;
    r.ctas = r.groups * int(want < parts ? (want > 0 ? want : 1) : parts);
    // Short caches take no list: a cluster of 1 to 8 CTAs has each (sequence, kv-head) and joins it through
    // distributed shared memory.  Finding a CTA's part of the list and the second kernel take 4 to 5 us, the
    // time of some 16384 / D tokens per warp; a cluster's warps have at most longest / c tokens, in an even
    // split longest * pairs / full.  Enough CTAs even themselves out, so that the list is worth its while from
    // 512 tokens per warp on.  So do clusters that reach every multiprocessor, one CTA on each loading about as
    // much as the memory gives (24 sequences of up to 2000 tokens, 8 kv-heads, 128 features, even lengths and
    // random ones: bf16 33 and 23 us, the list 40 and 28; 8 bits 25 and 21, the list 31 and 28).
    const int64_t pairs = int64_t(p.num_seqs) * blocks, longest = (most + s.warps - 1) / s.warps;
    int c = 1;
    while (c < 8 && pairs * c * 2 <= full && longest * p.D > int64_t(c) * CLUSTER_WORK) c *= 2;
    const bool brief = pairs >= full ? longest <= 512
                                     : (longest / c - longest * pairs / full) * p.D <= 16384 ||
                                           (p.dtype != GDN_FP32 && pairs * c >= sm_count_cached() && longest / c * (p.D > 128 ? p.D : 128) <= 65536);
    r.cluster = brief && pairs * c < (1 << 30) ? c : 0;
    if (r.cluster) r.ctas = int(pairs * c);
    // More short ones than CTAs at a time: CTAs of one warp, of which 8 to 12 fit a multiprocessor, as long as there
    // are so many that their warps alone keep it loading: 64 of them to a token and byte of a key's row, by the times
    // of 320 to 2000 pairs of up to 32 to 2000 tokens (2000 pairs, 128 bf16 features, CTAs of one warp and of four:
    // up to 32 tokens 10 and 19 us, 128 19 and 28, 256 32 and 35, 512 57 and 50; 512 pairs: 5.4 and 6.9, 8.9 and 8.1,
    // 14 and 10, 31 and 17).
    const int64_t row = int64_t(p.D) * (p.cache_dtype == GDN_E4M3 ? 1 : 2);
    r.solo = p.dtype != GDN_FP32 && r.cluster == 1 && pairs > full && most * (row < 256 ? row : 256) <= 64 * pairs;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    r.off_ml = up(size_t(p.num_seqs + 1) * sizeof(int64_t));
    r.off_part = r.off_ml + up(size_t(r.ctas) * 2 * s.rows * sizeof(float2));
    r.bytes = r.off_part + size_t(r.ctas) * 2 * s.rows * p.D * sizeof(float);
    if (r.cluster) r.off_ml = r.off_part = r.bytes = 0;
    return r;
}

cudaError_t launch_paged(const PagedArgs& A, cudaStream_t st) {
    const PagedPlan plan = paged_plan(A.p);
    if (A.p.dtype == GDN_FP32) return launch_paged_fp32(A, plan, st);
    return A.p.cache_dtype == GDN_BF16 ? launch_paged_bf16(A, plan, st) : launch_paged_f8(A, plan, st);
}

}  // namespace gdn
