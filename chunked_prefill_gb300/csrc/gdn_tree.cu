// Attention of a tree of drafted tokens over a paged key-value cache (include/gdn.h, gdn_paged_attn_tree).
//
// The drafted tokens of a sequence read the same cache: the rows (drafted token, query head) that share a
// kv-head go through it together, in blocks of rows.  As in gdn_paged_attn_decode the blocks are dealt to
// groups, a group's work is a list of tiles -- sequence by sequence, block by block, the cached tokens'
// tiles and one of the drafted tokens -- and the grid fills the GPU once, every CTA with an equal, contiguous
// part of its group's list.  A block that lies in one CTA's part is written out by it; of others every CTA
// leaves (accumulator, maximum, sum), and a second kernel joins them in the list's order.
// v_scale goes into the weights of the cached tokens, so that drafted ones join them as they are.
//
// bf16 and 8-bit caches: k_tree_tc (gdn_tree_tc.cuh), on the tensor cores.  fp32: k_tree_simt, here; bound by its products' 4 x 4
// values a thread, whose loads nothing overlaps: 32 sequences, 400 MB of keys and values, 32 / 8 heads, 8 drafted tokens 0.84, 1.35
// and 1.38 ms with 64, 128 and 256 features, 4 to 7 % of HBM's rate, whatever the page size; 64 drafted tokens 3.9, 6.5, 6.5 ms.
#include "gdn_attn_simt.cuh"
#include "gdn_tree.cuh"

namespace gdn {
namespace {

// ---- on the CUDA cores: 64 rows, tiles of 64 tokens
constexpr int TB = 64;
template <int D> constexpr int tree_smem() { return (3 * TB * (D + 4) + TB * (TB + 4)) * 4; }

template <int D>
__global__ void __launch_bounds__(ST) k_tree_simt(const TreeArgs A) {
    constexpr int MI = TB / 16;
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + TB * (D + 4), *V = K + TB * (D + 4), *P = V + TB * (D + 4);
    __shared__ Tree tree;
    __shared__ int page_s[TB];
    tc::pdl_launch_dependents();
    const gdn_tree_problem& p = A.p;
    const int G = p.Hq / p.Hkv, all_rows = p.T * G, nb = (all_rows + TB - 1) / TB, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    Part W = find_part<ST>(A, TB, 1);
    for (int64_t pos = W.lo; pos < W.hi;) {
        const int n = W.n, block = W.head * A.groups + W.group, hk = block / nb, r0 = (block % nb) * TB;
        const TreeRange R = range_of(A, n);
        const int tiles = R.tiles(TB), begin = W.at, end = int(min(int64_t(tiles), W.at + (W.hi - pos)));
        const bool whole = begin == 0 && end == tiles, began = begin > 0;
        pos += end - begin;
        W.at = 0;
        if (++W.head == A.heads) W.head = 0, ++W.n;
        const float ks = A.k_scale ? A.k_scale[hk] : 1.f, vs = A.v_scale ? A.v_scale[hk] : 1.f;
        read_tree(A, n, tree);
        for (int i = tid; i < TB * (D / 4); i += ST) {
            const int r = i / (D / 4), d = i % (D / 4) * 4, t = (r0 + r) / G, g = (r0 + r) % G;
            *reinterpret_cast<float4*>(Q + r * (D + 4) + d) =
                r0 + r < all_rows ? ld4(static_cast<const float*>(A.q) + (int64_t(n) * p.T + t) * p.q_stride + int64_t(hk * G + g) * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        float acc[MI][D / 16] = {}, m[MI], l[MI] = {};
        int first[MI];  // of the cached tokens; R.len where there are none
        uint64_t sees[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = r0 + ty + 16 * i, t = min(r / G, 63), depth = r < all_rows ? tree.depth[t] : -1;
            m[i] = -INFINITY;
            first[i] = depth < 0 ? R.len : first_cached(A, R, depth);
            sees[i] = depth < 0 ? 0 : tree.sees[t];
        }
        for (int tile = begin; tile < end; ++tile) {
            __syncthreads();
            const bool drafted = tile == tiles - 1;
            const int t0 = R.base + tile * TB;
            if (drafted) {
                load_rows<TB, D>(K, static_cast<const float*>(A.k_new) + int64_t(n) * p.T * p.k_new_stride + int64_t(hk) * D, p.k_new_stride, p.T);
                load_rows<TB, D>(V, static_cast<const float*>(A.v_new) + int64_t(n) * p.T * p.v_new_stride + int64_t(hk) * D, p.v_new_stride, p.T);
            } else {
                if (tid < TB) {
                    const int t = t0 + tid, page = t < R.len ? A.table[n * p.table_stride + A.page_div.of(t)] : -1;
                    page_s[tid] = page >= 0 && page < p.num_pages ? page : -1;
                }
                __syncthreads();
#pragma unroll 2
                for (int i = tid; i < TB * (D / 4); i += ST) {
                    const int r = i / (D / 4), d = i % (D / 4) * 4, page = page_s[r], t = t0 + r;
                    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
                    if (page >= 0) {
                        const int in = t - A.page_div.of(t) * p.page_size;
                        k = ld4(static_cast<const float*>(A.k_cache) + page * p.k_page_stride + in * p.k_token_stride + hk * p.k_head_stride + d);
                        v = ld4(static_cast<const float*>(A.v_cache) + page * p.v_page_stride + in * p.v_token_stride + hk * p.v_head_stride + d);
                    }
                    *reinterpret_cast<float4*>(K + r * (D + 4) + d) = k;
                    *reinterpret_cast<float4*>(V + r * (D + 4) + d) = v;
                }
            }
            __syncthreads();
            float z[MI][MI];
            mul_nt<MI, MI, D>(z, Q, K);
            const float zs = p.scale * (drafted ? 1.f : ks) * LOG2E;
            auto counts = [&](int i, int x) {
                if (drafted) return (sees[i] >> x & 1) != 0;
                return t0 + x >= first[i] && t0 + x < R.len && page_s[x] >= 0;
            };
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int x = 0; x < MI; ++x) z[i][x] = counts(i, tx + 16 * x) ? z[i][x] * zs : -INFINITY;
            softmax_step(z, m, l, acc, P);
            __syncthreads();
            if (!drafted) {
                for (int i = tid; i < TB * TB; i += ST) P[(i / TB) * (TB + 4) + i % TB] *= vs;
                __syncthreads();
            }
            mul_add<MI, D, false, true>(acc, TB, P, TB + 4, V, counts);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const float sum = row_sum(l[i]);
            const int r = r0 + ty + 16 * i;
            if (r >= all_rows) continue;
            if (whole) {
                const bool some = sum > 0.f || sum != sum;
                const float f = some ? 1.f / sum : 0.f;
                const int64_t at = (int64_t(n) * p.T + r / G) * p.Hq + hk * G + r % G;
#pragma unroll
                for (int v = 0; v < D / 64; ++v)
                    st4(static_cast<float*>(A.o) + at * D + 64 * v + 4 * tx, acc[i][4 * v] * f, acc[i][4 * v + 1] * f, acc[i][4 * v + 2] * f, acc[i][4 * v + 3] * f);
                if (A.lse && tx == 0) A.lse[at] = some ? (m[i] + log2f(sum)) * LN2 : -INFINITY;
            } else {
                const int64_t at = place_of(blockIdx.x, began, TB) + ty + 16 * i;
#pragma unroll
                for (int v = 0; v < D / 64; ++v) st4(A.part + at * D + 64 * v + 4 * tx, acc[i][4 * v], acc[i][4 * v + 1], acc[i][4 * v + 2], acc[i][4 * v + 3]);
                if (tx == 0) A.part_ml[at] = make_float2(m[i], sum);
            }
        }
        __syncthreads();
    }
}

template <int D>
cudaError_t simt(const TreeArgs& A, const TreePlan& plan, cudaStream_t st) {
    cudaError_t e = smem_attr(k_tree_simt<D>, tree_smem<D>());
    if (e != cudaSuccess) return e;
    timing_begin("tree_attn", st);
    k_tree_simt<D><<<plan.ctas, ST, tree_smem<D>(), st>>>(A);
    timing_end(st);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_tree_join<float, D>(A, plan, st);
}

TreeShape shape_of(const gdn_tree_problem& p) {
    if (p.dtype == GDN_FP32) return {TB, TB, p.D == 64 ? 2 : 1};
    return {p.D <= 128 && p.T * (p.Hq / p.Hkv) > 128 ? 256 : 128, p.D == 256 ? 64 : 128, 1};
}

}  // namespace

TreePlan tree_plan(const gdn_tree_problem& p) {
    const TreeShape s = shape_of(p);
    TreePlan r;
    r.rows = s.rows;
    r.tok = s.tok;
    const int blocks = p.Hkv * ((p.T * (p.Hq / p.Hkv) + s.rows - 1) / s.rows), full = s.ctas * sm_count_cached();
    // groups and CTAs as in paged_plan
    r.groups = 1;
    for (int g = 1; g <= blocks && g <= full; ++g)
        if (blocks % g == 0 && (full / g * g >= full / r.groups * r.groups || full / g * g * 50 >= full * 49)) r.groups = g;
    r.heads = blocks / r.groups;
    const int64_t cap = int64_t(p.max_pages) * p.page_size, most = p.window > 0 && p.window < cap - 16 ? p.window + 16 : cap;
    const int64_t tiles = ((most + s.tok - 1) / s.tok + 1) * r.heads * p.num_seqs;
    const int parts = full / r.groups;
    r.ctas = r.groups * int(tiles < parts ? tiles : parts);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    r.off_ml = up(size_t(p.num_seqs + 1) * sizeof(int64_t));
    r.off_part = r.off_ml + up(size_t(r.ctas) * 2 * s.rows * sizeof(float2));
    r.bytes = r.off_part + size_t(r.ctas) * 2 * s.rows * p.D * sizeof(float);
    return r;
}

cudaError_t launch_tree(const TreeArgs& A, cudaStream_t st) {
    const TreePlan plan = tree_plan(A.p);
    if (A.p.dtype == GDN_BF16) return A.p.cache_dtype == GDN_BF16 ? launch_tree_bf16(A, plan, st) : launch_tree_f8(A, plan, st);
    return A.p.D == 64 ? simt<64>(A, plan, st) : A.p.D == 128 ? simt<128>(A, plan, st) : simt<256>(A, plan, st);
}

}  // namespace gdn
