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
// fp32: k_paged, on the CUDA cores.
//
// Measured (of the copy bandwidth measured on the same GPUs): 64 sequences of up to 8192 tokens, 32 / 8 heads,
// 128 features, bf16, 162 us (6.7 TB/s, 1.00); 128 of up to 16384, 64 / 8, 8 bits, 316 us (6.7 TB/s, 1.00); one
// of 131071, 32 / 4, bf16, 47.5 us (5.7 TB/s, 0.84: finding the parts and the join take 6 us); 4 of up to 700,
// 16 / 2, 256 features, the new token written, 9.2 us (latency).
#include "gdn_paged.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------------------- fp32
constexpr int PT = 128;   // threads
constexpr int PW = PT / 32;
constexpr int GB = 4;     // query heads per block of heads
constexpr int PU = 4;     // tokens a warp takes at a time
constexpr int PTOK = 32;  // tokens to a tile of the list

template <int E>
__device__ __forceinline__ void load_row(const float* p, float (&x)[E]) {
    if constexpr (E == 2) {
        *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(p);
    } else {
#pragma unroll
        for (int b = 0; b < E / 4; ++b) *reinterpret_cast<float4*>(x + 4 * b) = *reinterpret_cast<const float4*>(p + 4 * b);
    }
}
// 16 values a lane, summed over the warp: lane l gets value l / 2 (bit 4 of the lane is bit 3 of the value).
__device__ __forceinline__ float sum16(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 8; n > 0; n >>= 1) {
        const bool up = lane & (2 * n);
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * n);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// A warp takes 4 tokens at a time, a lane D / 32 features of their rows and of 4 query heads.  The 16
// scores are summed across the warp so that each ends up in two lanes (16 exchanges instead of 80), which
// alone work out its weight; the next 4 tokens' rows are requested meanwhile.
template <int D>
__global__ void __launch_bounds__(PT, D == 256 ? 2 : 4) k_paged(const PagedArgs A) {
    constexpr int E = D / 32;
    __shared__ __align__(16) float acc_s[PW][GB][D], res_s[GB][D];
    __shared__ float ml_s[PW][GB][2];
    __shared__ float2 res_ml[GB];
    const gdn_paged_problem& p = A.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.Hq / p.Hkv, nb = (G + GB - 1) / GB;
    tc::pdl_launch_dependents();
    Part P = find_part<PT>(A, PTOK, 1);
    const Part P0 = P;
    if (A.cluster > 1 && tid < GB) res_ml[tid] = make_float2(-INFINITY, 0.f);
    for (int64_t pos = P.lo; pos < P.hi;) {
        const int n = P.n, block = P.head * A.groups + P.group, hk = block / nb, hb = (block % nb) * GB;
        const Range R = range_of(A, n);
        const int tiles = R.tiles(PTOK), end = int(min(int64_t(tiles), P.at + (P.hi - pos)));
        const bool whole = P.at == 0 && end == tiles, began = P.at > 0;
        const int start = R.base + P.at * PTOK;
        const int t0 = max(R.first, start), t1 = end == tiles ? R.len : R.base + end * PTOK;
        pos += end - P.at;
        P.at = 0;
        if (++P.head == A.heads) P.head = 0, ++P.n;

        const float ks = A.k_scale ? A.k_scale[hk] : 1.f, vs = A.v_scale ? A.v_scale[hk] : 1.f;
        const int32_t* table = A.table + n * p.table_stride;
        float* kc = static_cast<float*>(A.k_cache) + hk * p.k_head_stride;
        float* vc = static_cast<float*>(A.v_cache) + hk * p.v_head_stride;
        if (A.k_new && R.fits && end == tiles) {  // every block of heads writes the same bits before it reads them
            const int at = R.len - 1, page = table[A.page_div.of(at)], slot = at - A.page_div.of(at) * p.page_size;
            if (page >= 0 && page < p.num_pages) {
                const int64_t from = n * p.new_stride + int64_t(hk) * D;
                for (int i = tid; i < D; i += PT) {
                    kc[page * p.k_page_stride + slot * p.k_token_stride + i] = to_cache<float>(static_cast<const float*>(A.k_new)[from + i], ks);
                    vc[page * p.v_page_stride + slot * p.v_token_stride + i] = to_cache<float>(static_cast<const float*>(A.v_new)[from + i], vs);
                }
            }
            __syncthreads();
        }

        // page of token t + lane % 4, or -1 where there is nothing to attend to
        auto page_at = [&](int t) {
            t += lane & (PU - 1);
            if (t < t0 || t >= t1) return -1;
            const int page = table[A.page_div.of(t)];
            return page >= 0 && page < p.num_pages ? page : -1;
        };
        float kn[PU][E], vn[PU][E];
        auto fetch = [&](int t, int pages) {
#pragma unroll
            for (int u = 0; u < PU; ++u) {
                const int page = __shfl_sync(0xffffffffu, pages, u), slot = t + u - A.page_div.of(t + u) * p.page_size;
                if (page >= 0) {
                    load_row<E>(kc + page * p.k_page_stride + slot * p.k_token_stride + lane * E, kn[u]);
                    load_row<E>(vc + page * p.v_page_stride + slot * p.v_token_stride + lane * E, vn[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) kn[u][e] = vn[u][e] = 0.f;
                }
            }
        };
        constexpr int HOP = PW * PU;
        const int first = start + warp * PU;
        int pages = page_at(first);
        fetch(first, pages);
        int next = page_at(first + HOP);

        float q[GB][E], acc[GB][E];
#pragma unroll
        for (int h = 0; h < GB; ++h)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                acc[h][e] = 0.f;
                q[h][e] = hb + h < G ? static_cast<const float*>(A.q)[n * p.q_stride + (hk * G + hb + h) * D + lane * E + e] : 0.f;
            }
        const float zs = p.scale * ks * LOG2E;
        float m = -INFINITY, l = 0.f;  // of this lane's head, bits 1 and 2 of the lane; its token: bits 3 and 4
        for (int t = first; t < t1; t += HOP) {
            const bool live = __shfl_sync(0xffffffffu, pages, lane >> 3) >= 0;
            float k[PU][E], v[PU][E];
#pragma unroll
            for (int u = 0; u < PU; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) k[u][e] = kn[u][e], v[u][e] = vn[u][e];
            pages = next;
            fetch(t + HOP, pages);
            next = page_at(t + 2 * HOP);
            float z16[16];
#pragma unroll
            for (int u = 0; u < PU; ++u)
#pragma unroll
                for (int h = 0; h < GB; ++h) {
                    float z = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) z = fmaf(q[h][e], k[u][e], z);
                    z16[u * GB + h] = z;
                }
            float z = sum16(z16) * zs;
            if (!live) z = -INFINITY;
            float top = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 16));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            if (__any_sync(0xffffffffu, top > m)) {
                const float mn = fmaxf(m, top), c = mn == -INFINITY ? 1.f : exp2f(m - mn);
                m = mn;
                l *= c;
#pragma unroll
                for (int h = 0; h < GB; ++h) {
                    const float ch = __shfl_sync(0xffffffffu, c, 2 * h);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[h][e] *= ch;
                }
            }
            const float w = exp2f(z - (m == -INFINITY ? 0.f : m));
            l += w;
#pragma unroll
            for (int u = 0; u < PU; ++u)
#pragma unroll
                for (int h = 0; h < GB; ++h) {
                    const float wu = __shfl_sync(0xffffffffu, w, 8 * u + 2 * h);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[h][e] = fmaf(wu, v[u][e], acc[h][e]);
                }
        }
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
#pragma unroll
        for (int h = 0; h < GB; ++h)
#pragma unroll
            for (int e = 0; e < E; ++e) acc_s[warp][h][lane * E + e] = acc[h][e];
        if (lane < 8 && (lane & 1) == 0) {
            ml_s[warp][lane >> 1][0] = m;
            ml_s[warp][lane >> 1][1] = l;
        }
        __syncthreads();
        for (int i = tid; i < min(GB, G - hb) * D; i += PT) {
            const int h = i / D, d = i % D;
            float M = -INFINITY, S = 0.f, a = 0.f;
#pragma unroll
            for (int g = 0; g < PW; ++g) M = fmaxf(M, ml_s[g][h][0]);
#pragma unroll
            for (int g = 0; g < PW; ++g) {
                const float c = ml_s[g][h][0] == -INFINITY ? 0.f : exp2f(ml_s[g][h][0] - M);
                S = fmaf(ml_s[g][h][1], c, S);
                a = fmaf(acc_s[g][h][d], c, a);
            }
            if (A.cluster > 1) {
                res_s[h][d] = a;
                if (d == 0) res_ml[h] = make_float2(M, S);
            } else if (whole) {
                const int64_t row = int64_t(n) * p.Hq + hk * G + hb + h;
                const bool some = S > 0.f || S != S;
                static_cast<float*>(A.o)[row * D + d] = some ? a / S * vs : 0.f;
                if (A.lse && d == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
            } else {
                const int64_t at = place_of(blockIdx.x, began, GB) + h;
                A.part[at * D + d] = a;
                if (d == 0) A.part_ml[at] = make_float2(M, S);
            }
        }
        __syncthreads();  // the shared arrays are read before the next pair writes them
    }
    if (A.cluster > 1) {
        const int block = P0.head * A.groups + P0.group, hb = (block % nb) * GB;
        join_cluster<float, D, PT>(A, tc::smem_addr(res_s), tc::smem_addr(res_ml), P0.n, block / nb, hb, min(GB, G - hb));
    }
}

constexpr int CLUSTER_WORK = 4096;  // features times tokens per warp that are not worth splitting

template <int D> constexpr PagedShape fp32_shape() { return {PTOK, GB, 1, D == 256 ? 2 : 4}; }
PagedShape shape_of(const gdn_paged_problem& p) {
    if (p.dtype == GDN_FP32) return p.D == 64 ? fp32_shape<64>() : p.D == 128 ? fp32_shape<128>() : fp32_shape<256>();
    return p.cache_dtype == GDN_BF16 ? paged_shape_bf16(p.D) : paged_shape_f8(p.D);
}

template <int D>
cudaError_t launch_fp32(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    timing_begin("paged_attn", st);
    const cudaError_t e = launch_clusters(k_paged<D>, A, plan.ctas, PT, 0, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
    return launch_join<float, D>(A, plan, fp32_shape<D>(), st);
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
    // 512 tokens per warp on.
    const int64_t pairs = int64_t(p.num_seqs) * blocks, longest = (most + s.warps - 1) / s.warps;
    int c = 1;
    while (c < 8 && pairs * c * 2 <= full && longest * p.D > int64_t(c) * CLUSTER_WORK) c *= 2;
    const bool brief = pairs >= full ? longest <= 512 : (longest / c - longest * pairs / full) * p.D <= 16384;
    r.cluster = brief && pairs * c < (1 << 30) ? c : 0;
    if (r.cluster) r.ctas = int(pairs * c);
    // More short ones than CTAs at a time: CTAs of one warp, 8 to a multiprocessor (195 sequences of one token, 8
    // kv-heads: 13 us instead of 26; 250 of up to 500: 45 instead of 49; of up to 1000: 94 instead of 82).
    r.solo = p.dtype != GDN_FP32 && r.cluster == 1 && pairs > full && most * (p.D > 128 ? p.D : 128) <= 65536;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    r.off_ml = up(size_t(p.num_seqs + 1) * sizeof(int64_t));
    r.off_part = r.off_ml + up(size_t(r.ctas) * 2 * s.rows * sizeof(float2));
    r.bytes = r.off_part + size_t(r.ctas) * 2 * s.rows * p.D * sizeof(float);
    if (r.cluster) r.off_ml = r.off_part = r.bytes = 0;
    return r;
}

cudaError_t launch_paged(const PagedArgs& A, cudaStream_t st) {
    const PagedPlan plan = paged_plan(A.p);
    if (A.p.dtype == GDN_FP32)
        return A.p.D == 64 ? launch_fp32<64>(A, plan, st) : A.p.D == 128 ? launch_fp32<128>(A, plan, st) : launch_fp32<256>(A, plan, st);
    return A.p.cache_dtype == GDN_BF16 ? launch_paged_bf16(A, plan, st) : launch_paged_f8(A, plan, st);
}

}  // namespace gdn
