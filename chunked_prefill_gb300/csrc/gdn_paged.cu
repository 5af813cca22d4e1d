// Attention of one new token per sequence over a paged key-value cache (include/gdn.h,
// gdn_paged_attn_decode): o_h = sum_t softmax(scale <q_h, k_t>)_t v_t, lse_h = log sum_t e^{z_t}.
//
// The blocks of up to 16 query heads that share a kv-head are dealt to `groups` groups (block b to group
// b % groups).  A group's work is a list of tiles of tokens: sequence by sequence, its blocks of heads one
// after another, tile by tile.  The grid fills the GPU once, with the same number of CTAs to each group,
// each taking an equal, contiguous part of its group's list, so that uneven lengths neither leave a tail nor ask the host for the lengths; on each
// (sequence, kv-head) in its part it keeps a running maximum m, sum l of e^{z - m} and accumulator of
// e^{z - m} v: one pass over keys and values.  A pair that lies in one CTA's part is written out by
// it; of others every CTA leaves (accumulator, m, l) -- at most two per CTA, its first pair's and its
// last one's -- and a second kernel joins them in the list's order.  Bound: HBM, 2 D
// bytes-per-value per token and kv-head.
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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_common.cuh"
#include "gdn_decode.h"
#include "gdn_internal.h"
#include "tc05.cuh"

namespace gdn {
namespace {

constexpr float F8_MAX = 448.f;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Sequence n's tokens: those attended to are [first, len); its tiles of `tok` tokens start at base,
// which is first down to a multiple of 16 (a tile's rows then share a page of 16 k tokens).
struct Range {
    int len, first, base;
    __device__ __forceinline__ int tiles(int tok) const {  // one at least: an empty row is written too
        const int64_t n = (int64_t(len) - base + tok - 1) / tok;
        return n > 1 ? int(n) : 1;
    }
};
__device__ __forceinline__ Range range_of(const PagedArgs& A, int n) {
    const int64_t cap = int64_t(A.p.max_pages) * A.p.page_size;
    Range R;
    const int64_t len = A.lens[n];
    R.len = int(len < 0 ? 0 : len < cap ? len : cap);
    R.first = A.p.window > 0 && R.len > A.p.window ? R.len - A.p.window : 0;
    R.base = R.first & ~15;
    return R;
}

// A CTA's part [lo, hi) of the list of all tiles, and where it begins: tile `at` of block of heads
// `head` (of the group's A.heads) of sequence n.
struct Part {
    int64_t lo, hi;
    int n, group, head, at;
};
// a / b for a >= 0, b > 0; 64-bit division costs half a microsecond that small problems feel
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}
__device__ __forceinline__ int64_t share_of(int64_t total, int parts, int warps) {
    // a multiple of the warps (a power of two), so that none is left out
    return (quotient(total + parts - 1, parts) + warps - 1) & ~int64_t(warps - 1);
}
// CTA 0 also leaves the number of tiles before each sequence (per block of heads) in A.before.
template <int T>
__device__ Part find_part(const PagedArgs& A, int tok, int warps) {
    if (A.cluster) {  // a cluster of CTAs per (sequence, block of heads), equal parts of its tiles
        const int pair = blockIdx.x / A.cluster, r = blockIdx.x % A.cluster, blocks = A.groups * A.heads, n = pair / blocks, b = pair % blocks;
        const int tiles = range_of(A, n).tiles(tok), share = ((tiles + A.cluster - 1) / A.cluster + warps - 1) / warps * warps;
        const int at = min(r * share, tiles);
        return {0, min(share, tiles - at), n, b % A.groups, b / A.groups, at};
    }
    __shared__ int64_t wsum[T / 32];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 31, N = A.p.num_seqs;
    const int per = (N + T - 1) / T, n0 = min(N, tid * per), n1 = min(N, n0 + per);
    int64_t mine = 0;
    for (int n = n0; n < n1; ++n) mine += range_of(A, n).tiles(tok);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) wsum[tid >> 5] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
        if (w < tid >> 5) upto += wsum[w];
        total += wsum[w];
    }
    int64_t run = upto - mine;
    const int64_t share = share_of(total * A.heads, gridDim.x / A.groups, warps);
    Part P;
    P.lo = blockIdx.x / A.groups * share;
    P.hi = min(P.lo + share, total * A.heads);
    if (blockIdx.x == 0) {
        int64_t r = run;
        for (int n = n0; n < n1; ++n) {
            A.before[n] = r;
            r += range_of(A, n).tiles(tok);
        }
        if (tid == T - 1) A.before[N] = total;
    }
    if (P.lo < P.hi && run * A.heads <= P.lo && P.lo < upto * A.heads) {
        int n = n0, t = range_of(A, n).tiles(tok);
        while ((run + t) * A.heads <= P.lo) {
            run += t;
            t = range_of(A, ++n).tiles(tok);
        }
        const int64_t rest = P.lo - run * A.heads, head = quotient(rest, t);
        found[0] = n;
        found[1] = int(head);
        found[2] = int(rest - head * t);
    }
    __syncthreads();
    P.n = found[0], P.group = blockIdx.x % A.groups, P.head = found[1], P.at = found[2];
    return P;
}
// Where a CTA leaves rows [0, ROWS) of a pair that it has a part of: in its first place where the
// pair began before its part, in its second where the pair goes on after it.
__device__ __forceinline__ int64_t place_of(int cta, bool first, int rows) { return (int64_t(cta) * 2 + (first ? 0 : 1)) * rows; }

// ---- clusters: the join through distributed shared memory
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Joins the cluster's CTAs' results -- rows of D at `res`, (max, sum) pairs at `ml`, at the same places of
// every CTA's shared memory -- in rank order, each CTA a slice of the values, and writes them out.
template <typename Act, int D, int T>
__device__ void join_cluster(const PagedArgs& A, uint32_t res, uint32_t ml, int n, int hk, int hb, int rows) {
    const gdn_paged_problem& p = A.p;
    const int r = blockIdx.x % A.cluster, total = rows * (D / 4), each = (total + A.cluster - 1) / A.cluster;
    const float vs = A.v_scale ? A.v_scale[hk] : 1.f;
    cluster_sync();
    for (int i = r * each + threadIdx.x; i < min(total, (r + 1) * each); i += T) {
        const int h = i / (D / 4), d = i % (D / 4) * 4;
        float2 m[8];
        float4 x[8];
        float M = -INFINITY;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (c >= A.cluster) continue;
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];\n" : "=f"(m[c].x), "=f"(m[c].y) : "r"(in_cta(ml + h * 8, c)) : "memory");
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                         : "=f"(x[c].x), "=f"(x[c].y), "=f"(x[c].z), "=f"(x[c].w)
                         : "r"(in_cta(res + (h * D + d) * 4, c))
                         : "memory");
            M = fmaxf(M, m[c].x);
        }
        float S = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (c >= A.cluster || m[c].y == 0.f) continue;  // an empty part has no rows
            const float w = m[c].x == -INFINITY ? 0.f : exp2f(m[c].x - M);
            S = fmaf(m[c].y, w, S);
            a.x = fmaf(x[c].x, w, a.x);
            a.y = fmaf(x[c].y, w, a.y);
            a.z = fmaf(x[c].z, w, a.z);
            a.w = fmaf(x[c].w, w, a.w);
        }
        const int64_t row = int64_t(n) * p.Hq + hk * (p.Hq / p.Hkv) + hb + h;
        const bool some = S > 0.f || S != S;
        const float f = some ? vs / S : 0.f;
        Act* o = static_cast<Act*>(A.o) + row * D + d;
        st2(o, a.x * f, a.y * f);
        st2(o + 2, a.z * f, a.w * f);
        if (A.lse && d == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
    }
    cluster_sync();  // the others have read this CTA's results
}

// a value of the new token's row in the cache's type
template <typename C> __device__ __forceinline__ C to_cache(float x, float scale);
template <> __device__ __forceinline__ float to_cache<float>(float x, float scale) { return x / scale; }
template <> __device__ __forceinline__ __nv_bfloat16 to_cache<__nv_bfloat16>(float x, float scale) {
    return __float2bfloat16_rn(x / scale);
}
template <> __device__ __forceinline__ __nv_fp8_e4m3 to_cache<__nv_fp8_e4m3>(float x, float scale) {
    const float y = x / scale;
    return __nv_fp8_e4m3(y != y ? y : fminf(fmaxf(y, -F8_MAX), F8_MAX));
}

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
        if (A.k_new && R.len > 0 && end == tiles) {  // every block of heads writes the same bits before it reads them
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

// ---------------------------------------------------------------- bf16 and 8-bit caches
// 2^x to 2^-22 of itself; -inf gives 0
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename C> struct Frag;
template <> struct Frag<__nv_bfloat16> {
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return tc::pack_bf16(lo, hi); }
};
template <> struct Frag<__nv_fp8_e4m3> {
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
// four 8-bit values as two pairs of fp16
__device__ __forceinline__ void f8x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
// the product of 8-bit operands over 32 features
__device__ __forceinline__ void mma_f8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// x, y, z, w (magnitudes below 448) as four 8-bit values, and what is left of them in their place
__device__ __forceinline__ uint32_t split_f8(float& x, float& y, float& z, float& w) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(z, w), __NV_SATFINITE, __NV_E4M3);
    uint32_t lo, hi;
    f8x4(a | b << 16, lo, hi);
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo)), q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x -= p.x, y -= p.y, z -= q.x, w -= q.y;
    return a | b << 16;
}

// copy of 16 bytes to shared memory, zeros where !in (the address is not read then)
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

template <typename C, int D> struct Tile {
    static constexpr int E = int(sizeof(C));
    static constexpr int TT = D * E <= 128 ? 2 : 1;                // 16-token blocks of a tile
    static constexpr int TOK = 16 * TT;                            // tokens of a tile
    static constexpr int W = D * E > 256 ? 2 : 4;                  // warps
    static constexpr int T = 32 * W;                               // threads
    static constexpr int CTAS = D == 64 && E == 2 ? 3 : 2;         // per multiprocessor
    static constexpr int ROW = D * E;                              // bytes of a row
    static constexpr int CPR = ROW / 16;                           // 16-byte pieces of a row
    static constexpr int RPI = 32 / CPR;                           // rows per copy instruction of a warp
    static constexpr int VB = ROW / 8 >= 16 ? 16 : ROW / 8;        // 8-bit: bytes of a piece of a value row
    static constexpr int VC = E == 1 ? ROW / (8 * VB) : 0;         // 8-bit: pieces of a value row per thread
    static constexpr int BLOCK = 16 * ROW;                         // bytes of 16 rows
    static constexpr int BYTES = 2 * TT * BLOCK;                   // of a warp's tile: K's blocks, V's blocks
    static constexpr int FIT = (CTAS == 3 ? 65536 : 98304) / (W * BYTES), STAGES = FIT < 8 ? FIT : 8;
    static constexpr int PAD = D + 4;                              // floats between rows of the joined accumulators
    static constexpr int SMEM = STAGES * W * BYTES;
    static_assert(STAGES >= 2 && W * 16 * PAD * 4 + 16 * D * 4 <= SMEM, "the warps' accumulators are joined in the stages' memory");
    // what a row's pieces are exchanged by
    static __host__ __device__ constexpr int swap(int row) { return CPR == 4 ? (row >> 1) & 3 : row & 7; }
};
__device__ __forceinline__ void ldmatrix4(uint32_t from, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(from)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t from, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(from)
                 : "memory");
}

template <typename C, int D, bool HALF, bool TILED>
__global__ void __launch_bounds__(Tile<C, D>::T, Tile<C, D>::CTAS) k_paged_mma(const PagedArgs A) {
    using L = Tile<C, D>;
    constexpr int TT = L::TT, TOK = L::TOK, STAGES = L::STAGES, W = L::W, R2 = HALF ? 1 : 2;
    constexpr int CPR = L::CPR, RPI = L::RPI, ROW = L::ROW, VB = L::VB, VC = L::VC;
    constexpr int VE = VB / L::E;                 // 8-bit: values per piece of a value row
    constexpr int KS = D / 16;                    // k16 steps
    constexpr int QF = KS;                        // entries of the query fragments (2 per step of 32 with 8 bits)
    constexpr bool F8 = L::E == 1;
    // fp16 weights are 2^14 e^{z - m}: those down to 2^-38 of the largest count then (2^-24 without; a long
    // sequence's many small weights add up beside one large one)
    constexpr float LIFT = F8 ? 14.f : 0.f;
    // query fragments in shared memory: of 256 features, the registers hold the accumulators; 8-bit ones are
    // much work to make, shared out to the warps
    constexpr bool QS = D == 256 || F8;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float ml_s[W][16][2];
    __shared__ uint4 q_s[QS ? QF * R2 / 2 : 1][32];
    const gdn_paged_problem& p = A.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.Hkv, nb = (G + 15) / 16;
    const uint32_t mem = tc::smem_addr(smem) + warp * STAGES * L::BYTES;  // this warp's stages
    // copies: row copy_row + RPI j, piece copy_piece; a row's exchange is that of copy_row and that of RPI j
    const int copy_row = lane / CPR, copy_piece = lane % CPR;
    const uint32_t copy_to = mem + copy_row * ROW + ((copy_piece ^ L::swap(copy_row)) << 4);
    // key fragments of 16 tokens: two consecutive pieces of tokens 0-7, then of 8-15
    const int k_row = (lane & 7) + 8 * (lane >> 4);
    const uint32_t k_at = mem + k_row * ROW + (((lane >> 3 & 1) ^ L::swap(k_row)) << 4);
    // value fragments, bf16: piece c of tokens 0-7 and 8-15, then piece c + 1
    const int v_row = (lane & 7) + 8 * (lane >> 3 & 1);
    const uint32_t v_at = mem + TT * L::BLOCK + v_row * ROW + (((lane >> 4) ^ L::swap(v_row)) << 4);
    // 8-bit: this thread's rows of 16 tokens 2t, 2t + 1, 2t + 8, 2t + 9 and its pieces g + 8 c of VB bytes
    auto v8_at = [&](int r, int c) {
        const int row = 2 * t + (r & 1) + 8 * (r >> 1), byte = (g + 8 * c) * VB;
        return mem + TT * L::BLOCK + row * ROW + (((byte >> 4) ^ L::swap(row)) << 4) + (byte & 15);
    };
    auto slot_of = [&](int tok) { return tok - A.page_div.of(tok) * p.page_size; };

    tc::pdl_launch_dependents();
    Part P = find_part<L::T>(A, TOK, W);
    const Part P0 = P;
    float* res = reinterpret_cast<float*>(smem) + W * 16 * L::PAD;  // clusters: this CTA's result
    __shared__ float2 res_ml[16];
    if (A.cluster > 1 && tid < 16) res_ml[tid] = make_float2(-INFINITY, 0.f);
    for (int64_t pos = P.lo; pos < P.hi;) {
        // ---- the next (sequence, block of heads) and this CTA's tiles of it
        const int n = P.n, block = P.head * A.groups + P.group, hk = block / nb, hb = (block % nb) * 16;
        const Range R = range_of(A, n);
        const int tiles_n = R.tiles(TOK), end = int(min(int64_t(tiles_n), P.at + (P.hi - pos)));
        const bool whole = P.at == 0 && end == tiles_n, began = P.at > 0;
        const int start = R.base + P.at * TOK;
        const int t0 = max(R.first, start), t1 = end == tiles_n ? R.len : R.base + end * TOK;
        const int all = end - P.at;
        pos += all;
        P.at = 0;
        if (++P.head == A.heads) P.head = 0, ++P.n;
        const float ks = A.k_scale ? A.k_scale[hk] : 1.f, vs = A.v_scale ? A.v_scale[hk] : 1.f;
        const int32_t* table = A.table + n * p.table_stride;
        C* kc = static_cast<C*>(A.k_cache) + hk * p.k_head_stride;
        C* vc = static_cast<C*>(A.v_cache) + hk * p.v_head_stride;

        // ---- this warp's tiles: tokens from start + TOK (warp + W i)
        const int tiles = all > warp ? (all - warp + W - 1) / W : 0;
        auto token_of = [&](int i) { return start + TOK * (warp + W * i); };
        // The page(s) of block b of tile i: with TILED (a page holds whole blocks) the block's page, in
        // every lane; else lane l has that of token l % 16.  -1 where there is nothing to attend to.
        auto page_at = [&](int i, int b) {
            const int tok = token_of(i) + 16 * b + (TILED ? 0 : lane & 15);
            if (i >= tiles || tok >= t1 || (!TILED && tok < t0)) return -1;
            const int page = table[A.page_div.of(tok)];
            return page >= 0 && page < p.num_pages ? page : -1;
        };
        int first[STAGES - 1][TT];  // of the tiles requested ahead
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i)
#pragma unroll
            for (int b = 0; b < TT; ++b) first[i][b] = page_at(i, b);

        if (A.k_new && R.len > 0 && end == tiles_n) {  // every block of heads writes the same bits before it reads them
            const int at = R.len - 1, page = table[A.page_div.of(at)], slot = slot_of(at);
            if (page >= 0 && page < p.num_pages) {
                C* kd = kc + page * p.k_page_stride + slot * p.k_token_stride;
                C* vd = vc + page * p.v_page_stride + slot * p.v_token_stride;
                const int64_t from = n * p.new_stride + int64_t(hk) * D;
                for (int i = tid; i < D; i += L::T) {
                    kd[i] = to_cache<C>(to_f(static_cast<const __nv_bfloat16*>(A.k_new)[from + i]), ks);
                    vd[i] = to_cache<C>(to_f(static_cast<const __nv_bfloat16*>(A.v_new)[from + i]), vs);
                }
            }
            __syncthreads();
        }

        // Requests the rows of block b of tile i (zeros where masked); returns which tokens count.
        auto issue = [&](int i, int b, int stage, int pages) -> uint32_t {
            const int tok = token_of(i) + 16 * b;
            const uint32_t to = copy_to + stage * L::BYTES + b * L::BLOCK;
            uint32_t valid;
            if constexpr (TILED) {
                valid = 0u;
                if (pages >= 0) {
                    valid = 0xffffu;
                    if (t0 > tok) valid &= 0xffffu << (t0 - tok);
                    if (t1 - tok < 16) valid &= 0xffffu >> (16 - (t1 - tok));
                }
                const int slot = slot_of(tok) + copy_row, page = pages < 0 ? 0 : pages;
                const C* kt = kc + (page * p.k_page_stride + slot * p.k_token_stride) + copy_piece * (16 / L::E);
                const C* vt = vc + (page * p.v_page_stride + slot * p.v_token_stride) + copy_piece * (16 / L::E);
#pragma unroll
                for (int j = 0; j < 16 / RPI; ++j) {
                    const bool in = valid >> (copy_row + RPI * j) & 1;
                    const uint32_t at = (to ^ (L::swap(RPI * j) << 4)) + RPI * j * ROW;
                    cp_async(at, kt, in);
                    cp_async(at + TT * L::BLOCK, vt, in);
                    kt += RPI * p.k_token_stride;
                    vt += RPI * p.v_token_stride;
                }
            } else {
                valid = __ballot_sync(0xffffffffu, pages >= 0) & 0xffffu;
#pragma unroll
                for (int j = 0; j < 16 / RPI; ++j) {
                    const int row = copy_row + RPI * j, page = __shfl_sync(0xffffffffu, pages, row), slot = slot_of(tok + row);
                    const C *kt = kc, *vt = vc;
                    if (page >= 0) {
                        kt += page * p.k_page_stride + slot * p.k_token_stride + copy_piece * (16 / L::E);
                        vt += page * p.v_page_stride + slot * p.v_token_stride + copy_piece * (16 / L::E);
                    }
                    const uint32_t at = (to ^ (L::swap(RPI * j) << 4)) + RPI * j * ROW;
                    cp_async(at, kt, page >= 0);
                    cp_async(at + TT * L::BLOCK, vt, page >= 0);
                }
            }
            return valid << (16 * b);
        };

        uint32_t mask[STAGES];  // which tokens of the tiles in flight count, oldest first
        int pages[TT];
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            mask[i] = 0u;
            if (i < tiles)
#pragma unroll
                for (int b = 0; b < TT; ++b) mask[i] |= issue(i, b, i, first[i][b]);
            cp_commit();
        }
#pragma unroll
        for (int b = 0; b < TT; ++b) pages[b] = page_at(STAGES - 1, b);

        // ---- query fragments, of 16-feature step s: features 2t, + 1 and 8 + 2t, + 1.  8-bit caches, of
        // 32-feature step s: features 4t .. 4t + 3 and 16 + 4t .., each value the sum of two 8-bit ones of
        // the row scaled to [128, 256): exact for bf16's 8 significant bits down to 2^-9 of the row's
        // largest value (4 bits each, the second with a sign of its own), off by 2^-18 of it below.
        alignas(16) uint32_t qf[QF][2 * R2];
        float zs[R2];
#pragma unroll
        for (int r = 0; r < R2; ++r) {
            const int h = hb + g + 8 * r;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(A.q) + n * p.q_stride + int64_t(hk * G + h) * D;
            zs[r] = p.scale * ks * LOG2E;
            if constexpr (F8) {
                uint2 raw[KS];  // features 16 s + 4t .. + 3
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    raw[s] = h < G ? *reinterpret_cast<const uint2*>(q + 16 * s + 4 * t) : make_uint2(0u, 0u);
                    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[s].x));
                    const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[s].y));
                    top = mag_max(top, mag_max(mag_max(fabsf(x.x), fabsf(x.y)), mag_max(fabsf(y.x), fabsf(y.y))));
                }
                top = mag_max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = mag_max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const bool fine = top > 0.f && top < INFINITY;
                const int e = fine ? ilogbf(top) - 7 : 0;
                const float down = fine ? ldexpf(1.f, -e) : 1.f;
                // an infinite or NaN query makes every score NaN (as inf - inf does in the definition)
                const float bad = top < INFINITY ? 0.f : NAN;
                zs[r] = ldexpf(zs[r], e) + bad;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    if (s / 2 % W != warp) continue;
                    float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[s].x));
                    float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[s].y));
                    x.x *= down, x.y *= down, y.x *= down, y.y *= down;
                    // step s / 2, features 0-15 or 16-31 of it; HALF: rows 0-7 the first, 8-15 the second values
                    const uint32_t first = split_f8(x.x, x.y, y.x, y.y), second = split_f8(x.x, x.y, y.x, y.y);
                    qf[HALF ? s / 2 * 2 + s % 2 : s / 2 * 2][HALF ? 0 : (s % 2) * 2 + r] = first;
                    qf[HALF ? s / 2 * 2 + s % 2 : s / 2 * 2 + 1][HALF ? 1 : (s % 2) * 2 + r] = second;
                }
            } else {
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qf[s][r] = h < G ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * t) : 0u;
                    qf[s][R2 + r] = h < G ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 8 + 2 * t) : 0u;
                }
            }
        }
        if constexpr (QS) {
#pragma unroll
            for (int i = 0; i < QF * R2 / 2; ++i)
                if (F8 ? i / R2 % W == warp : warp == 0) q_s[i][lane] = reinterpret_cast<const uint4*>(&qf[0][0])[i];
            __syncthreads();
        }

        float acc[D / 8][4], m[R2], l[R2];  // with HALF the upper two of a quad are the empty rows
#pragma unroll
        for (int r = 0; r < R2; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        auto mma = [&](float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
            if constexpr (HALF) {
                const uint32_t af[4] = {a[0], 0u, a[1], 0u};
                Frag<C>::mma(c, af, b0, b1);
            } else {
                const uint32_t af[4] = {a[0], a[1], a[2], a[3]};
                Frag<C>::mma(c, af, b0, b1);
            }
        };

        int stage = 0;
        for (int i = 0; i < tiles; ++i) {
            cp_wait<STAGES - 2>();
            __syncwarp();  // every lane's copies of tile i have landed, and tile i - 1 has been read
            {
                const int next = i + STAGES - 1;
                mask[STAGES - 1] = 0u;
                if (next < tiles)
#pragma unroll
                    for (int b = 0; b < TT; ++b) mask[STAGES - 1] |= issue(next, b, stage == 0 ? STAGES - 1 : stage - 1, pages[b]);
                cp_commit();
#pragma unroll
                for (int b = 0; b < TT; ++b) pages[b] = page_at(next + 1, b);
            }
            const uint32_t kd = k_at + stage * L::BYTES;
            float s[2 * TT][4] = {};  // of 8 tokens each
#pragma unroll
            for (int c = 0; c < KS / 2; ++c) {  // 32 features
                alignas(16) uint32_t qc[2][2 * R2];
                if constexpr (QS) {
#pragma unroll
                    for (int i = 0; i < R2; ++i) reinterpret_cast<uint4*>(&qc[0][0])[i] = q_s[c * R2 + i][lane];
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2 * R2; ++e) qc[i][e] = qf[2 * c + i][e];
                }
#pragma unroll
                for (int b = 0; b < TT; ++b) {
                    uint32_t k[4];
                    if constexpr (F8) {  // both pieces of tokens 0-7, then of 8-15
                        ldmatrix4((kd ^ (c << 5)) + b * L::BLOCK, k);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if constexpr (HALF) {
                                mma_f8(s[2 * b + u], qc[0][0], qc[0][1], qc[1][0], qc[1][1], k[2 * u], k[2 * u + 1]);
                            } else {
                                mma_f8(s[2 * b + u], qc[0][0], qc[0][1], qc[0][2], qc[0][3], k[2 * u], k[2 * u + 1]);
                                mma_f8(s[2 * b + u], qc[1][0], qc[1][1], qc[1][2], qc[1][3], k[2 * u], k[2 * u + 1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            ldmatrix4((kd ^ ((2 * c + u) << 5)) + b * L::BLOCK, k);
                            mma(s[2 * b], qc[u], k[0], k[1]);
                            mma(s[2 * b + 1], qc[u], k[2], k[3]);
                        }
                    }
                }
            }
            if constexpr (F8 && HALF) {  // the two values' products
#pragma unroll
                for (int r = 0; r < 2 * TT; ++r) {
                    s[r][0] += s[r][2];
                    s[r][1] += s[r][3];
                }
            }
            // scores in units of log 2: s[r][e] is token 8 r + 2 t + e % 2
            const uint32_t mk = mask[0];
            float top[R2];
#pragma unroll
            for (int r = 0; r < R2; ++r) top[r] = -INFINITY;
#pragma unroll
            for (int r = 0; r < 2 * TT; ++r)
#pragma unroll
                for (int e = 0; e < 2 * R2; ++e) s[r][e] *= zs[e >> 1];
            if (mk != (TT == 2 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
                for (int r = 0; r < 2 * TT; ++r)
#pragma unroll
                    for (int e = 0; e < 2 * R2; ++e)
                        if (!(mk >> (8 * r + 2 * t + (e & 1)) & 1)) s[r][e] = -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 2 * TT; ++r)
#pragma unroll
                for (int e = 0; e < 2 * R2; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[r][e]);
            bool grows = false;
#pragma unroll
            for (int r = 0; r < R2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                grows |= top[r] > m[r];
            }
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int r = 0; r < R2; ++r) {
                    const float mn = fmaxf(m[r], top[r]), c = mn == -INFINITY ? 1.f : ex2(m[r] - mn);
                    m[r] = mn;
                    l[r] *= c;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        acc[j][2 * r] *= c;
                        acc[j][2 * r + 1] *= c;
                    }
                }
            }
            uint32_t pf[TT][2 * R2];
#pragma unroll
            for (int r = 0; r < R2; ++r) {
                const float sub = m[r] == -INFINITY ? 0.f : m[r] - LIFT;
#pragma unroll
                for (int b = 0; b < TT; ++b) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = ex2(s[2 * b + (e >> 1)][2 * r + (e & 1)] - sub);
                    l[r] += (w[0] + w[1]) + (w[2] + w[3]);
                    pf[b][r] = Frag<C>::pack(w[0], w[1]);
                    pf[b][R2 + r] = Frag<C>::pack(w[2], w[3]);
                }
            }
#pragma unroll
            for (int b = 0; b < TT; ++b) {
                const uint32_t off = stage * L::BYTES + b * L::BLOCK;
                if constexpr (F8) {
#pragma unroll
                    for (int c = 0; c < VC; ++c) {
                        uint32_t v[4][VB / 4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if constexpr (VB == 16) {
                                const uint4 x = tc::lds128(v8_at(r, c) + off);
                                v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                            } else {
                                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v[r][0]), "=r"(v[r][1]) : "r"(v8_at(r, c) + off) : "memory");
                            }
                        }
#pragma unroll
                        for (int x = 0; x < VB / 4; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {  // features 4x + 2y, 4x + 2y + 1
                                const uint32_t lo = __byte_perm(v[0][x], v[1][x], y ? 0x7362 : 0x5140);
                                const uint32_t hi = __byte_perm(v[2][x], v[3][x], y ? 0x7362 : 0x5140);
                                uint32_t b0[2], b1[2];
                                f8x4(lo, b0[0], b0[1]);
                                f8x4(hi, b1[0], b1[1]);
                                mma(acc[c * VE + 4 * x + 2 * y], pf[b], b0[0], b1[0]);
                                mma(acc[c * VE + 4 * x + 2 * y + 1], pf[b], b0[1], b1[1]);
                            }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < D / 8; c += 2) {
                        uint32_t v[4];
                        ldmatrix4t((v_at ^ (c << 4)) + off, v);
                        mma(acc[c], pf[b], v[0], v[1]);
                        mma(acc[c + 1], pf[b], v[2], v[3]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j + 1 < STAGES; ++j) mask[j] = mask[j + 1];
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }

        // ---- join the warps: sums over a row's 4 lanes, then over the warps in order
        cp_wait<0>();
        __syncthreads();
        float* accs = reinterpret_cast<float*>(smem) + warp * 16 * L::PAD;
#pragma unroll
        for (int r = 0; r < R2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t == 0) {
                ml_s[warp][g + 8 * r][0] = m[r] - LIFT;
                ml_s[warp][g + 8 * r][1] = l[r];
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                const int d = F8 ? (2 * t + 8 * (j / VE)) * VE + j % VE : 8 * j + 2 * t;
                accs[(g + 8 * r) * L::PAD + d] = acc[j][2 * r];
                accs[(g + 8 * r) * L::PAD + d + (F8 ? VE : 1)] = acc[j][2 * r + 1];
            }
        }
        __syncthreads();
        const float* all_acc = reinterpret_cast<const float*>(smem);
        const int rows = min(16, G - hb);
        for (int i = tid; i < rows * (D / 4); i += L::T) {
            const int h = i / (D / 4), d = i % (D / 4) * 4;
            float M = -INFINITY, S = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, ml_s[w][h][0]);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float c = ml_s[w][h][0] == -INFINITY ? 0.f : ex2(ml_s[w][h][0] - M);
                const float4 x = *reinterpret_cast<const float4*>(all_acc + (w * 16 + h) * L::PAD + d);
                S = fmaf(ml_s[w][h][1], c, S);
                a.x = fmaf(x.x, c, a.x);
                a.y = fmaf(x.y, c, a.y);
                a.z = fmaf(x.z, c, a.z);
                a.w = fmaf(x.w, c, a.w);
            }
            if (A.cluster > 1) {
                *reinterpret_cast<float4*>(res + h * D + d) = a;
                if (d == 0) res_ml[h] = make_float2(M, S);
            } else if (whole) {
                const int64_t row = int64_t(n) * p.Hq + hk * G + hb + h;
                const bool some = S > 0.f || S != S;
                const float f = some ? vs / S : 0.f;
                const uint2 o = make_uint2(tc::pack_bf16(a.x * f, a.y * f), tc::pack_bf16(a.z * f, a.w * f));
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.o) + row * D + d) = o;
                if (A.lse && d == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
            } else {
                const int64_t at = place_of(blockIdx.x, began, 16) + h;
                *reinterpret_cast<float4*>(A.part + at * D + d) = a;
                if (d == 0) A.part_ml[at] = make_float2(M, S);
            }
        }
        __syncthreads();  // the stages and ml_s are read before the next pair writes them
    }
    if (A.cluster > 1) {
        const int block = P0.head * A.groups + P0.group, hb = (block % nb) * 16;
        join_cluster<__nv_bfloat16, D, L::T>(A, tc::smem_addr(res), tc::smem_addr(res_ml), P0.n, block / nb, hb, min(16, G - hb));
    }
}

// Joins the parts of the rows that several CTAs have parts of, in the list's order.  A block of 8
// warps takes RPB rows: a warp each (8), or all 8 warps one row's parts (1: few rows, many parts).
constexpr int JW = 8;
template <typename Act, int D, int RPB>
__global__ void __launch_bounds__(32 * JW) k_paged_join(const PagedArgs A, int tok, int rows, int ctas, int warps) {
    constexpr int E = D / 32;
    __shared__ float acc_s[RPB == 1 ? JW : 1][D], ml_s[RPB == 1 ? JW : 1][2];
    tc::pdl_wait();
    const gdn_paged_problem& p = A.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = RPB == 1 ? blockIdx.x : int64_t(blockIdx.x) * JW + warp;
    if (row >= int64_t(p.num_seqs) * p.Hq) return;  // with RPB == 1 never
    const int n = int(quotient(row, p.Hq)), h = int(row - int64_t(n) * p.Hq), G = p.Hq / p.Hkv, nb = (G + rows - 1) / rows;
    const int block = (h / G) * nb + (h % G) / rows, in = (h % G) % rows;
    const int head = block / A.groups, group = block % A.groups;
    const int64_t before = A.before[n], tiles = A.before[n + 1] - before;
    const int64_t share = share_of(A.before[p.num_seqs] * A.heads, ctas / A.groups, warps);
    const int64_t at0 = before * A.heads + head * tiles, at1 = at0 + tiles;
    const int c0 = int(quotient(at0, share)), c1 = int(quotient(at1 - 1, share));
    if (c0 == c1) return;  // that CTA wrote it out
    // parts c0 .. c1; this warp's: c0 + first, first + step, ...
    const int parts = c1 - c0 + 1, first = RPB == 1 ? warp : 0, step = RPB == 1 ? JW : 1;
    auto place = [&](int i) { return place_of((c0 + i) * A.groups + group, i > 0 || at0 < c0 * share, rows) + in; };
    float M = -INFINITY, S = 0.f, acc[E] = {};
    // batches of parts, everything of a batch requested at once
    constexpr int NB = D == 256 ? 4 : 8;
    for (int i0 = first; i0 < parts; i0 += step * NB) {
        float2 ml[NB];
        float x[NB][E];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int i = i0 + step * b;
            ml[b] = make_float2(-INFINITY, 0.f);
            if (i < parts) {
                const int64_t at = place(i);
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
            const float w = ml[b].x == -INFINITY ? 0.f : ex2(ml[b].x - M);
            S = fmaf(ml[b].y, w, S);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(x[b][e], w, acc[e]);
        }
    }
    if constexpr (RPB == 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc_s[warp][32 * e + lane] = acc[e];
        if (lane == 0) {
            ml_s[warp][0] = M;
            ml_s[warp][1] = S;
        }
        __syncthreads();
        if (warp > 0) return;
        S = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < JW; ++w) M = fmaxf(M, ml_s[w][0]);
#pragma unroll
        for (int w = 0; w < JW; ++w) {
            const float c = ml_s[w][0] == -INFINITY ? 0.f : ex2(ml_s[w][0] - M);
            S = fmaf(ml_s[w][1], c, S);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(acc_s[w][32 * e + lane], c, acc[e]);
        }
    }
    const bool some = S > 0.f || S != S;
    const float f = some ? (A.v_scale ? A.v_scale[h / G] : 1.f) / S : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) static_cast<Act*>(A.o)[row * D + 32 * e + lane] = from_f<Act>(acc[e] * f);
    if (A.lse && lane == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
}

constexpr int CLUSTER_WORK = 4096;  // values of a key row's feature times tokens per warp that are not worth splitting

// What the launches need to know of a kernel.
struct Shape {
    int tok, rows, warps, ctas;  // tokens of a tile, rows of a block of heads, warps that share tiles, CTAs per multiprocessor
};
template <typename C, int D> constexpr Shape mma_shape() { return {Tile<C, D>::TOK, 16, Tile<C, D>::W, Tile<C, D>::CTAS}; }
template <int D> constexpr Shape fp32_shape() { return {PTOK, GB, 1, D == 256 ? 2 : 4}; }
Shape shape_of(const gdn_paged_problem& p) {
    if (p.dtype == GDN_FP32) return p.D == 64 ? fp32_shape<64>() : p.D == 128 ? fp32_shape<128>() : fp32_shape<256>();
    if (p.cache_dtype == GDN_BF16)
        return p.D == 64 ? mma_shape<__nv_bfloat16, 64>() : p.D == 128 ? mma_shape<__nv_bfloat16, 128>() : mma_shape<__nv_bfloat16, 256>();
    return p.D == 64 ? mma_shape<__nv_fp8_e4m3, 64>() : p.D == 128 ? mma_shape<__nv_fp8_e4m3, 128>() : mma_shape<__nv_fp8_e4m3, 256>();
}

template <typename... K>
cudaError_t launch_clusters(void (*kern)(K...), const PagedArgs& A, int ctas, int threads, size_t smem, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = A.cluster > 1 ? A.cluster : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = A.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, A);
}

template <typename Act, int D>
cudaError_t launch_join(const PagedArgs& A, const PagedPlan& plan, const Shape& s, cudaStream_t st) {
    if (plan.cluster) return cudaGetLastError();
    const int64_t rows = int64_t(A.p.num_seqs) * A.p.Hq;
    timing_begin("paged_attn_join", st);
    const cudaError_t e =
        rows <= 1024 ? launch_pdl(k_paged_join<Act, D, 1>, dim3(unsigned(rows)), dim3(32 * JW), 0, st, A, s.tok, s.rows, plan.ctas, s.warps)
                     : launch_pdl(k_paged_join<Act, D, JW>, dim3(unsigned((rows + JW - 1) / JW)), dim3(32 * JW), 0, st, A, s.tok, s.rows, plan.ctas, s.warps);
    timing_end(st);
    return e;
}

template <int D>
cudaError_t launch_fp32(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    timing_begin("paged_attn", st);
    const cudaError_t e = launch_clusters(k_paged<D>, A, plan.ctas, PT, 0, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
    return launch_join<float, D>(A, plan, fp32_shape<D>(), st);
}

template <typename C, int D, bool HALF, bool TILED>
cudaError_t launch_mma(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    using L = Tile<C, D>;
    cudaError_t e = smem_attr(k_paged_mma<C, D, HALF, TILED>, L::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin("paged_attn", st);
    e = launch_clusters(k_paged_mma<C, D, HALF, TILED>, A, plan.ctas, L::T, L::SMEM, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
    return launch_join<__nv_bfloat16, D>(A, plan, mma_shape<C, D>(), st);
}

template <typename C, int D>
cudaError_t launch_dim(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    const bool half = A.p.Hq / A.p.Hkv <= 8, tiled = A.p.page_size % 16 == 0;
    if (half) return tiled ? launch_mma<C, D, true, true>(A, plan, st) : launch_mma<C, D, true, false>(A, plan, st);
    return tiled ? launch_mma<C, D, false, true>(A, plan, st) : launch_mma<C, D, false, false>(A, plan, st);
}

template <typename C>
cudaError_t launch_type(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    return A.p.D == 64 ? launch_dim<C, 64>(A, plan, st) : A.p.D == 128 ? launch_dim<C, 128>(A, plan, st) : launch_dim<C, 256>(A, plan, st);
}

}  // namespace

PagedPlan paged_plan(const gdn_paged_problem& p) {
    const Shape s = shape_of(p);
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
    const int64_t cap = int64_t(p.max_pages) * p.page_size, most = p.window > 0 && p.window + 16 < cap ? p.window + 16 : cap;
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
    return A.p.cache_dtype == GDN_BF16 ? launch_type<__nv_bfloat16>(A, plan, st) : launch_type<__nv_fp8_e4m3>(A, plan, st);
}

}  // namespace gdn
