// Attention of one new token per sequence over a paged key-value cache (include/gdn.h,
// gdn_paged_attn_decode): o_h = sum_t softmax(scale <q_h, k_t>)_t v_t, lse_h = log sum_t e^{z_t}.
//
// A sequence's tokens are cut into ranges of split_len tokens; a CTA takes one range of one
// kv-head (and a block of its query heads), keeping a running maximum m, sum l of e^{z - m} and
// accumulator of e^{z - m} v: one pass over keys and values.  Ranges are joined by a second
// kernel from (accumulator, m, l) triples in range order; a sequence of one range is written out
// directly.  Bound: HBM, 2 D bytes-per-value per token and kv-head.
//
// bf16 and 8-bit caches: k_paged_mma.  A warp takes tiles of 16 tokens.  Both products run on
// m16n8k16 tensor-core fragments (up to 16 query heads are the 16 rows), whose operands a thread
// can load straight from the cache in 16-byte pieces, because the order of a contraction index and
// of output columns is free as long as both sides agree:
//   S = Q K^T   thread (g = lane / 4, t = lane % 4) has token g of each 8 and the pieces t + 4 i of
//               its row: 4 consecutive features stand for the fragment's k = 2t, 2t+1, 2t+8, 2t+9;
//   O = P V     P is S's accumulator as it lies; the thread has tokens 2t, 2t+1, 2t+8, 2t+9 and the
//               pieces g + 8 m of their rows: feature e of a piece is column g of n-tile e.
// So no value is exchanged between threads: a thread copies its own pieces to its own slots in
// shared memory (cp.async, STAGES tiles deep) and reads them back, without a barrier in the loop,
// whatever the page size.  With 16 query rows a tcgen05 tile would be mostly padding, and its
// operands would need the shared-memory layout that this avoids.
// 8-bit values are converted to fp16 (exactly), with the query rows scaled by a power of two to
// [-2, 2] for the fp16 range; the weights are rounded to bf16 (fp16 for 8-bit caches) for the second
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

// What a CTA has to do for sequence n.
struct Range {
    int len, first, base, count;  // tokens, the first one attended to, it down to a tile's start, ranges
};
__device__ __forceinline__ Range range_of(const PagedArgs& A, int n) {
    const int64_t cap = int64_t(A.p.max_pages) * A.p.page_size;
    Range R;
    const int64_t len = A.lens[n];
    R.len = int(len < 0 ? 0 : len < cap ? len : cap);
    R.first = A.p.window > 0 && R.len > A.p.window ? R.len - A.p.window : 0;
    R.base = R.first & ~15;
    R.count = int((int64_t(R.len) - R.base + A.split_len - 1) / A.split_len);
    if (R.count < 1) R.count = 1;
    return R;
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
__device__ __forceinline__ float from_cache(float x) { return x; }

constexpr int PT = 128;  // threads
constexpr int GB = 4;    // query heads per CTA

template <typename C, int D> struct Lanes {
    static constexpr int E = (16 / int(sizeof(C)) > D / 32) ? 16 / int(sizeof(C)) : D / 32;  // values per lane
    static constexpr int LP = D / E;                                                         // lanes per token
    static constexpr int GROUPS = PT / LP;
};

template <typename C, int E>
__device__ __forceinline__ void load_row(const C* p, float (&x)[E]) {
    constexpr int W = 16 / int(sizeof(C));
#pragma unroll
    for (int b = 0; b < E / W; ++b) {
        C v[W];
        *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p + b * W);
#pragma unroll
        for (int e = 0; e < W; ++e) x[b * W + e] = from_cache(v[e]);
    }
}

template <typename Act, typename C, int D>
__global__ void __launch_bounds__(PT) k_paged(const PagedArgs A) {
    using L = Lanes<C, D>;
    constexpr int E = L::E, LP = L::LP, GROUPS = L::GROUPS;
    __shared__ __align__(16) float acc_s[GROUPS][GB][D];
    __shared__ float ml_s[GROUPS][GB][2];
    __shared__ __align__(16) C new_s[2][D];
    const gdn_paged_problem& p = A.p;
    const int tid = threadIdx.x, lane = tid % LP, grp = tid / LP;
    const int G = p.Hq / p.Hkv, nb = (G + GB - 1) / GB;
    const int split = blockIdx.x, hk = blockIdx.y / nb, hb = (blockIdx.y % nb) * GB, n = blockIdx.z;
    const Range R = range_of(A, n);
    if (split >= R.count) return;
    const int start = R.base + split * A.split_len;
    const int t0 = max(R.first, start), t1 = min(R.len, start + A.split_len);
    const float ks = A.k_scale ? A.k_scale[hk] : 1.f, vs = A.v_scale ? A.v_scale[hk] : 1.f;
    const int32_t* table = A.table + n * p.table_stride;
    const C* kc = static_cast<const C*>(A.k_cache) + hk * p.k_head_stride;
    const C* vc = static_cast<const C*>(A.v_cache) + hk * p.v_head_stride;

    int t_new = -1;  // the position whose row comes from k_new, v_new
    if (A.k_new && R.len > 0 && R.len == t1) {
        t_new = R.len - 1;
        const int page = table[t_new / p.page_size], slot = t_new % p.page_size;
        const bool in = page >= 0 && page < p.num_pages;
        for (int i = tid; i < D; i += PT) {
            const int64_t at = n * p.new_stride + hk * D + i;
            new_s[0][i] = to_cache<C>(to_f(static_cast<const Act*>(A.k_new)[at]), ks);
            new_s[1][i] = to_cache<C>(to_f(static_cast<const Act*>(A.v_new)[at]), vs);
            if (in && hb == 0) {
                const_cast<C*>(kc)[page * p.k_page_stride + slot * p.k_token_stride + i] = new_s[0][i];
                const_cast<C*>(vc)[page * p.v_page_stride + slot * p.v_token_stride + i] = new_s[1][i];
            }
        }
        __syncthreads();
    }

    float q[GB][E], acc[GB][E], m[GB], l[GB];
#pragma unroll
    for (int h = 0; h < GB; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[h][e] = 0.f;
            q[h][e] = hb + h < G ? to_f(static_cast<const Act*>(A.q)[n * p.q_stride + (hk * G + hb + h) * D + lane * E + e]) : 0.f;
        }
    }
    const float zs = p.scale * ks;
    for (int t = t0 + grp; t - grp < t1; t += GROUPS) {
        bool live = t < t1;
        float kx[E] = {}, vx[E] = {};
        if (live) {
            if (t == t_new) {
                load_row<C, E>(&new_s[0][lane * E], kx);
                load_row<C, E>(&new_s[1][lane * E], vx);
                const int page = table[t / p.page_size];
                live = page >= 0 && page < p.num_pages;
            } else {
                const int page = table[t / p.page_size], slot = t % p.page_size;
                live = page >= 0 && page < p.num_pages;
                if (live) {
                    load_row<C, E>(kc + page * p.k_page_stride + slot * p.k_token_stride + lane * E, kx);
                    load_row<C, E>(vc + page * p.v_page_stride + slot * p.v_token_stride + lane * E, vx);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) z = fmaf(q[h][e], kx[e], z);
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            if (live) {
                z *= zs;
                const float mn = fmaxf(m[h], z), c = m[h] == -INFINITY ? 0.f : expf(m[h] - mn);
                const float e0 = mn == -INFINITY ? 0.f : expf(z - mn);
                l[h] = fmaf(l[h], c, e0);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[h][e] = fmaf(acc[h][e], c, e0 * vx[e]);
                m[h] = mn;
            }
        }
    }
#pragma unroll
    for (int h = 0; h < GB; ++h) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc_s[grp][h][lane * E + e] = acc[h][e];
        if (lane == 0) {
            ml_s[grp][h][0] = m[h];
            ml_s[grp][h][1] = l[h];
        }
    }
    __syncthreads();
    for (int i = tid; i < GB * D; i += PT) {
        const int h = i / D, d = i % D;
        if (hb + h >= G) break;
        float M = -INFINITY, S = 0.f, a = 0.f;
        for (int g = 0; g < GROUPS; ++g) M = fmaxf(M, ml_s[g][h][0]);
        for (int g = 0; g < GROUPS; ++g) {
            const float c = ml_s[g][h][0] == -INFINITY ? 0.f : expf(ml_s[g][h][0] - M);
            S = fmaf(ml_s[g][h][1], c, S);
            a = fmaf(acc_s[g][h][d], c, a);
        }
        const int64_t row = int64_t(n) * p.Hq + hk * G + hb + h;
        if (R.count == 1) {
            static_cast<Act*>(A.o)[row * D + d] = from_f<Act>(S > 0.f || S != S ? a / S * vs : 0.f);
            if (A.lse && d == 0) A.lse[row] = M + logf(S);
        } else {
            A.part[(row * A.splits + split) * D + d] = a;
            if (d == 0) {
                float* ml = A.part + int64_t(p.num_seqs) * p.Hq * A.splits * D + (row * A.splits + split) * 2;
                ml[0] = M * LOG2E;
                ml[1] = S;
            }
        }
    }
}

// ---------------------------------------------------------------- bf16 and 8-bit caches
__device__ __forceinline__ float ex2(float x) { return exp2f(x); }

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
// two 8-bit values (the low 16 bits) as fp16
__device__ __forceinline__ uint32_t f8x2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xffffu), __NV_E4M3);
    return uint32_t(h.x) | (uint32_t(h.y) << 16);
}

// copy of B bytes to shared memory, zeros where !in (the address is not read then)
template <int B>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool in) {
    if constexpr (B == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(in ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

template <typename C, int D> struct Tile {
    static constexpr int E = int(sizeof(C));
    static constexpr int W = D * E > 256 ? 2 : 4;                  // warps
    static constexpr int T = 32 * W;                               // threads
    static constexpr int KC = D * E / 64;                          // pieces of a key row per thread
    static constexpr int VB = D * E / 8 >= 16 ? 16 : D * E / 8;    // bytes of a piece of a value row
    static constexpr int VC = D * E / (8 * VB);                    // pieces of a value row per thread
    static constexpr int BYTES = 32 * KC + 4 * VC * VB;            // per thread and tile
    static constexpr int STAGES = 98304 / (T * BYTES) < 8 ? 98304 / (T * BYTES) : 8;
    static constexpr int PAD = D + 4;                              // floats between rows of the joined accumulators
    static constexpr int SMEM = STAGES * T * BYTES;
    static_assert(STAGES >= 2 && W * 16 * PAD * 4 <= SMEM, "the warps' accumulators are joined in the stages' memory");
};

template <typename C, int D, bool HALF>
__global__ void __launch_bounds__(Tile<C, D>::T) k_paged_mma(const PagedArgs A) {
    using L = Tile<C, D>;
    constexpr int KC = L::KC, VC = L::VC, VB = L::VB, STAGES = L::STAGES, W = L::W, R2 = HALF ? 1 : 2;
    constexpr int CB = 16 / L::E;                 // values per 16-byte piece
    constexpr int KS = D / 16;                    // k16 steps
    constexpr bool F8 = L::E == 1;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float ml_s[W][16][2];
    const gdn_paged_problem& p = A.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.Hkv, nb = (G + 15) / 16;
    const int split = blockIdx.x, hk = blockIdx.y / nb, hb = (blockIdx.y % nb) * 16, n = blockIdx.z;
    tc::pdl_launch_dependents();
    const Range R = range_of(A, n);
    if (split >= R.count) return;
    const int start = R.base + split * A.split_len;
    const int t0 = max(R.first, start), t1 = min(R.len, start + A.split_len);
    const float ks = A.k_scale ? A.k_scale[hk] : 1.f, vs = A.v_scale ? A.v_scale[hk] : 1.f;
    const int32_t* table = A.table + n * p.table_stride;
    C* kc = static_cast<C*>(A.k_cache) + hk * p.k_head_stride;
    C* vc = static_cast<C*>(A.v_cache) + hk * p.v_head_stride;
    const unsigned psize = unsigned(p.page_size);

    if (A.k_new && R.len > 0 && R.len == t1) {  // every block of heads writes the same bits before it reads them
        const int at = R.len - 1, page = table[at / psize];
        if (page >= 0 && page < p.num_pages) {
            C* kd = kc + page * p.k_page_stride + (at % psize) * p.k_token_stride;
            C* vd = vc + page * p.v_page_stride + (at % psize) * p.v_token_stride;
            const int64_t from = n * p.new_stride + int64_t(hk) * D;
            for (int i = tid; i < D; i += L::T) {
                kd[i] = to_cache<C>(to_f(static_cast<const __nv_bfloat16*>(A.k_new)[from + i]), ks);
                vd[i] = to_cache<C>(to_f(static_cast<const __nv_bfloat16*>(A.v_new)[from + i]), vs);
            }
        }
        __syncthreads();
    }

    // ---- this warp's tiles: tokens start + 16 (warp + W i)
    const int all = t1 > start ? (t1 - start + 15) / 16 : 0;
    const int tiles = all > warp ? (all - warp + W - 1) / W : 0;
    auto token_of = [&](int i) { return start + 16 * (warp + W * i); };
    // lane l < 16: page of token l of tile i, or -1 where there is nothing to attend to
    auto page_at = [&](int i) {
        const int tok = token_of(i) + (lane & 15);
        if (i >= tiles || tok < t0 || tok >= t1) return -1;
        const int page = table[unsigned(tok) / psize];
        return page >= 0 && page < p.num_pages ? page : -1;
    };
    const uint32_t kslot = tc::smem_addr(smem) + tid * 16, vslot = tc::smem_addr(smem) + L::T * 32 * KC + tid * VB;
    auto issue = [&](int i, int stage, int pages) -> uint32_t {
        const uint32_t valid = __ballot_sync(0xffffffffu, pages >= 0) & 0xffffu;
        const int tok = token_of(i);
        const uint32_t kd = kslot + stage * (L::T * L::BYTES), vd = vslot + stage * (L::T * L::BYTES);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r, page = __shfl_sync(0xffffffffu, pages, row);
            const C* src = kc;
            if (page >= 0) src += page * p.k_page_stride + int64_t(unsigned(tok + row) % psize) * p.k_token_stride + t * CB;
#pragma unroll
            for (int c = 0; c < KC; ++c) cp_async<16>(kd + (r * KC + c) * (L::T * 16), src + c * 4 * CB, page >= 0);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + 8 * (r >> 1), page = __shfl_sync(0xffffffffu, pages, row);
            const C* src = vc;
            if (page >= 0) src += page * p.v_page_stride + int64_t(unsigned(tok + row) % psize) * p.v_token_stride + g * (VB / L::E);
#pragma unroll
            for (int c = 0; c < VC; ++c) cp_async<VB>(vd + (r * VC + c) * (L::T * VB), src + c * 8 * (VB / L::E), page >= 0);
        }
        return valid;
    };

    uint32_t mask[STAGES];  // which tokens of the tiles in flight count, oldest first
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
        mask[i] = i < tiles ? issue(i, i, page_at(i)) : 0u;
        cp_commit();
    }
    int pages = page_at(STAGES - 1);

    // ---- query fragments, in the key pieces' order of features
    uint32_t qf[KS][2 * R2];
    float zs[R2];
#pragma unroll
    for (int r = 0; r < R2; ++r) {
        const int h = hb + g + 8 * r;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(A.q) + n * p.q_stride + int64_t(hk * G + h) * D;
        uint2 raw[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s)
            raw[s] = h < G ? *reinterpret_cast<const uint2*>(q + (t + 4 * (s / (CB / 4))) * CB + 4 * (s % (CB / 4))) : make_uint2(0u, 0u);
        zs[r] = p.scale * ks * LOG2E;
        if constexpr (F8) {
            float top = 0.f;
            float2 f[KS][2];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                f[s][0] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[s].x));
                f[s][1] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[s].y));
                top = fmaxf(top, fmaxf(fmaxf(fabsf(f[s][0].x), fabsf(f[s][0].y)), fmaxf(fabsf(f[s][1].x), fabsf(f[s][1].y))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = top > 0.f && top < INFINITY ? ilogbf(top) : 0;
            const float down = ldexpf(1.f, -e);
            zs[r] = ldexpf(zs[r], e);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[s][r] = Frag<C>::pack(f[s][0].x * down, f[s][0].y * down);
                qf[s][R2 + r] = Frag<C>::pack(f[s][1].x * down, f[s][1].y * down);
            }
        } else {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[s][r] = raw[s].x;
                qf[s][R2 + r] = raw[s].y;
            }
        }
    }

    float acc[D / 8][2 * R2], m[R2], l[R2];
#pragma unroll
    for (int r = 0; r < R2; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 2 * R2; ++e) acc[i][e] = 0.f;
    // the fragments of 16 rows, the lower 8 alone being real with HALF
    auto mma = [&](float (&c)[2 * R2], const uint32_t* a, uint32_t b0, uint32_t b1) {
        if constexpr (HALF) {
            float full[4] = {c[0], c[1], 0.f, 0.f};
            const uint32_t af[4] = {a[0], 0u, a[1], 0u};
            Frag<C>::mma(full, af, b0, b1);
            c[0] = full[0];
            c[1] = full[1];
        } else {
            const uint32_t af[4] = {a[0], a[1], a[2], a[3]};
            Frag<C>::mma(c, af, b0, b1);
        }
    };

    int stage = 0;
    for (int i = 0; i < tiles; ++i) {
        {
            const int next = i + STAGES - 1;
            mask[STAGES - 1] = next < tiles ? issue(next, stage == 0 ? STAGES - 1 : stage - 1, pages) : 0u;
            cp_commit();
            pages = page_at(next + 1);
        }
        cp_wait<STAGES - 1>();
        const uint32_t kd = kslot + stage * (L::T * L::BYTES), vd = vslot + stage * (L::T * L::BYTES);
        float s[2][2 * R2] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 k = tc::lds128(kd + (r * KC + c) * (L::T * 16));
                const uint32_t kw[4] = {k.x, k.y, k.z, k.w};
                if constexpr (F8) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) mma(s[r], qf[4 * c + u], f8x2(kw[u]), f8x2(kw[u] >> 16));
                } else {
#pragma unroll
                    for (int u = 0; u < 2; ++u) mma(s[r], qf[2 * c + u], kw[2 * u], kw[2 * u + 1]);
                }
            }
        }
        // scores in units of log 2; token 2t + e of 8 r'
        const uint32_t mk = mask[0];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2 * R2; ++e) {
                s[r][e] *= zs[e >> 1];
                if (mk != 0xffffu && !(mk >> (8 * r + 2 * t + (e & 1)) & 1)) s[r][e] = -INFINITY;
            }
        bool grows = false;
        float top[R2];
#pragma unroll
        for (int r = 0; r < R2; ++r) {
            float x = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            top[r] = fmaxf(m[r], x);
            grows |= top[r] > m[r];
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
            for (int r = 0; r < R2; ++r) {
                const float c = top[r] == -INFINITY ? 1.f : ex2(m[r] - top[r]);
                m[r] = top[r];
                l[r] *= c;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    acc[j][2 * r] *= c;
                    acc[j][2 * r + 1] *= c;
                }
            }
        }
        uint32_t pf[2 * R2];
#pragma unroll
        for (int r = 0; r < R2; ++r) {
            const float sub = m[r] == -INFINITY ? 0.f : m[r];
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(s[e >> 1][2 * r + (e & 1)] - sub);
            l[r] += (w[0] + w[1]) + (w[2] + w[3]);
            pf[r] = Frag<C>::pack(w[0], w[1]);
            pf[R2 + r] = Frag<C>::pack(w[2], w[3]);
        }
#pragma unroll
        for (int c = 0; c < VC; ++c) {
            uint32_t v[4][VB / 4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t from = vd + (r * VC + c) * (L::T * VB);
                if constexpr (VB == 16) {
                    const uint4 x = tc::lds128(from);
                    v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                } else {
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v[r][0]), "=r"(v[r][1]) : "r"(from) : "memory");
                }
            }
#pragma unroll
            for (int x = 0; x < VB / 4; ++x) {
                if constexpr (F8) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {  // features 4x + 2y, 4x + 2y + 1
                        const uint32_t a = __byte_perm(v[0][x], v[1][x], y ? 0x7362 : 0x5140);
                        const uint32_t b = __byte_perm(v[2][x], v[3][x], y ? 0x7362 : 0x5140);
                        mma(acc[c * VB + 4 * x + 2 * y], pf, f8x2(a), f8x2(b));
                        mma(acc[c * VB + 4 * x + 2 * y + 1], pf, f8x2(a >> 16), f8x2(b >> 16));
                    }
                } else {
                    mma(acc[c * 8 + 2 * x], pf, __byte_perm(v[0][x], v[1][x], 0x5410), __byte_perm(v[2][x], v[3][x], 0x5410));
                    mma(acc[c * 8 + 2 * x + 1], pf, __byte_perm(v[0][x], v[1][x], 0x7632), __byte_perm(v[2][x], v[3][x], 0x7632));
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
            ml_s[warp][g + 8 * r][0] = m[r];
            ml_s[warp][g + 8 * r][1] = l[r];
        }
        constexpr int VE = VB / L::E;  // features of a value piece
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            const int d = (2 * t + 8 * (j / VE)) * VE + j % VE;
            accs[(g + 8 * r) * L::PAD + d] = acc[j][2 * r];
            accs[(g + 8 * r) * L::PAD + d + VE] = acc[j][2 * r + 1];
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
        const int64_t row = int64_t(n) * p.Hq + hk * G + hb + h;
        if (R.count == 1) {
            const float f = S > 0.f || S != S ? vs / S : 0.f;
            const uint2 o = make_uint2(tc::pack_bf16(a.x * f, a.y * f), tc::pack_bf16(a.z * f, a.w * f));
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.o) + row * D + d) = o;
            if (A.lse && d == 0) A.lse[row] = S > 0.f || S != S ? (M + log2f(S)) * LN2 : -INFINITY;
        } else {
            *reinterpret_cast<float4*>(A.part + (row * A.splits + split) * D + d) = a;
            if (d == 0) {
                float* ml = A.part + int64_t(p.num_seqs) * p.Hq * A.splits * D + (row * A.splits + split) * 2;
                *reinterpret_cast<float2*>(ml) = make_float2(M, S);
            }
        }
    }
}

// Joins the ranges of one (sequence, query head) in order.
template <typename Act>
__global__ void k_paged_join(const PagedArgs A) {
    tc::pdl_wait();
    const gdn_paged_problem& p = A.p;
    const int64_t row = blockIdx.x;
    const int n = int(row / p.Hq), h = int(row % p.Hq), d = threadIdx.x, D = p.D;
    const Range R = range_of(A, n);
    if (R.count == 1) return;
    const float* ml = A.part + int64_t(p.num_seqs) * p.Hq * A.splits * D + row * A.splits * 2;
    float M = -INFINITY, S = 0.f, a = 0.f;
    for (int i = 0; i < R.count; ++i) M = fmaxf(M, ml[2 * i]);
#pragma unroll 4
    for (int i = 0; i < R.count; ++i) {
        const float c = ml[2 * i] == -INFINITY ? 0.f : ex2(ml[2 * i] - M);
        S = fmaf(ml[2 * i + 1], c, S);
        a = fmaf(A.part[(row * A.splits + i) * D + d], c, a);
    }
    const float vs = A.v_scale ? A.v_scale[h / (p.Hq / p.Hkv)] : 1.f;
    static_cast<Act*>(A.o)[row * D + d] = from_f<Act>(S > 0.f || S != S ? a / S * vs : 0.f);
    if (A.lse && d == 0) A.lse[row] = S > 0.f || S != S ? (M + log2f(S)) * LN2 : -INFINITY;
}

template <typename Act>
cudaError_t launch_join(const PagedArgs& A, cudaStream_t st) {
    if (A.splits == 1) return cudaGetLastError();
    timing_begin("paged_attn_join", st);
    const cudaError_t e = launch_pdl(k_paged_join<Act>, dim3(unsigned(int64_t(A.p.num_seqs) * A.p.Hq)), dim3(unsigned(A.p.D)), 0, st, A);
    timing_end(st);
    return e;
}

template <int D>
cudaError_t launch_fp32(const PagedArgs& A, cudaStream_t st) {
    const int G = A.p.Hq / A.p.Hkv;
    timing_begin("paged_attn", st);
    k_paged<float, float, D><<<dim3(A.splits, A.p.Hkv * ((G + GB - 1) / GB), A.p.num_seqs), PT, 0, st>>>(A);
    timing_end(st);
    return launch_join<float>(A, st);
}

template <typename C, int D, bool HALF>
cudaError_t launch_mma(const PagedArgs& A, cudaStream_t st) {
    using L = Tile<C, D>;
    const int G = A.p.Hq / A.p.Hkv;
    const cudaError_t e = smem_attr(k_paged_mma<C, D, HALF>, L::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin("paged_attn", st);
    k_paged_mma<C, D, HALF><<<dim3(A.splits, A.p.Hkv * ((G + 15) / 16), A.p.num_seqs), L::T, L::SMEM, st>>>(A);
    timing_end(st);
    return launch_join<__nv_bfloat16>(A, st);
}

template <typename C>
cudaError_t launch_type(const PagedArgs& A, cudaStream_t st) {
    const bool half = A.p.Hq / A.p.Hkv <= 8;
    if (A.p.D == 64) return half ? launch_mma<C, 64, true>(A, st) : launch_mma<C, 64, false>(A, st);
    if (A.p.D == 128) return half ? launch_mma<C, 128, true>(A, st) : launch_mma<C, 128, false>(A, st);
    return half ? launch_mma<C, 256, true>(A, st) : launch_mma<C, 256, false>(A, st);
}

}  // namespace

void paged_plan(const gdn_paged_problem& p, int* splits, int* split_len) {
    const int64_t cap = int64_t(p.max_pages) * p.page_size;
    int64_t most = p.window > 0 && p.window + 16 < cap ? p.window + 16 : cap;  // a range's start goes down to a tile's
    if (most < 1) most = 1;
    const int G = p.Hq / p.Hkv;
    const int64_t groups = int64_t(p.num_seqs > 0 ? p.num_seqs : 1) * p.Hkv * ((G + 15) / 16);
    const int64_t slots = 2 * int64_t(sm_count_cached());  // two CTAs run on a multiprocessor at a time
    // One wave of equal ranges where that gives short ones; else ranges short enough that uneven
    // sequences leave no long tail, with the number of partial results bounded.
    int64_t len = (groups * most + slots - 1) / slots;
    if (len > 2048) len = len / 32 > 512 ? len / 32 : 512;
    if (len < 256) len = 256;
    if (len > most) len = most;
    len = (len + 63) / 64 * 64;
    *split_len = int(len);
    *splits = int((most + len - 1) / len);
}

cudaError_t launch_paged(const PagedArgs& A, cudaStream_t st) {
    if (A.p.dtype == GDN_FP32)
        return A.p.D == 64 ? launch_fp32<64>(A, st) : A.p.D == 128 ? launch_fp32<128>(A, st) : launch_fp32<256>(A, st);
    return A.p.cache_dtype == GDN_BF16 ? launch_type<__nv_bfloat16>(A, st) : launch_type<__nv_fp8_e4m3>(A, st);
}

}  // namespace gdn
