// Attention over a bf16 or 8-bit paged cache on tensor-core fragments (see gdn_paged.cu).
#pragma once
#include "gdn_paged.cuh"

namespace gdn {
namespace {

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

// SOLO: a CTA of one warp per (sequence, block of heads), for many short caches.
template <typename C, int D, bool SOLO = false> struct Tile {
    static constexpr int E = int(sizeof(C));
    static constexpr int TT = D * E <= 128 ? 2 : 1;                // 16-token blocks of a tile
    static constexpr int TOK = 16 * TT;                            // tokens of a tile
    static constexpr int W = SOLO ? 1 : D * E > 256 ? 2 : 4;       // warps
    static constexpr int T = 32 * W;                               // threads
    static constexpr int CTAS = SOLO ? (D * E > 256 ? 4 : D == 256 ? 8 : D == 128 ? 10 : 12) : D == 64 && E == 2 ? 3 : 2;  // per multiprocessor
    static constexpr int ROW = D * E;                              // bytes of a row
    static constexpr int CPR = ROW / 16;                           // 16-byte pieces of a row
    static constexpr int RPI = 32 / CPR;                           // rows per copy instruction of a warp
    static constexpr int VB = ROW / 8 >= 16 ? 16 : ROW / 8;        // 8-bit: bytes of a piece of a value row
    static constexpr int VC = E == 1 ? ROW / (8 * VB) : 0;         // 8-bit: pieces of a value row per thread
    static constexpr int BLOCK = 16 * ROW;                         // bytes of 16 rows
    static constexpr int BYTES = 2 * TT * BLOCK;                   // of a warp's tile: K's blocks, V's blocks
    static constexpr int FIT = (SOLO ? 196608 / CTAS : CTAS == 3 ? 65536 : 98304) / (W * BYTES);
    static constexpr int STAGES = FIT < 3 ? FIT : 3;               // more take more time (8 bits, 64 features: 6 of them 2 to 8 %)
    static constexpr int PAD = D + 4;                              // floats between rows of the joined accumulators
    static constexpr int SMEM = STAGES * W * BYTES;
    static_assert(STAGES >= 2 && W * 16 * PAD * 4 + (SOLO ? 0 : 16 * D * 4) <= SMEM, "the warps' accumulators are joined in the stages' memory");
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

template <typename C, int D, bool HALF, bool TILED, bool SOLO>
__global__ void __launch_bounds__(Tile<C, D, SOLO>::T, Tile<C, D, SOLO>::CTAS) k_paged_mma(const PagedArgs A) {
    using L = Tile<C, D, SOLO>;
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
        // The lanes look after the page table together: of LOOK blocks of 16 tokens, one lane each with TILED (a
        // page holds whole blocks), else a lane to each token.  A lane reads its page (AHEAD looks ahead) and
        // works out where its rows begin and which count; the copies take the offsets from that lane.  With a
        // look and the arithmetic in every lane for every tile, 16 sequences of up to 48828 tokens, 8 kv-heads,
        // took 96 us instead of 77 (8 bits, 64 features, pages of 16 tokens), of up to 6103 92 us instead of 67 (bf16,
        // 256 features, pages of one).  -1 where there is nothing to attend to.
        constexpr int LOOK = TILED ? 32 : 2, AHEAD = TILED ? 1 : 2;
        auto block_of = [&](int x) { return x + (TILED ? lane : lane >> 4); };
        auto first_of = [&](int x) { return token_of(x / TT) + 16 * (x % TT) + (TILED ? 0 : lane & 15); };
        auto page_at = [&](int from) {
            const int x = block_of(from), tok = first_of(x);
            const bool in = x / TT < tiles && tok < t1 && (TILED || tok >= t0);
            return in ? __ldg(table + A.page_div.of(tok)) : -1;  // looked at in locate: the load is not waited for here
        };
        constexpr int PRO = (TT * (STAGES - 1) + LOOK - 1) / LOOK;  // looks that the tiles requested ahead need
        int first[PRO + AHEAD];
#pragma unroll
        for (int i = 0; i < PRO + AHEAD; ++i) first[i] = page_at(i * LOOK);
        int64_t ko = 0, vo = 0;
        uint32_t counts = 0u;  // TILED: tokens of this lane's block; else tokens of both blocks, in every lane
        auto locate = [&](int from, int page) {
            if (page >= p.num_pages) page = -1;
            const int tok = first_of(block_of(from)), slot = slot_of(tok);
            if constexpr (TILED) {
                counts = page < 0 ? 0u : 0xffffu;
                if (t0 > tok) counts &= 0xffffu << min(t0 - tok, 16);
                if (t1 - tok < 16) counts &= 0xffffu >> min(16 - (t1 - tok), 16);
            } else {
                counts = __ballot_sync(0xffffffffu, page >= 0);
            }
            ko = page < 0 ? 0 : page * p.k_page_stride + slot * p.k_token_stride;
            vo = page < 0 ? 0 : page * p.v_page_stride + slot * p.v_token_stride;
        };

        if (A.k_new && R.fits && end == tiles_n) {  // every block of heads writes the same bits before it reads them
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

        // where block b of tile i lies, and which of its tokens count
        const C* kl = kc + copy_piece * (16 / L::E) + (TILED ? copy_row * p.k_token_stride : 0);
        const C* vl = vc + copy_piece * (16 / L::E) + (TILED ? copy_row * p.v_token_stride : 0);
        struct Place {
            const C *k, *v;
            uint32_t valid;
            int x;
        };
        auto place = [&](int i, int b) -> Place {
            const int x = (i * TT + b) % LOOK;
            if (TILED) return {kl + __shfl_sync(0xffffffffu, ko, x), vl + __shfl_sync(0xffffffffu, vo, x), __shfl_sync(0xffffffffu, counts, x), x};
            return {kl, vl, counts >> (16 * x) & 0xffffu, x};
        };
        // Requests its rows (zeros where masked).
        auto issue = [&](const Place& P, int b, int stage) {
            const uint32_t to = copy_to + stage * L::BYTES + b * L::BLOCK, valid = P.valid;
            if constexpr (TILED) {
                const C *kt = P.k, *vt = P.v;
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
#pragma unroll
                for (int j = 0; j < 16 / RPI; ++j) {
                    const int row = copy_row + RPI * j;
                    const bool in = valid >> row & 1;
                    const uint32_t at = (to ^ (L::swap(RPI * j) << 4)) + RPI * j * ROW;
                    cp_async(at, P.k + __shfl_sync(0xffffffffu, ko, 16 * P.x + row), in);
                    cp_async(at + TT * L::BLOCK, P.v + __shfl_sync(0xffffffffu, vo, 16 * P.x + row), in);
                }
            }
        };

        uint32_t mask[STAGES];  // which tokens of the tiles in flight count, oldest first
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            mask[i] = 0u;
            if (i * TT % LOOK == 0) locate(i * TT, first[i * TT / LOOK]);
            if (i < tiles)
#pragma unroll
                for (int b = 0; b < TT; ++b) {
                    const Place at = place(i, b);
                    issue(at, b, i);
                    mask[i] |= at.valid << (16 * b);
                }
            cp_commit();
        }
        int pages[AHEAD];  // of the next looks
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) pages[i] = first[PRO + i];

        // ---- query fragments, of 16-feature step s: features 2t, + 1 and 8 + 2t, + 1.  8-bit caches, of
        // 32-feature step s: features 4t .. 4t + 3 and 16 + 4t .., each value the sum of two 8-bit ones of
        // the row scaled to [128, 256): exact for bf16's 8 significant bits down to 2^-9 of the row's
        // largest value (4 bits each, the second with a sign of its own), off by 2^-18 of it below.  A row
        // below 2^-119 is scaled by 2^126 (beyond 2^127 the factor would be infinite): bf16's values, all
        // multiples of 2^-133, are then multiples of 2^-7, and exact.
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
                const int e = fine ? max(ilogbf(top) - 7, -126) : 0;
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
        Place at[TT];  // of the next tile to request
        auto look_on = [&](int next) {
            if (next * TT % LOOK == 0) {
                locate(next * TT, pages[0]);
#pragma unroll
                for (int j = 1; j < AHEAD; ++j) pages[j - 1] = pages[j];
                pages[AHEAD - 1] = page_at(next * TT + AHEAD * LOOK);
            }
#pragma unroll
            for (int b = 0; b < TT; ++b) at[b] = place(next, b);
        };
        look_on(STAGES - 1);
        for (int i = 0; i < tiles; ++i) {
            const int next = i + STAGES - 1;
            cp_wait<STAGES - 2>();
            __syncwarp();  // every lane's copies of tile i have landed, and tile i - 1 has been read
            mask[STAGES - 1] = 0u;
            if (next < tiles)
#pragma unroll
                for (int b = 0; b < TT; ++b) {
                    issue(at[b], b, stage == 0 ? STAGES - 1 : stage - 1);
                    mask[STAGES - 1] |= at[b].valid << (16 * b);
                }
            cp_commit();
            look_on(next + 1);
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

template <typename C, int D> constexpr PagedShape mma_shape() { return {Tile<C, D>::TOK, 16, Tile<C, D>::W, Tile<C, D>::CTAS}; }

template <typename C, int D, bool HALF, bool TILED, bool SOLO>
cudaError_t launch_mma(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    using L = Tile<C, D, SOLO>;
    cudaError_t e = smem_attr(k_paged_mma<C, D, HALF, TILED, SOLO>, L::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin("paged_attn", st);
    e = launch_clusters(k_paged_mma<C, D, HALF, TILED, SOLO>, A, plan.ctas, L::T, L::SMEM, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
    return launch_join<__nv_bfloat16, D>(A, plan, mma_shape<C, D>(), st);
}

template <typename C, int D, bool SOLO>
cudaError_t launch_warps(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    const bool half = A.p.Hq / A.p.Hkv <= 8, tiled = A.p.page_size % 16 == 0;
    if (half) return tiled ? launch_mma<C, D, true, true, SOLO>(A, plan, st) : launch_mma<C, D, true, false, SOLO>(A, plan, st);
    return tiled ? launch_mma<C, D, false, true, SOLO>(A, plan, st) : launch_mma<C, D, false, false, SOLO>(A, plan, st);
}

template <typename C>
cudaError_t launch_type(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    if (plan.solo)
        return A.p.D == 64 ? launch_warps<C, 64, true>(A, plan, st) : A.p.D == 128 ? launch_warps<C, 128, true>(A, plan, st) : launch_warps<C, 256, true>(A, plan, st);
    return A.p.D == 64 ? launch_warps<C, 64, false>(A, plan, st) : A.p.D == 128 ? launch_warps<C, 128, false>(A, plan, st) : launch_warps<C, 256, false>(A, plan, st);
}

template <typename C>
PagedShape shape_type(int D) {
    return D == 64 ? mma_shape<C, 64>() : D == 128 ? mma_shape<C, 128>() : mma_shape<C, 256>();
}

}  // namespace
}  // namespace gdn
