// The gradient of causal attention over prompts in bf16 on the tensor cores (include/gdn.h, gdn_prompt_attn_bwd).
//
// Two launches of one kernel, each recomputing the weights from the forward's lse.  A CTA keeps 128 rows of one
// side and walks over the other side's in tiles of BN (128; 64 with 256 features):
//   keys     K and V of a kv-head stay; Q and dO of the query heads that share it pass, head by head:
//            S = K Q^T, P = e^{S - lse}, dV += P dO; dP = V dO^T, dS = P (dP - D), dK += dS Q.
//   queries  Q and dO of a head stay; K and V pass:  S = Q K^T, dP = dO V^T, dQ += dS K.
// That is 7 products of a tile pair where one pass that adds up dQ in memory would take 5, but dQ needs neither
// atomics (whose order changes results) nor an fp32 copy of itself, and both passes are the same pipeline:
// S and dP lie in tensor memory, two warpgroups (half of a tile's columns each, a thread to a row) make P and dS of
// them in place, in bf16, from where the next product reads them as its left operand.  While P of one tile is made
// the tensor cores work on dK of the one before and on dP; while dS is made, on dV and the next tile's S.
// With 256 features the accumulators of dK and dV would fill tensor memory: a CTA has half of their columns.
// Where there are too few tiles of keys to even out over the multiprocessors, the query heads of a kv-head are
// dealt to several CTAs, whose fp32 sums a last kernel adds up in order.
// Streamed rows behind the sequence are made zeros, for a product of a weight of 0 with what lies there could be NaN.
// Bound: the tensor cores.  Measured, of the 10 D flops per pair that one pass would take (these do 14 D), with the
// statistics and sums, TFLOP/s: 1 x 32768 tokens, 16 / 4 heads, 128 features 9.73 ms, 1130; 2 x 8192, 32 / 8,
// 128 2.51 ms, 1097; 1 x 16384, 32 / 8, 64 4.06 ms, 676 (the weights); 1 x 16384, 16 / 2, 256 7.4 to 7.5 ms, 732 to 741 (S and
// dP of a tile of keys made by two CTAs, one stage of dO).  The keys' pass keeps the tensor cores 69 % busy, the queries' 63 %.
#include "gdn_attn_tc.cuh"

namespace gdn {
namespace {

template <int D, bool KEYS> struct Bwd {
    static constexpr int BN = D == 256 ? 64 : 128;                 // streamed rows of a tile
    static constexpr int RES = 128 * D * 2, STR = BN * D * 2;      // bytes of a resident, of a streamed tile
    static constexpr int N0 = D == 64 ? 3 : 2, N1 = D == 64 ? 3 : D == 128 ? 2 : 1;  // stages of the two streams
    static constexpr int SMEM = 1024 + 2 * RES + (N0 + N1) * STR;
    static constexpr int HALVES = KEYS && D == 256 ? 2 : 1, ND = D / HALVES;  // columns of an accumulator
    static constexpr int T = 352;                                  // 8 warps of weights, then products, loads, statistics
    static constexpr int S = 0, DP = 128, OUT0 = 256, OUT1 = KEYS ? 384 : 256;  // tensor memory columns
    static constexpr int CW = BN / 2;                              // columns of a warpgroup
};

template <int BN> struct BwdShared {
    uint64_t full0[3], empty0[3], full1[3], empty1[3], res_full, s_ready, p_ready, dp_ready, ds_ready, stat_full[2], stat_empty[2], issued[4], clean[4], done, drain;
    alignas(16) float nlse[2][BN];  // of the streamed queries, negated
    float ndrop[2][BN];
    uint32_t tmem;
};

struct BwdMaps {
    CUtensorMap res0, res1, str0, str1;
};

// rows [valid, R) of a swizzled tile of R rows x D values become zeros; by one warp
template <int R, int D>
__device__ __forceinline__ void zero_rows(uint32_t tile, int valid) {
    const int lane = threadIdx.x & 31;
    for (int part = 0; part < D / 64; ++part)
        for (int i = valid * 8 + lane; i < R * 8; i += 32) tc::sts128(tile + part * (R * 128) + i * 16, make_uint4(0u, 0u, 0u, 0u));
}

// parts: of the query heads of a kv-head (KEYS)
template <int D, bool KEYS>
__global__ void __launch_bounds__(Bwd<D, KEYS>::T, 1) k_prompt_bwd_tc(const PromptArgs A, const __grid_constant__ BwdMaps M, int tiles, int parts, float* partial) {
    using L = Bwd<D, KEYS>;
    constexpr int BN = L::BN, CW = L::CW, ND = L::ND;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) BwdShared<BN> sh;
    const gdn_prompt_problem& p = A.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.Hq / p.Hkv;
    const int per = KEYS ? p.Hkv * parts * L::HALVES : p.Hq, number = blockIdx.x / per, sub = blockIdx.x - number * per;
    const int half = KEYS ? sub % L::HALVES : 0, part = KEYS ? sub / L::HALVES % parts : 0;
    const int hk = KEYS ? sub / L::HALVES / parts : sub / G, heads = KEYS ? G / parts : 1, h0 = KEYS ? hk * G + part * heads : sub;
    Seq s;
    int row;
    if (!find_tile<128>(p, KEYS, KEYS ? number : tiles - 1 - number, s, row)) return;  // of a sequence those with the most to do first
    const int rows = min(128, (KEYS ? s.lk : s.lq) - row), streamed = KEYS ? s.lq : s.lk;
    const int64_t res0 = (KEYS ? s.k0 : s.q0) + int64_t(row);
    const int str_at = KEYS ? s.q0 : s.k0;
    // tiles of the streamed side that some row meets
    int lo = 0, hi = 0;
    if (!s.rest) {
        const int first = KEYS ? first_query(s, row) : first_key(p, s, row), last = KEYS ? last_query(p, s, row + rows - 1) : min(s.lk - 1, last_key(s, row + rows - 1));
        if (last >= first) lo = first / BN, hi = last / BN + 1;
    }
    const int per_head = hi - lo, NT = per_head * heads;
    auto tile_row = [&](int i) { return (lo + i % per_head) * BN; };
    auto tail = [&](int i) { return tile_row(i) + BN > streamed; };
    const uint32_t base = (tc::smem_addr(raw) + 1023u) & ~1023u, ring0 = base + 2 * L::RES, ring1 = ring0 + L::N0 * L::STR;
    unsigned char* mem = raw + (base - tc::smem_addr(raw));
    if (NT > 0) {
        if (warp == 8) tc::tmem_alloc(&sh.tmem, 512);
        if (tid == 0) {
            for (int i = 0; i < 3; ++i) {
                tc::mbar_init(&sh.full0[i], 1);
                tc::mbar_init(&sh.empty0[i], 1);
                tc::mbar_init(&sh.full1[i], 1);
                tc::mbar_init(&sh.empty1[i], 1);
            }
            tc::mbar_init(&sh.res_full, 1);
            tc::mbar_init(&sh.s_ready, 1);
            tc::mbar_init(&sh.p_ready, 8);
            tc::mbar_init(&sh.dp_ready, 1);
            tc::mbar_init(&sh.ds_ready, 8);
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(&sh.stat_full[i], 1);
                tc::mbar_init(&sh.stat_empty[i], 8);
            }
            for (int i = 0; i < 4; ++i) {
                tc::mbar_init(&sh.issued[i], 1);
                tc::mbar_init(&sh.clean[i], 1);
            }
            tc::mbar_init(&sh.done, 1);
            tc::mbar_init(&sh.drain, 1);
            tc::mbar_fence_init();
        }
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
    }
    const uint32_t tmem = sh.tmem;
    bool ok = true;

    if (NT == 0) {
        // nothing meets these rows: zeros below
    } else if (warp == 9) {  // ---- loads
        if (lane == 0) {
            tc::mbar_expect_tx(&sh.res_full, 2 * L::RES);
            for (int c = 0; c < D / 64; ++c) {
                tc::tma_load_3d(mem + c * 16384, &M.res0, &sh.res_full, c * 64, KEYS ? hk : h0, int(res0));
                tc::tma_load_3d(mem + L::RES + c * 16384, &M.res1, &sh.res_full, c * 64, KEYS ? hk : h0, int(res0));
            }
            int tails = 0, n0 = 0, n1 = 0;
            for (int i = 0; i < NT; ++i) {
                const int head = KEYS ? h0 + i / per_head : hk, at = str_at + tile_row(i);
                if (i >= L::N0 && !(ok = bounded_wait(&sh.empty0[i % L::N0], (i / L::N0 - 1) & 1))) break;
                tc::mbar_expect_tx(&sh.full0[i % L::N0], L::STR);
                for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(mem + 2 * L::RES + (i % L::N0) * L::STR + c * (BN * 128), &M.str0, &sh.full0[i % L::N0], c * 64, head, at);
                ++n0;
                if (i >= L::N1 && !(ok = bounded_wait(&sh.empty1[i % L::N1], (i / L::N1 - 1) & 1))) break;
                tc::mbar_expect_tx(&sh.full1[i % L::N1], L::STR);
                for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(mem + 2 * L::RES + (L::N0 + i % L::N1) * L::STR + c * (BN * 128), &M.str1, &sh.full1[i % L::N1], c * 64, head, at);
                ++n1;
                if (tail(i)) tc::mbar_arrive(&sh.issued[tails++ & 3]);
            }
            if (!ok) {  // the copies in flight land before the CTA ends
                for (int i = max(0, n0 - L::N0); i < n0; ++i) bounded_wait(&sh.full0[i % L::N0], (i / L::N0) & 1);
                for (int i = max(0, n1 - L::N1); i < n1; ++i) bounded_wait(&sh.full1[i % L::N1], (i / L::N1) & 1);
                bounded_wait(&sh.res_full, 0);
            }
        }
    } else if (warp == 10) {  // ---- the streamed queries' statistics, and rows behind the sequence
        int tails = 0;
        for (int i = 0; i < NT && ok; ++i) {
            if (KEYS) {
                const int st = i & 1, r0 = tile_row(i);
                if (i >= 2) ok = warp_wait(&sh.stat_empty[st], (i / 2 - 1) & 1);
                if (!ok) break;
                const float2* from = A.stat + (h0 + i / per_head) * A.stat_rows + s.q0;
#pragma unroll
                for (int x = 0; x < BN; x += 32) {
                    const int r = r0 + x + lane;
                    const float2 v = r < s.lq ? from[r] : make_float2(0.f, 0.f);
                    sh.nlse[st][x + lane] = -v.x;
                    sh.ndrop[st][x + lane] = -v.y;
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.stat_full[st]);
            }
            if (tail(i)) {
                ok = warp_wait(&sh.issued[tails & 3], (tails >> 2) & 1);  // from then on the stages' barriers are in this tile's phase
                ok = ok && warp_wait(&sh.full0[i % L::N0], (i / L::N0) & 1) && warp_wait(&sh.full1[i % L::N1], (i / L::N1) & 1);
                if (!ok) break;
                zero_rows<BN, D>(ring0 + (i % L::N0) * L::STR, streamed - tile_row(i));
                if (KEYS) zero_rows<BN, D>(ring1 + (i % L::N1) * L::STR, streamed - tile_row(i));
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.clean[tails & 3]);
                ++tails;
            }
        }
    } else if (warp == 8) {  // ---- products
        {
            const bool el = elected();
            const uint32_t tm = same(tmem);
            const int NTu = same(NT), tail_from = same(per_head - (tail(per_head - 1) ? 1 : 0)), per_u = same(per_head), half_u = same(half);
            constexpr uint32_t IS = tc::make_idesc(128, BN, 0, 0), IO = tc::make_idesc(128, ND, 0, 1);
            auto scores = [&](uint32_t res, uint32_t str, uint32_t to, uint64_t* bar) {
                tc::fence_after_sync();
                const uint64_t a = desc_k<128>(res, 0), b = desc_k<BN>(str, 0);
                if (el) {
#pragma unroll
                    for (int x = 0; x < D; x += 16) tc::mma_bf16(tm + to, step_k<128>(a, x), step_k<BN>(b, x), IS, x > 0);
                    tc::commit(bar);
                }
            };
            // columns [0, CW) of the left operand lie at `from`, the others BN / 2 columns on
            auto sum = [&](uint32_t from, uint32_t str, uint32_t to, bool more) {
                tc::fence_after_sync();
                const uint64_t b = desc_mn<BN>(str + half_u * (ND / 64) * (BN * 128), 0);
                if (el)
#pragma unroll
                    for (int x = 0; x < BN; x += 16) tc::mma_bf16_ta(tm + to, tm + from + (x < CW ? 0 : CW) + (x % CW) / 2, step_mn(b, x), IO, more || x > 0);
            };
            auto s0 = [&](int i) { return ring0 + (i % L::N0) * L::STR; };
            auto s1 = [&](int i) { return ring1 + (i % L::N1) * L::STR; };
            auto first = [&](int i) {
                ok = ok && warp_spin(&sh.full0[i % L::N0], (i / L::N0) & 1);
                if (ok) scores(base, s0(i), L::S, &sh.s_ready);
            };
            auto second = [&](int i) {
                ok = ok && warp_spin(&sh.full1[i % L::N1], (i / L::N1) & 1);
                if (!ok) return;
                scores(base + L::RES, s1(i), L::DP, &sh.dp_ready);
                if (!KEYS && el) tc::commit(&sh.empty1[i % L::N1]);
            };
            int tails = 0;
            ok = warp_spin(&sh.res_full, 0);
            first(0);
            second(0);
            int in_head = 0;
            for (int i = 0; i < NTu && ok; ++i) {
                if (!(ok = warp_spin(&sh.p_ready, i & 1))) break;
                const bool is_tail = in_head >= tail_from;
                if (++in_head == per_u) in_head = 0;
                if (is_tail) {
                    if (!(ok = warp_spin(&sh.clean[tails & 3], (tails >> 2) & 1))) break;
                    ++tails;
                }
                if (KEYS) {
                    sum(L::S, s1(i), L::OUT0, i > 0);
                    if (el) tc::commit(&sh.empty1[i % L::N1]);
                }
                if (i + 1 < NTu) first(i + 1);
                if (!(ok = ok && warp_spin(&sh.ds_ready, i & 1))) break;
                sum(L::DP, s0(i), L::OUT1, i > 0);
                if (el) tc::commit(&sh.empty0[i % L::N0]);
                if (i + 1 < NTu) second(i + 1);
            }
            if (el) tc::commit(ok ? &sh.done : &sh.drain);
            if (!ok) warp_spin(&sh.drain, 0);  // the products in flight end before tensor memory is freed
        }
    }
    if (warp < 8) {  // ---- weights: thread to a row, warpgroup to half of the columns
        const int wg = warp >> 2, r = (warp & 3) * 32 + lane, c0 = wg * CW;
        const uint32_t mine = tmem + (uint32_t(warp & 3) << 21);
        const float zs = p.scale * LOG2E;
        const int at = min(row + r, (KEYS ? s.lk : s.lq) - 1);
        const int from = KEYS ? first_query(s, at) : first_key(p, s, at), to = KEYS ? last_query(p, s, at) : min(last_key(s, at), s.lk - 1);
        uint64_t nlse2 = 0, ndrop2 = 0;
        if (!KEYS && NT > 0) {
            const float2 v = A.stat[h0 * A.stat_rows + s.q0 + at];
            nlse2 = tc::dup2(-v.x);
            ndrop2 = tc::dup2(-v.y);
        }
        const uint64_t zs2 = tc::dup2(zs);
        for (int i = 0; i < NT; ++i) {
            const int st = i & 1, x0 = tile_row(i) + c0, a = from - x0, b = to - x0;  // columns [a, b] count
            const bool masked = __any_sync(0xffffffffu, a > 0 || b < CW - 1);
            if (KEYS && !(ok = warp_wait(&sh.stat_full[st], (i >> 1) & 1))) break;
            if (!(ok = warp_wait(&sh.s_ready, i & 1))) break;
            tc::fence_after_sync();
            float v[CW];
#pragma unroll
            for (int c = 0; c < CW; c += 32) tc::tmem_ld32(mine + L::S + c0 + c, v + c);
            tc::tmem_ld_wait();
            const uint32_t stat_l = tc::smem_addr(&sh.nlse[st][c0]), stat_d = tc::smem_addr(&sh.ndrop[st][c0]);
#pragma unroll
            for (int c = 0; c < CW; c += 4) {
                uint64_t l0 = nlse2, l1 = nlse2;
                if (KEYS) {
                    const float4 x = tc::lds128f(stat_l + c * 4);
                    l0 = tc::pk2(x.x, x.y), l1 = tc::pk2(x.z, x.w);
                }
                float e[4];
                tc::unpk2(tc::ffma2(tc::pk2(v[c], v[c + 1]), zs2, l0), e[0], e[1]);
                tc::unpk2(tc::ffma2(tc::pk2(v[c + 2], v[c + 3]), zs2, l1), e[2], e[3]);
#pragma unroll
                for (int x = 0; x < 4; ++x) v[c + x] = ex2(e[x]);
            }
            uint32_t counted[CW / 32];  // a bit to a column
#pragma unroll
            for (int c = 0; c < CW; c += 32) counted[c / 32] = span_of(a - c, b - c);
            if (masked) {
#pragma unroll
                for (int c = 0; c < CW; ++c)
                    if (!(counted[c / 32] >> (c % 32) & 1)) v[c] = 0.f;
            }
            uint32_t w[CW / 2];
            if (KEYS) {
#pragma unroll
                for (int c = 0; c < CW / 2; ++c) w[c] = tc::pack_bf16(v[2 * c], v[2 * c + 1]);
                if constexpr (CW == 64)
                    tmem_st32u(mine + L::S + c0, w);
                else
                    tc::tmem_st16(mine + L::S + c0, reinterpret_cast<const float*>(w));
                tc::tmem_st_wait();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.p_ready);
            if (!(ok = warp_wait(&sh.dp_ready, i & 1))) break;
            tc::fence_after_sync();
#pragma unroll
            for (int c1 = 0; c1 < CW; c1 += 32) {
                float d[32];
                tc::tmem_ld32(mine + L::DP + c0 + c1, d);
                tc::tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    uint64_t d0 = ndrop2, d1 = ndrop2;
                    if (KEYS) {
                        const float4 x = tc::lds128f(stat_d + (c1 + c) * 4);
                        d0 = tc::pk2(x.x, x.y), d1 = tc::pk2(x.z, x.w);
                    }
                    float e[4];
                    tc::unpk2(tc::fmul2(tc::pk2(v[c1 + c], v[c1 + c + 1]), fadd2(tc::pk2(d[c], d[c + 1]), d0)), e[0], e[1]);
                    tc::unpk2(tc::fmul2(tc::pk2(v[c1 + c + 2], v[c1 + c + 3]), fadd2(tc::pk2(d[c + 2], d[c + 3]), d1)), e[2], e[3]);
                    if (masked) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (!(counted[c1 / 32] >> (c + x) & 1)) e[x] = 0.f;
                    }
                    w[(c1 + c) / 2] = tc::pack_bf16(e[0], e[1]);
                    w[(c1 + c) / 2 + 1] = tc::pack_bf16(e[2], e[3]);
                }
            }
            if constexpr (CW == 64)
                tmem_st32u(mine + L::DP + c0, w);
            else
                tc::tmem_st16(mine + L::DP + c0, reinterpret_cast<const float*>(w));
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&sh.ds_ready);
                if (KEYS) tc::mbar_arrive(&sh.stat_empty[st]);
            }
        }
        if (NT > 0 && ok) {
            ok = warp_wait(&sh.done, 0);
            tc::fence_after_sync();
        }
        // keys: dV by the first warpgroup, dK by the second; queries: half of dQ's columns each
        const bool is_dv = KEYS && wg == 0;
        const int cols = KEYS ? ND : D / 2, col0 = KEYS ? half * ND : wg * cols;
        const uint32_t acc = mine + (is_dv ? L::OUT0 : L::OUT1) + (KEYS ? 0 : col0);
        const float f = is_dv ? 1.f : p.scale;
        const int64_t out = KEYS ? (res0 + r) * p.Hkv + hk : (res0 + r) * p.Hq + h0;
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
            float x[32];
            __syncwarp();
            if (NT > 0 && ok) {
                tc::tmem_ld32(acc + c, x);
                tc::tmem_ld_wait();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
            }
            if (r >= rows) {
            } else if (KEYS && parts > 1) {
                float* to32 = partial + ((int64_t(is_dv ? 0 : 1) * parts + part) * p.total_k * p.Hkv + out) * D + col0 + c;
#pragma unroll
                for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(to32 + e) = make_float4(x[e] * f, x[e + 1] * f, x[e + 2] * f, x[e + 3] * f);
            } else {
                __nv_bfloat16* to16 = static_cast<__nv_bfloat16*>(KEYS ? (is_dv ? A.dv : A.dk) : A.dq) + out * D + col0 + c;
                store_bf16x32(to16, x, f, wide_aligned(to16));
            }
        }
    }
    if (!ok) g_gave_up = 1;
    if (NT > 0) {
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        if (warp == 8) tc::tmem_dealloc(tmem, 512);
    }
}

// dv and dk from the parts' sums, in order; rows that no sequence covers were written by the parts, or are left
__global__ void __launch_bounds__(256) k_prompt_bwd_sum(const PromptArgs A, int parts, const float* partial) {
    const gdn_prompt_problem& p = A.p;
    const int64_t per_row = int64_t(p.Hkv) * p.D / 4, all = p.total_k * per_row;
    const int32_t* cu = p.cu_seqlens_k ? p.cu_seqlens_k : p.cu_seqlens;
    const int64_t lo = cu && !p.clear_rest ? cut(cu[0], 0, p.total_k) * per_row : 0, hi = cu && !p.clear_rest ? cut(cu[p.num_seqs], 0, p.total_k) * per_row : all;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < 2 * all; i += int64_t(gridDim.x) * 256) {
        const bool is_dk = i >= all;
        const int64_t at = is_dk ? i - all : i;
        if (at < lo || at >= hi) continue;
        const float4* from = reinterpret_cast<const float4*>(partial) + (is_dk ? parts * all : 0) + at;
        float4 x = from[0];
        for (int k = 1; k < parts; ++k) {
            const float4 y = from[k * all];
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(is_dk ? A.dk : A.dv) + at * 4) = make_uint2(tc::pack_bf16(x.x, x.y), tc::pack_bf16(x.z, x.w));
    }
}

template <int D, bool KEYS>
cudaError_t pass(const PromptArgs& A, int parts, float* partial, cudaStream_t st) {
    using L = Bwd<D, KEYS>;
    const gdn_prompt_problem& p = A.p;
    const int64_t tiles = tile_numbers(p, KEYS, 128), ctas = tiles * (KEYS ? int64_t(p.Hkv) * parts * L::HALVES : p.Hq);
    if (ctas == 0) return cudaSuccess;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    BwdMaps m;
    const void *q = p.total_q ? A.q : A.k, *g = p.total_q ? A.dO : A.k, *k = p.total_k ? A.k : A.q, *v = p.total_k ? A.v : A.q;  // a side without rows is not read
    const int64_t gs = int64_t(p.Hq) * D;
    const bool made = KEYS ? make_tokens_map(&m.res0, k, D, p.Hkv, p.total_k, p.k_stride, 128) && make_tokens_map(&m.res1, v, D, p.Hkv, p.total_k, p.v_stride, 128) &&
                                 make_tokens_map(&m.str0, q, D, p.Hq, p.total_q, p.q_stride, L::BN) && make_tokens_map(&m.str1, g, D, p.Hq, p.total_q, gs, L::BN)
                           : make_tokens_map(&m.res0, q, D, p.Hq, p.total_q, p.q_stride, 128) && make_tokens_map(&m.res1, g, D, p.Hq, p.total_q, gs, 128) &&
                                 make_tokens_map(&m.str0, k, D, p.Hkv, p.total_k, p.k_stride, L::BN) && make_tokens_map(&m.str1, v, D, p.Hkv, p.total_k, p.v_stride, L::BN);
    if (!made) return cudaErrorInvalidValue;
    cudaError_t e = smem_attr(k_prompt_bwd_tc<D, KEYS>, L::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin(KEYS ? "prompt_attn_dkv" : "prompt_attn_dq", st);
    k_prompt_bwd_tc<D, KEYS><<<unsigned(ctas), L::T, L::SMEM, st>>>(A, m, int(tiles), parts, partial);
    timing_end(st);
    return cudaGetLastError();
}
template <int D>
cudaError_t both(const PromptArgs& A, cudaStream_t st) {
    const int parts = prompt_bwd_parts(A.p);
    float* partial = reinterpret_cast<float*>(A.stat + A.stat_rows * A.p.Hq);
    cudaError_t e = pass<D, true>(A, parts, partial, st);
    if (e != cudaSuccess) return e;
    if (parts > 1 && A.p.total_k > 0) {
        const int64_t blocks = (int64_t(A.p.total_k) * A.p.Hkv * D / 2 + 255) / 256, most = int64_t(16) * sm_count_cached();
        timing_begin("prompt_attn_sum", st);
        k_prompt_bwd_sum<<<unsigned(blocks < most ? blocks : most), 256, 0, st>>>(A, parts, partial);
        timing_end(st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return pass<D, false>(A, 1, nullptr, st);
}

}  // namespace

// How many CTAs share the query heads of a kv-head: the least divisor that gives four CTAs to a multiprocessor (the first
// tiles of keys have the most queries, and one CTA with all of them could take longer than the others together), or all.
int prompt_bwd_parts(const gdn_prompt_problem& p) {
    if (p.dtype != GDN_BF16) return 1;
    const int G = p.Hq / p.Hkv;
    const int64_t ctas = (int64_t(p.total_k) / 128 + 1) * p.Hkv * (p.D == 256 ? 2 : 1), want = int64_t(4) * sm_count_cached();
    for (int n = 1; n < G; ++n)
        if (G % n == 0 && ctas * n >= want) return n;
    return G;
}

cudaError_t launch_prompt_bwd_tc(const PromptArgs& A, cudaStream_t st) { return A.p.D == 64 ? both<64>(A, st) : A.p.D == 128 ? both<128>(A, st) : both<256>(A, st); }

int prompt_bwd_status() { return take_gave_up(); }
cudaError_t prompt_bwd_wait_out(int32_t limit_us, cudaStream_t st) { return launch_wait_out(limit_us, st); }

}  // namespace gdn
