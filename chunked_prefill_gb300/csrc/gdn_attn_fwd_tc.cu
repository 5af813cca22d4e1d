// Causal attention over prompts in bf16 on the tensor cores (include/gdn.h, gdn_prompt_attn_fwd).
//
// A CTA has 256 queries of one head as two tiles of 128 (one tile with 256 features, whose accumulator takes half
// of tensor memory) and walks over their keys in tiles of 128: S = Q K^T into tensor memory; a warpgroup per query
// tile, a thread to a row, turns it into weights in place (running maximum and sum in registers, no exchange between
// threads); O += P V with P read from tensor memory.  The two query tiles (with 256 features: two key tiles) take
// turns, so that the tensor cores work on one while the other's weights are made.  The accumulator is rescaled only
// where a row's maximum has grown by more than 2^8 since the last time: the weights are then up to 2^8, which bf16
// and the fp32 sums hold as well as 1, and in most tiles O is not touched.
// One warp issues the products, one the TMA loads (a ring of pieces of 128 keys x up to 128 features, keys and values
// in the order in which they are used), one cleans tiles of values in which some query masks some key: a weight of 0
// would make NaN of an infinite value, so rows behind the sequence and infinite or NaN values become zeros there, and
// the latter are added to the rows that see them at the end.
// Tiles are dealt out by descending length, all heads of one after another, so that neighbours read the same keys.
// Bound: the tensor cores (4 D flops per pair); a tile's weights (a max, a multiply-add, an exponential, an addition
// and half a conversion for each of 16384 scores) take about as long as its products with 128 features.
#include "gdn_attn_tc.cuh"

namespace gdn {
namespace {

template <int D> struct Fwd {
    static constexpr int NQ = D == 256 ? 1 : 2;            // query tiles
    static constexpr int DC = D < 128 ? D : 128, NC = D / DC;  // features of a piece, pieces of a tile
    static constexpr int PIECE = 128 * DC * 2;             // bytes
    static constexpr int QT = 128 * D * 2;                 // of a query tile
    static constexpr int SLOTS = D == 64 ? 8 : 5;
    static constexpr int SMEM = 1024 + NQ * QT + SLOTS * PIECE;
    static constexpr int T = NQ * 128 + 96;                // softmax warps, then products, loads, cleaning
    static constexpr int O = 256;                          // first column of the accumulators
};
constexpr int SPECIAL = 8;  // tiles with masked keys in them: at most 3 at either end of the keys seen

struct Shared {
    uint64_t full[8], empty[8], q_full, s_ready[2], p_ready[2], pv_done[2], issued[SPECIAL], clean[SPECIAL], drain;
    uint32_t tmem;
    uint32_t bad[SPECIAL][4];
    int bad_tile[SPECIAL], bad_count;
};

// A CTA's key tiles: of query tile w [begin[w], end[w]); all of them [lo, hi).
struct Walk {
    int begin[2], end[2], lo, hi;
    int row0, rows;  // of the CTA
    __device__ __forceinline__ bool in(int w, int j) const { return j >= begin[w] && j < end[w]; }
};
template <int NQ>
__device__ __forceinline__ Walk walk_of(const gdn_prompt_problem& p, const Seq& s, int row) {
    Walk k;
    k.row0 = row;
    k.rows = min(NQ * 128, s.lq - row);
    k.lo = 0x7fffffff;
    k.hi = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        k.begin[w] = k.end[w] = 0;
        const int first = row + w * 128, rows = min(128, s.lq - first);
        if (w >= NQ || rows <= 0 || s.rest) continue;
        const int last = min(s.lk - 1, last_key(s, first + rows - 1));
        if (last < 0) continue;
        k.begin[w] = first_key(p, s, first) / 128;
        k.end[w] = last / 128 + 1;
        k.lo = min(k.lo, k.begin[w]);
        k.hi = max(k.hi, k.end[w]);
    }
    if (k.lo > k.hi) k.lo = k.hi;
    return k;
}
// Whether some query of the CTA masks some key of tile j (or the tile goes past the keys).
__device__ __forceinline__ bool special(const gdn_prompt_problem& p, const Seq& s, const Walk& k, int j) {
    return j * 128 + 127 > last_key(s, k.row0) || j * 128 + 127 >= s.lk || j * 128 < first_key(p, s, k.row0 + k.rows - 1);
}

// The order of the pieces in the ring: tiles of keys and values as the products need them.  With two query tiles K0 V0
// K1 V1 ..; with one, whose products run a tile further ahead, K0 K1 V0 K2 V1 .. .  Calls f(is_value, tile) in order.
template <int NQ, typename F>
__device__ __forceinline__ void in_order(const Walk& k, F f) {
    if (NQ == 2) {
        for (int j = k.lo; j < k.hi; ++j)
            if (!f(false, j) || !f(true, j)) return;
    } else {
        if (k.lo < k.hi && !f(false, k.lo)) return;
        for (int j = k.lo; j < k.hi; ++j) {
            if (j + 1 < k.hi && !f(false, j + 1)) return;
            if (!f(true, j)) return;
        }
    }
}
// The place of a tile in that order.
template <int NQ>
__device__ __forceinline__ int place_in_ring(const Walk& k, bool value, int j) {
    const int i = j - k.lo, n = k.hi - k.lo;
    if (NQ == 2) return 2 * i + (value ? 1 : 0);
    if (!value) return i == 0 ? 0 : 2 * i - 1;
    return i + 1 < n ? 2 * i + 2 : 2 * i + 1;
}

template <int D>
__global__ void __launch_bounds__(Fwd<D>::T, 1)
    k_prompt_fwd_tc(const PromptArgs A, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, int tiles) {
    using L = Fwd<D>;
    constexpr int NQ = L::NQ, NC = L::NC, DC = L::DC, SLOTS = L::SLOTS;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    const gdn_prompt_problem& p = A.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.Hq, hk = h / (p.Hq / p.Hkv);
    Seq s;
    int row;
    if (!find_tile<NQ * 128>(p, false, tiles - 1 - blockIdx.x / p.Hq, s, row)) return;
    const Walk k = walk_of<NQ>(p, s, row);
    const uint32_t q_at = (tc::smem_addr(raw) + 1023u) & ~1023u, ring = q_at + NQ * L::QT;
    unsigned char* base = raw + (q_at - tc::smem_addr(raw));
    const bool any = k.lo < k.hi;
    if (any) {
        if (warp == NQ * 4) tc::tmem_alloc(&sh.tmem, 512);
        if (tid == 0) {
            for (int i = 0; i < SLOTS; ++i) {
                tc::mbar_init(&sh.full[i], 1);
                tc::mbar_init(&sh.empty[i], 1);
            }
            tc::mbar_init(&sh.q_full, 1);
            for (int b = 0; b < 2; ++b) {
                tc::mbar_init(&sh.s_ready[b], 1);
                tc::mbar_init(&sh.p_ready[b], 4);
                tc::mbar_init(&sh.pv_done[b], 1);
            }
            for (int i = 0; i < SPECIAL; ++i) {
                tc::mbar_init(&sh.issued[i], 1);
                tc::mbar_init(&sh.clean[i], 1);
            }
            tc::mbar_init(&sh.drain, 1);
            tc::mbar_fence_init();
            sh.bad_count = 0;
        }
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
    }
    const uint32_t tmem = sh.tmem;
    bool ok = true;

    if (!any) {
        // nothing to attend to: zeros below
    } else if (warp == NQ * 4 + 1) {  // ---- loads
        if (lane == 0) {
            tc::mbar_expect_tx(&sh.q_full, NQ * L::QT);
            for (int w = 0; w < NQ; ++w)
                for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(base + w * L::QT + c * 16384, &qm, &sh.q_full, c * 64, h, s.q0 + row + w * 128);
            int n = 0, specials = 0;  // pieces, special tiles of values so far
            in_order<NQ>(k, [&](bool value, int j) {
                for (int c = 0; c < NC; ++c, ++n) {
                    const int slot = n % SLOTS;
                    if (n >= SLOTS && !bounded_wait(&sh.empty[slot], (n / SLOTS - 1) & 1)) return ok = false;
                    tc::mbar_expect_tx(&sh.full[slot], L::PIECE);
                    for (int b = 0; b < DC / 64; ++b)
                        tc::tma_load_3d(base + NQ * L::QT + slot * L::PIECE + b * 16384, value ? &vm : &km, &sh.full[slot], c * DC + b * 64, hk, s.k0 + j * 128);
                }
                if (value && special(p, s, k, j)) tc::mbar_arrive(&sh.issued[specials++]);
                return true;
            });
            if (!ok) {  // the copies in flight land before the CTA ends
                for (int i = n < SLOTS ? 0 : n - SLOTS; i < n; ++i) bounded_wait(&sh.full[i % SLOTS], (i / SLOTS) & 1);
                bounded_wait(&sh.q_full, 0);
            }
        }
    } else if (warp == NQ * 4 + 2) {  // ---- cleaning
        int done = 0;
        for (int j = k.lo; j < k.hi && ok; ++j) {
            if (!special(p, s, k, j)) continue;
            uint32_t bad[4] = {};
            ok = warp_wait(&sh.issued[done], 0);  // from then on the slots' barriers are in these pieces' phase
            for (int c = 0; c < NC && ok; ++c) {
                const int n = place_in_ring<NQ>(k, true, j) * NC + c, slot = n % SLOTS;
                ok = warp_wait(&sh.full[slot], (n / SLOTS) & 1);
                if (ok) clean_tile<DC>(ring + slot * L::PIECE, s.lk - j * 128, bad);
            }
            if (lane == 0 && (bad[0] | bad[1] | bad[2] | bad[3]) && sh.bad_count < SPECIAL) {
                const int i = sh.bad_count++;
                sh.bad_tile[i] = j;
                for (int w = 0; w < 4; ++w) sh.bad[i][w] = bad[w];
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.clean[done]);
            ++done;
        }
    } else if (warp == NQ * 4) {  // ---- products
        if (lane == 0) {
            constexpr uint32_t IS = tc::make_idesc(128, 128, 0, 0), IO = tc::make_idesc(128, DC, 0, 1);
            int cleaned = 0;
            auto full = [&](bool value, int j, int c) {
                const int n = place_in_ring<NQ>(k, value, j) * NC + c;
                return ok = ok && bounded_wait(&sh.full[n % SLOTS], (n / SLOTS) & 1);
            };
            auto at = [&](bool value, int j, int c) { return ring + (place_in_ring<NQ>(k, value, j) * NC + c) % SLOTS * L::PIECE; };
            auto release = [&](bool value, int j) {
                for (int c = 0; c < NC; ++c) tc::commit(&sh.empty[(place_in_ring<NQ>(k, value, j) * NC + c) % SLOTS]);
            };
            auto scores = [&](int w, int j, int buf) {
                for (int c = 0; c < NC; ++c) {
                    if (!full(false, j, c)) return;
                    tc::fence_after_sync();
                    const uint32_t a = q_at + w * L::QT + c * (DC * 256), b = at(false, j, c);
#pragma unroll
                    for (int x = 0; x < DC; x += 16) tc::mma_bf16(tmem + buf * 128, desc_k<128>(a, x), desc_k<128>(b, x), IS, c > 0 || x > 0);
                }
                tc::commit(&sh.s_ready[buf]);
            };
            auto values = [&](int w, int j, int buf, bool more) {
                for (int c = 0; c < NC; ++c) {
                    if (!full(true, j, c)) return;
                    tc::fence_after_sync();
                    const uint32_t b = at(true, j, c);
#pragma unroll
                    for (int x = 0; x < 128; x += 16) tc::mma_bf16_ta(tmem + L::O + w * D + c * DC, tmem + buf * 128 + x / 2, desc_mn<128>(b, x), IO, more || x > 0);
                }
                tc::commit(&sh.pv_done[buf]);
            };
            ok = bounded_wait(&sh.q_full, 0);
            if (NQ == 2) {
                for (int w = 0; w < NQ; ++w)
                    if (ok && k.in(w, k.lo)) scores(w, k.lo, w);
                release(false, k.lo);
                for (int j = k.lo; j < k.hi && ok; ++j) {
                    if (special(p, s, k, j)) {
                        ok = bounded_wait(&sh.clean[cleaned], 0);
                        ++cleaned;
                    }
                    for (int w = 0; w < NQ && ok; ++w) {
                        if (k.in(w, j)) {
                            ok = bounded_wait(&sh.p_ready[w], (j - k.begin[w]) & 1);
                            if (ok) values(w, j, w, j > k.begin[w]);
                        }
                        if (ok && j + 1 < k.hi && k.in(w, j + 1)) scores(w, j + 1, w);
                    }
                    release(true, j);
                    if (j + 1 < k.hi) release(false, j + 1);
                }
            } else {
                for (int j = k.lo; j < k.lo + 2 && j < k.hi && ok; ++j) {
                    scores(0, j, (j - k.lo) & 1);
                    release(false, j);
                }
                for (int j = k.lo; j < k.hi && ok; ++j) {
                    const int i = j - k.lo;
                    if (special(p, s, k, j)) {
                        ok = bounded_wait(&sh.clean[cleaned], 0);
                        ++cleaned;
                    }
                    ok = ok && bounded_wait(&sh.p_ready[i & 1], (i >> 1) & 1);
                    if (ok) values(0, j, i & 1, j > k.lo);
                    release(true, j);
                    if (ok && j + 2 < k.hi) {
                        scores(0, j + 2, i & 1);
                        release(false, j + 2);
                    }
                }
            }
            if (!ok) {  // the products in flight end before tensor memory is freed
                tc::commit(&sh.drain);
                bounded_wait(&sh.drain, 0);
            }
        }
    }
    if (warp < NQ * 4) {  // ---- softmax: thread to a row
        const int w = warp >> 2, r = row + tid, i_row = min(r, s.lq - 1);
        const bool live = r < s.lq;
        const int first = first_key(p, s, i_row), last = min(last_key(s, i_row), s.lk - 1);
        const uint32_t mine = tmem + (uint32_t(warp & 3) << 21);
        const float zs = p.scale * LOG2E;
        float m = -INFINITY, l = 0.f;
        for (int j = k.begin[w]; j < k.end[w]; ++j) {
            const int i = j - k.begin[w], buf = NQ == 2 ? w : i & 1;
            if (!(ok = warp_wait(&sh.s_ready[buf], NQ == 2 ? i & 1 : (i >> 1) & 1))) break;
            tc::fence_after_sync();
            const uint32_t at = mine + buf * 128;
            float v[128];
#pragma unroll
            for (int c = 0; c < 128; c += 32) tc::tmem_ld32(at + c, v + c);
            tc::tmem_ld_wait();
            const int lo = first - j * 128, hi = last - j * 128;
            if (__any_sync(0xffffffffu, lo > 0 || hi < 127)) {
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (c < lo || c > hi) v[c] = -INFINITY;
            }
            float t[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int c = 4; c < 128; c += 4)
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = fmaxf(t[e], v[c + e]);
            const float top = fmaxf(m, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * zs);
            if (__any_sync(0xffffffffu, top > m + 8.f)) {
                if (i > 0) {
                    const float f = top == -INFINITY ? 1.f : ex2(m - top);
                    if (!(ok = warp_wait(&sh.pv_done[NQ == 2 ? w : (i - 1) & 1], (NQ == 2 ? i - 1 : (i - 1) >> 1) & 1))) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float x[32];
                        tc::tmem_ld32(mine + L::O + w * D + c, x);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] *= f;
                        tc::tmem_st32(mine + L::O + w * D + c, x);
                    }
                    l *= f;
                }
                m = top;
            }
            const float sub = m == -INFINITY ? 0.f : m;
            const uint64_t zs2 = tc::dup2(zs), sub2 = tc::dup2(-sub);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 128; c += 64) {
                uint32_t w32[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    float a, b;
                    tc::unpk2(tc::ffma2(tc::pk2(v[c + e], v[c + e + 1]), zs2, sub2), a, b);
                    a = ex2(a);
                    b = ex2(b);
                    sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], tc::pk2(a, b));
                    w32[e / 2] = tc::pack_bf16(a, b);
                }
                tmem_st32u(at + c / 2, w32);
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.p_ready[buf]);
            float a, b;
            tc::unpk2(fadd2(sum[0], sum[1]), a, b);
            l += a + b;
        }
        const int steps = k.end[w] - k.begin[w];
        if (ok && steps > 0) {
            // With one query tile the scores run two tiles ahead and the last two products may both be open, or both done:
            // each has a barrier of its own, for a phase that another has followed can no longer be waited for.
            const int l_tile = steps - 1;
            ok = ok && warp_wait(&sh.pv_done[NQ == 2 ? w : l_tile & 1], (NQ == 2 ? l_tile : l_tile >> 1) & 1);
            tc::fence_after_sync();
        }
        const bool some = ok && (l > 0.f || l != l);
        const float f = some ? 1.f / l : 0.f;
        const int64_t out = (int64_t(s.q0) + r) * p.Hq + h;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(A.o) + out * D;
        const int bad_tiles = any ? sh.bad_count : 0;  // written before the last pv_done
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            float x[32];
            __syncwarp();
            if (steps > 0 && ok) {
                tc::tmem_ld32(mine + L::O + w * D + c, x);
                tc::tmem_ld_wait();
            }
            if (!some)
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
            for (int i = 0; i < bad_tiles; ++i)  // infinite and NaN values that this row sees
                for (int t = 0; t < 128; ++t) {
                    const int key = sh.bad_tile[i] * 128 + t;
                    if (!(sh.bad[i][t >> 5] >> (t & 31) & 1) || key < first || key > last) continue;
                    const __nv_bfloat16* bv = static_cast<const __nv_bfloat16*>(A.v) + (int64_t(s.k0) + key) * p.v_stride + int64_t(hk) * D + c;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float b = to_f(bv[e]);
                        if (!(fabsf(b) < INFINITY)) x[e] += b;
                    }
                }
            if (live) {
                store_bf16x16(o + c, x, f);
                store_bf16x16(o + c + 16, x + 16, f);
            }
        }
        if (live && A.lse) A.lse[out] = some ? (m + log2f(l)) * LN2 : -INFINITY;
    }
    if (!ok) g_gave_up = 1;
    if (any) {
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        if (warp == NQ * 4) tc::tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch_d(const PromptArgs& A, cudaStream_t st) {
    using L = Fwd<D>;
    const gdn_prompt_problem& p = A.p;
    const int64_t tiles = tile_numbers(p, false, L::NQ * 128);
    if (tiles == 0) return cudaSuccess;
    if (tiles * p.Hq > 0x7fffffff) return cudaErrorInvalidConfiguration;
    CUtensorMap q, k, v;
    const void* any = A.q;  // no keys: the maps are not used
    if (!make_tokens_map(&q, A.q, D, p.Hq, p.total_q, p.q_stride, 128) || !make_tokens_map(&k, p.total_k ? A.k : any, D, p.Hkv, p.total_k, p.k_stride, 128) ||
        !make_tokens_map(&v, p.total_k ? A.v : any, D, p.Hkv, p.total_k, p.v_stride, 128))
        return cudaErrorInvalidValue;
    cudaError_t e = smem_attr(k_prompt_fwd_tc<D>, L::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin("prompt_attn_fwd", st);
    k_prompt_fwd_tc<D><<<unsigned(tiles * p.Hq), L::T, L::SMEM, st>>>(A, q, k, v, int(tiles));
    timing_end(st);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_fwd_tc(const PromptArgs& A, cudaStream_t st) { return A.p.D == 64 ? launch_d<64>(A, st) : A.p.D == 128 ? launch_d<128>(A, st) : launch_d<256>(A, st); }

int prompt_fwd_status() { return take_gave_up(); }

}  // namespace gdn
