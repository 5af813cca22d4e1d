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
// Tiles of queries go from the last to the first, so that of each sequence those with the most keys come first, all heads
// of one after another, so that neighbours read the same keys; a CTA has one, or takes one after another (see launch_d):
// while one tile's result is written the next one's queries and keys come and its first scores are made.
// Bound: the tensor cores (4 D flops per pair of a query and a key that it attends to); a tile's weights (a max, a
// multiply-add, an exponential, an addition and half a conversion for each of 16384 scores) take about as long as its
// products with 128 features, and longer with 64.  Measured, TFLOP/s: 1 x 32768 tokens, 16 / 4 heads, 128 features
// 2.72 to 2.85 ms, 1545 to 1615; 2 x 8192, 32 / 8, 128 0.80 ms, 1383; 1 x 16384, 32 / 8, 64 1.28 ms, 859; 1 x 16384,
// 16 / 2, 256 1.34 ms, 1646; 2 x 8192, 32 / 8, 128 with a window of 512 0.25 ms, 523.  Short sequences: a tile's setup, masked softmax and end, which do not shrink with its products.
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
    static constexpr int T = NQ * 128 + 128;               // softmax warps, then products, loads, two that clean
    // 384 threads start with 168 registers each: 256 x 208 + 128 x 88 = 384 x 168
    static constexpr int MORE = 208, FEWER = 88;
    static constexpr int O = 256;                          // first column of the accumulators
};
// Tiles with masked keys in them on their way at a time: each holds its values' place in the ring.
constexpr int SPECIAL = 8;

struct Shared {
    uint64_t full[8], empty[8], q_full, q_empty, s_ready[2], p_half[2], p_ready[2], pv_done[2], o_free[2], issued[SPECIAL], clean[SPECIAL], bad_free[2][4], drain;
    uint32_t tmem;
    // Infinite and NaN values of the last four tiles of queries with masked keys, counted by themselves: which of them had any,
    // and of each of its tiles with masked keys which one it is and which keys.  A place is written again when the warps of
    // weights of either half are done with it (bad_free).
    int bad_item[4], bad_tile[4][SPECIAL];
    uint32_t bad[4][SPECIAL][4];
};

// A CTA's key tiles: of query tile w [begin[w], end[w]); all of them [lo, hi).
struct Walk {
    int begin[2], end[2], lo, hi;
    int clean_to, clean_from;  // tiles below and from which on some query of the CTA masks some key (or the tile goes past the keys)
    __device__ __forceinline__ bool special(int j) const { return j < clean_to || j >= clean_from; }
    __device__ __forceinline__ int specials() const { return hi - lo - max(0, min(hi, clean_from) - max(lo, clean_to)); }
    // Whether a record of bad values is kept of it.  With one tile of queries of every one: each has results, for which the next
    // one's products wait, and its queries' place keeps the cleaning within two tiles of them.
    template <int NQ> __device__ __forceinline__ bool recorded() const { return NQ == 2 ? specials() > 0 : lo < hi; }
    __device__ __forceinline__ bool in(int w, int j) const { return w == 0 ? j >= begin[0] && j < end[0] : j >= begin[1] && j < end[1]; }
};
template <int NQ>
__device__ __forceinline__ Walk walk_of(const gdn_prompt_problem& p, const Seq& s, int row) {
    Walk k;
    k.clean_to = (first_key(p, s, row + min(NQ * 128, s.lq - row) - 1) + 127) / 128;
    k.clean_from = max(0, min(last_key(s, row), s.lk - 1) + 1) / 128;
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

// The tiles of queries that a CTA takes in turn.
template <int NQ> struct Items {
    int64_t at, all;
    int tiles;
    Seq s;
    int row, h;
    Walk k;
    __device__ __forceinline__ Items(const gdn_prompt_problem& p, int tiles_) : at(blockIdx.x), all(int64_t(tiles_) * p.Hq), tiles(tiles_) {}
    __device__ __forceinline__ bool next(const gdn_prompt_problem& p) {
        for (; at < all; at += gridDim.x) {
            const int number = int(at / p.Hq);
            if (!find_tile<NQ * 128>(p, false, tiles - 1 - number, s, row)) continue;  // of a sequence those with the most keys first
            h = int(at - int64_t(number) * p.Hq);
            k = walk_of<NQ>(p, s, row);
            at += gridDim.x;
            return true;
        }
        return false;
    }
};

template <int D>
__global__ void __launch_bounds__(Fwd<D>::T, 1)
    k_prompt_fwd_tc(const PromptArgs A, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, int tiles) {
    using L = Fwd<D>;
    constexpr int NQ = L::NQ, NC = L::NC, DC = L::DC, SLOTS = L::SLOTS;
    extern __shared__ unsigned char raw[];
    __shared__ Shared sh;
    const gdn_prompt_problem& p = A.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.Hq / p.Hkv;
    const uint32_t q_at = (tc::smem_addr(raw) + 1023u) & ~1023u, ring = q_at + NQ * L::QT;
    unsigned char* base = raw + (q_at - tc::smem_addr(raw));
    if (warp == NQ * 4) tc::tmem_alloc(&sh.tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            tc::mbar_init(&sh.full[i], 1);
            tc::mbar_init(&sh.empty[i], 1);
        }
        tc::mbar_init(&sh.q_full, 1);
        tc::mbar_init(&sh.q_empty, 1);
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&sh.s_ready[b], 1);
            tc::mbar_init(&sh.p_half[b], 4);
            tc::mbar_init(&sh.p_ready[b], 4);
            tc::mbar_init(&sh.pv_done[b], 1);
            tc::mbar_init(&sh.o_free[b], 4);
        }
        for (int i = 0; i < SPECIAL; ++i) {
            tc::mbar_init(&sh.issued[i], 1);
            tc::mbar_init(&sh.clean[i], 2);
        }
        for (int i = 0; i < 4; ++i)
            for (int w = 0; w < 2; ++w) tc::mbar_init(&sh.bad_free[w][i], 4);
        tc::mbar_init(&sh.drain, 1);
        tc::mbar_fence_init();
        for (int i = 0; i < 4; ++i) sh.bad_item[i] = -1;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    bool ok = true;
    Items<NQ> it(p, tiles);
    const Walk& k = it.k;
    const Seq& s = it.s;

    if (NQ == 2 && warp >= NQ * 4) fewer_registers<L::FEWER>();
    if (warp == NQ * 4 + 1) {  // ---- loads
        if (lane == 0) {
            prefetch_map(&qm);
            prefetch_map(&km);
            prefetch_map(&vm);
        }
        int n = 0, specials = 0, item = 0;  // pieces, special tiles of values, tiles of queries so far
        while (ok && it.next(p)) {
            if (k.lo >= k.hi) continue;
            if (lane == 0) {
                const int hk = it.h / G;
                if (item > 0) ok = bounded_wait(&sh.q_empty, (item - 1) & 1);
                if (ok) {
                    tc::mbar_expect_tx(&sh.q_full, NQ * L::QT);
                    for (int w = 0; w < NQ; ++w)
                        for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(base + w * L::QT + c * 16384, &qm, &sh.q_full, c * 64, it.h, s.q0 + it.row + w * 128);
                    in_order<NQ>(k, [&](bool value, int j) {
                        for (int c = 0; c < NC; ++c, ++n) {
                            const int slot = n % SLOTS;
                            if (n >= SLOTS && !bounded_wait(&sh.empty[slot], (n / SLOTS - 1) & 1)) return ok = false;
                            tc::mbar_expect_tx(&sh.full[slot], L::PIECE);
                            for (int b = 0; b < DC / 64; ++b)
                                tc::tma_load_3d(base + NQ * L::QT + slot * L::PIECE + b * 16384, value ? &vm : &km, &sh.full[slot], c * DC + b * 64, hk, s.k0 + j * 128);
                        }
                        if (value && k.special(j)) tc::mbar_arrive(&sh.issued[specials++ % SPECIAL]);
                        return true;
                    });
                    if (!ok) bounded_wait(&sh.q_full, item & 1);
                }
                if (!ok)  // the copies in flight land before the CTA ends
                    for (int i = n < SLOTS ? 0 : n - SLOTS; i < n; ++i) bounded_wait(&sh.full[i % SLOTS], (i / SLOTS) & 1);
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            ++item;
        }
    } else if (warp >= NQ * 4 + 2) {  // ---- cleaning: half of the rows each
        const int half = warp - (NQ * 4 + 2);
        int n0 = 0, done = 0, record = 0;
        uint32_t used = 0, odd = 0;  // a bit to a half and a place: whether it was used, and whether an odd number of times
        while (ok && it.next(p)) {
            if (k.lo >= k.hi) continue;
            // A place is free when the halves that used it are done with it.  The products do not see to that: a tile of queries
            // of which one half has no rows, or sees no key, waits for the other half's results alone, and the warps of this one
            // may be several tiles behind, or ahead.  A half uses the places of the records in which it sees keys; it cannot be done
            // with one before its tiles are cleaned here, so no phase is passed over.
            if (NQ == 2 && k.recorded<NQ>()) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t bit = 1u << (w * 4 + (record & 3));
                    if (ok && (used & bit)) ok = warp_wait(&sh.bad_free[w][record & 3], odd & bit ? 0 : 1);
                    if (k.end[w] > k.begin[w]) used |= bit, odd ^= bit;
                }
                if (!ok) break;
            }
            int nth = 0;
            for (int j = k.lo; j < k.hi && ok; ++j) {
                if (!k.special(j)) continue;
                uint32_t bad[2] = {};
                ok = warp_wait(&sh.issued[done % SPECIAL], (done / SPECIAL) & 1);  // from then on the slots' barriers are in these pieces' phase
                for (int c = 0; c < NC && ok; ++c) {
                    const int n = n0 + place_in_ring<NQ>(k, true, j) * NC + c, slot = n % SLOTS;
                    ok = warp_wait(&sh.full[slot], (n / SLOTS) & 1);
                    if (ok) clean_tile<DC>(ring + slot * L::PIECE, s.lk - j * 128, half, bad);
                }
                if (lane == 0 && nth < SPECIAL) {
                    const int at = record & 3;  // (a tile of queries has 6 at most, 3 at either end of the keys that it sees)
                    sh.bad_tile[at][nth] = j;
                    sh.bad[at][nth][2 * half] = bad[0];
                    sh.bad[at][nth][2 * half + 1] = bad[1];
                    if (bad[0] | bad[1]) sh.bad_item[at] = record;
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.clean[done % SPECIAL]);
                ++done;
                ++nth;
            }
            n0 += 2 * (k.hi - k.lo) * NC;
            record += k.recorded<NQ>();
        }
    } else if (warp == NQ * 4) {  // ---- products
        constexpr uint32_t IS = tc::make_idesc(128, 128, 0, 0), IO = tc::make_idesc(128, DC, 0, 1);
        int n0 = 0, cleaned = 0, item = 0, count[2] = {0, 0}, uses[2] = {0, 0};  // pieces; per query tile: key tiles, tiles of queries
        const bool el = elected();
        const uint32_t tm = same(tmem);
        // the next tile of queries that sees any keys
        auto next = [&] {
            while (it.next(p))
                if (it.k.lo < it.k.hi) return true;
            return false;
        };
        bool more = next();
        while (ok && more) {
            Walk k;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                k.begin[w] = same(it.k.begin[w]);
                k.end[w] = same(it.k.end[w]);
            }
            k.lo = same(it.k.lo);
            k.hi = same(it.k.hi);
            k.clean_to = same(it.k.clean_to);
            k.clean_from = same(it.k.clean_from);
            {
                // The pieces are used in the ring's order.
                struct Place {
                    int slot;
                    uint32_t phase;
                    __device__ __forceinline__ void next() {
                        if (++slot == SLOTS) slot = 0, phase ^= 1;
                    }
                };
                auto after = [](Place x) {
                    for (int c = 0; c < NC; ++c) x.next();
                    return x;
                };
                auto release = [&](Place x) {
#pragma unroll
                    for (int c = 0; c < NC; ++c, x.next())
                        if (el) tc::commit(&sh.empty[x.slot]);
                };
                auto scores = [&](int w, Place x, int buf) {
#pragma unroll
                    for (int c = 0; c < NC; ++c, x.next()) {
                        if (!(ok = ok && warp_spin(&sh.full[x.slot], x.phase))) return;
                        tc::fence_after_sync();
                        const uint64_t a = desc_k<128>(q_at + w * L::QT + c * (DC * 256), 0), b = desc_k<128>(ring + x.slot * L::PIECE, 0);
                        if (el)
#pragma unroll
                            for (int y = 0; y < DC; y += 16) tc::mma_bf16(tm + buf * 128, step_k<128>(a, y), step_k<128>(b, y), IS, c > 0 || y > 0);
                    }
                    if (el) tc::commit(&sh.s_ready[buf]);
                };
                // with the accumulator begun (first) only when the last result has been read from it
                auto values = [&](int w, Place x, int buf, uint32_t phase, bool first) {
                    ok = ok && warp_spin(&sh.p_half[buf], phase);
                    if (first && uses[w] > 0) ok = ok && warp_wait(&sh.o_free[w], (uses[w] - 1) & 1);
                    uint64_t b[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c, x.next()) {
                        if (!(ok = ok && warp_spin(&sh.full[x.slot], x.phase))) return;
                        b[c] = desc_mn<128>(ring + x.slot * L::PIECE, 0);
                    }
#pragma unroll
                    for (int half = 0; half < 128; half += 64) {
                        if (half && !(ok = warp_spin(&sh.p_ready[buf], phase))) return;
                        tc::fence_after_sync();
                        if (el)
#pragma unroll
                            for (int c = 0; c < NC; ++c)
#pragma unroll
                                for (int y = half; y < half + 64; y += 16)
                                    tc::mma_bf16_ta(tm + L::O + w * D + c * DC, tm + buf * 128 + y / 2, step_mn(b[c], y), IO, !first || y > 0);
                    }
                    if (el) tc::commit(&sh.pv_done[buf]);
                };
                auto wait_clean = [&](int j) {
                    if (!k.special(j)) return;
                    ok = ok && warp_wait(&sh.clean[cleaned % SPECIAL], (cleaned / SPECIAL) & 1);
                    ++cleaned;
                };
                Place at{n0 % SLOTS, uint32_t(n0 / SLOTS) & 1};
                ok = warp_wait(&sh.q_full, item & 1);
                if (NQ == 2) {
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        if (ok && k.in(w, k.lo)) scores(w, at, w);
                    release(at);
                    at = after(at);
                    if (k.hi - k.lo == 1 && el) tc::commit(&sh.q_empty);
                    more = next();  // while the first weights are made
                    for (int j = k.lo; j < k.hi && ok; ++j) {
                        const Place keys = after(at);
                        wait_clean(j);
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            if (ok && k.in(w, j)) values(w, at, w, (count[w] + j - k.begin[w]) & 1, j == k.begin[w]);
                            if (ok && j + 1 < k.hi && k.in(w, j + 1)) scores(w, keys, w);
                        }
                        release(at);
                        if (j + 1 < k.hi) release(keys);
                        if (j + 2 == k.hi && el) tc::commit(&sh.q_empty);
                        at = after(keys);
                    }
                } else {
                    int c = count[0];  // the tile of keys among all
                    for (int j = k.lo; j < k.lo + 2 && j < k.hi && ok; ++j) {
                        scores(0, at, (c + j - k.lo) & 1);
                        release(at);
                        at = after(at);
                        if (j + 1 == k.hi && el) tc::commit(&sh.q_empty);
                    }
                    more = next();
                    for (int j = k.lo; j < k.hi && ok; ++j, ++c) {
                        wait_clean(j);
                        values(0, at, c & 1, (c >> 1) & 1, j == k.lo);
                        release(at);
                        at = after(at);
                        if (ok && j + 2 < k.hi) {
                            scores(0, at, c & 1);
                            release(at);
                            at = after(at);
                            if (j + 3 == k.hi && el) tc::commit(&sh.q_empty);
                        }
                    }
                }
                if (!ok) {  // the products in flight end before tensor memory is freed
                    if (el) tc::commit(&sh.drain);
                    warp_wait(&sh.drain, 0);
                }
            }
            n0 += 2 * (k.hi - k.lo) * NC;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                count[w] += k.end[w] - k.begin[w];
                uses[w] += k.end[w] > k.begin[w];
            }
            ++item;
        }
    } else {  // ---- softmax: thread to a row
        if (NQ == 2) more_registers<L::MORE>();
        const int w = warp >> 2;
        const uint32_t mine = tmem + (uint32_t(warp & 3) << 21);
        const float zs = p.scale * LOG2E;
        const bool wide = wide_aligned(A.o) && wide_aligned(A.o_rest);
        int count = 0, record = 0;  // key tiles, tiles of queries with masked keys so far
        while (ok && it.next(p)) {
            const int r = it.row + tid, i_row = min(r, s.lq - 1), begin = w == 0 ? k.begin[0] : k.begin[1], steps = (w == 0 ? k.end[0] : k.end[1]) - begin;
            const bool live = r < s.lq;
            const int first = first_key(p, s, i_row), last = min(last_key(s, i_row), s.lk - 1);
            float m = -INFINITY, l = 0.f;
            for (int j = begin; j < begin + steps; ++j) {
                const int i = j - begin, c_at = count + i, buf = NQ == 2 ? w : c_at & 1;
                if (!(ok = warp_wait(&sh.s_ready[buf], NQ == 2 ? c_at & 1 : (c_at >> 1) & 1))) break;
                tc::fence_after_sync();
                const uint32_t at = mine + buf * 128;
                float v[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tc::tmem_ld32(at + c, v + c);
                tc::tmem_ld_wait();
                const int lo = first - j * 128, hi = last - j * 128;
                if (__any_sync(0xffffffffu, lo > 0 || hi < 127)) {
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        const uint32_t counted = span_of(lo - c, hi - c);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(counted >> e & 1)) v[c + e] = -INFINITY;
                    }
                }
                const float top = fmaxf(m, max_of<128>(v) * zs);
                if (__any_sync(0xffffffffu, top > m + 8.f)) {
                    if (i > 0) {
                        const float f = top == -INFINITY ? 1.f : ex2(m - top);
                        const int before = c_at - 1;
                        if (!(ok = warp_wait(&sh.pv_done[NQ == 2 ? w : before & 1], (NQ == 2 ? before : before >> 1) & 1))) break;
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
                    tc::tmem_st_wait();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(c == 0 ? &sh.p_half[buf] : &sh.p_ready[buf]);  // the product begins with the first half
                }
                float a, b;
                tc::unpk2(fadd2(sum[0], sum[1]), a, b);
                l += a + b;
            }
            // While the last product is on its way: all that does not need it.
            const bool some = l > 0.f || l != l;
            const float f = some ? 1.f / l : 0.f;
            const int64_t out = (int64_t(s.q0) + r) * p.Hq + it.h;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16*>(A.o) + out * D, *rest = A.o_rest ? static_cast<__nv_bfloat16*>(A.o_rest) + out * D : nullptr;
            if (live && A.lse) A.lse[out] = some ? (m + log2f(l)) * LN2 : -INFINITY;
            if (ok && steps > 0) {
                // With one query tile the scores run two tiles ahead and the last two products may both be open, or both done:
                // each has a barrier of its own, for a phase that another has followed can no longer be waited for.
                const int end = count + steps - 1;
                ok = warp_wait(&sh.pv_done[NQ == 2 ? w : end & 1], (NQ == 2 ? end : end >> 1) & 1);
                tc::fence_after_sync();
            }
            if (!ok) break;
            // written before the last product
            const bool recorded = k.recorded<NQ>();
            const int bad_tiles = steps > 0 && recorded && sh.bad_item[record & 3] == record ? k.specials() : 0;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float x[32];
                __syncwarp();
                if (steps > 0) {
                    tc::tmem_ld32(mine + L::O + w * D + c, x);
                    tc::tmem_ld_wait();
                }
                if (!some)
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0.f;
#pragma unroll 1
                for (int i = 0; i < min(bad_tiles, SPECIAL); ++i)  // infinite and NaN values that this row sees
#pragma unroll 1
                    for (int t = 0; t < 128; ++t) {
                        const int key = sh.bad_tile[record & 3][i] * 128 + t;
                        if (!(sh.bad[record & 3][i][t >> 5] >> (t & 31) & 1) || key < first || key > last) continue;
                        const __nv_bfloat16* bv = static_cast<const __nv_bfloat16*>(A.v) + (int64_t(s.k0) + key) * p.v_stride + int64_t(it.h / G) * D + c;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float b = to_f(bv[e]);
                            if (!(fabsf(b) < INFINITY)) x[e] += b;
                        }
                    }
                if (live) {
                    store_bf16x32(o + c, x, f, wide);
                    if (rest) {  // what the rounding leaves
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = x[e] * f - to_f(__float2bfloat16_rn(x[e] * f));
                        store_bf16x32(rest + c, x, 1.f, wide);
                    }
                }
            }
            if (steps > 0) {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&sh.o_free[w]);
                    if (NQ == 2 && recorded) tc::mbar_arrive(&sh.bad_free[w][record & 3]);
                }
            }
            count += steps;
            record += recorded;
        }
    }
    if (!ok) g_gave_up = 1;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == NQ * 4) tc::tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_d(const PromptArgs& A, cudaStream_t st) {
    using L = Fwd<D>;
    const gdn_prompt_problem& p = A.p;
    const int64_t tiles = tile_numbers(p, false, L::NQ * 128);
    if (tiles == 0) return cudaSuccess;
    CUtensorMap q, k, v;
    const void* any = A.q;  // no keys: the maps are not used
    if (!make_tokens_map(&q, A.q, D, p.Hq, p.total_q, p.q_stride, 128) || !make_tokens_map(&k, p.total_k ? A.k : any, D, p.Hkv, p.total_k, p.k_stride, 128) ||
        !make_tokens_map(&v, p.total_k ? A.v : any, D, p.Hkv, p.total_k, p.v_stride, 128))
        return cudaErrorInvalidValue;
    cudaError_t e = smem_attr(k_prompt_fwd_tc<D>, L::SMEM);
    if (e != cudaSuccess) return e;
    // One tile of queries to a CTA where sequences are long: the hardware deals CTAs out as others end, more evenly than taking
    // turns does.  Short ones take turns, for the overlap of one tile's end with the next one's begin.  32 / 8 heads, 128 features,
    // turns and one each: 16 x 512 tokens 90 and 105 us, 8 x 2048 296 and 315, 4 x 4096 464 and 474, 2 x 8192 815 and 796,
    // 1 x 32768 (16 / 4) 2862 and 2724; 64 features, 4 x 4096: 384 and 404; 256 features (16 / 2): 413 and 421.
    const int64_t all = tiles * p.Hq, sms = sm_count_cached();
    const bool turns = p.num_seqs == 0 || p.total_k / p.num_seqs <= 4096 || all > 0x7fffffff;  // a grid has 2^31 - 1 CTAs at most
    timing_begin("prompt_attn_fwd", st);
    k_prompt_fwd_tc<D><<<unsigned(turns && all > sms ? sms : all), L::T, L::SMEM, st>>>(A, q, k, v, int(tiles));
    timing_end(st);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_fwd_tc(const PromptArgs& A, cudaStream_t st) { return A.p.D == 64 ? launch_d<64>(A, st) : A.p.D == 128 ? launch_d<128>(A, st) : launch_d<256>(A, st); }

int prompt_fwd_status() { return take_gave_up(); }
cudaError_t prompt_fwd_wait_out(int32_t limit_us, cudaStream_t st) { return launch_wait_out(limit_us, st); }

}  // namespace gdn
