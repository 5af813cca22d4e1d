// Attention of drafted trees over a bf16 or 8-bit paged cache on the tensor cores (see gdn_tree.cu).
//
// A CTA has blocks of 128 rows (drafted token, query head), or of 256 as two tiles of 128 that share the loaded keys
// and values (more than 128 rows, up to 128 features), and walks over its part of the list of tiles of 128 cached tokens
// (64 with 256 features).  As in the attention over prompts: S = Q K^T into tensor memory, a warpgroup per tile of rows and
// a thread to a row makes weights of it in place, O += P V with P read from tensor memory, O rescaled only where a
// maximum has grown by more than 2^8.  A row is read twice from tensor memory, once for its maximum, in pieces of 32
// values: the registers are the loading warps'.
// Pages lie anywhere, so those warps copy rows in 16-byte pieces (cp.async) straight into the swizzled tiles that the
// tensor cores read; of 8-bit caches into a ring of their own, from where every thread widens the pieces it copied
// itself to bf16 (exactly).  Tokens without a page, and those behind the sequence, become zeros.
// Where some row masks a token that others see (drafted tokens, the edge of a window) infinite and NaN values are made
// zeros, for a weight of 0 would make NaN of them, and are added at the end to the rows that see them.
// Bound: HBM, up to some 128 rows to a kv-head with bf16; the tensor cores and the widening beyond.
#pragma once
#include "gdn_attn_tc.cuh"
#include "gdn_tree.cuh"

namespace gdn {
namespace {

template <typename C, int D, int NQ> struct TreeTc {
    static constexpr int E = int(sizeof(C));
    static constexpr int TOK = D == 256 ? 64 : 128;      // tokens of a tile
    static constexpr int ROWS = NQ * 128;
    static constexpr int QB = ROWS * D * 2;              // bytes of the queries
    static constexpr int SLOT = TOK * D * 2;             // of a tile of keys or values
    static constexpr int NL = 224, NLW = NL / 32;        // loading threads, warps: with the others 16 warps, 128 registers a thread
    static constexpr int STG = E == 1 ? 3 : 0, STGB = TOK * D;    // 8-bit tiles on their way
    static constexpr int FIT = (228352 - QB - STG * STGB) / SLOT, SLOTS = FIT < 6 ? FIT : 6;
    static constexpr int LAG = 1;                         // tiles requested ahead of the one handed over
    static constexpr int SMEM = 1024 + QB + SLOTS * SLOT + STG * STGB;
    static constexpr int T = 256 + 32 + NL;               // 8 warps of weights, then products, loads
    static constexpr int CW = NQ == 2 ? TOK : TOK / 2;   // columns of a thread: with one tile of rows the two warpgroups share them
    static constexpr int S = 0, O = 2 * TOK;             // tensor memory columns
    static constexpr int CPR = D * E / 16, PIECES = TOK * CPR, U = (PIECES + NL - 1) / NL;  // 16-byte pieces of a row, of a tile, of a thread at most
    static_assert(SLOTS >= 3 && O + NQ * D <= 512, "");
};

template <int TOK> struct TreeShared {
    uint64_t full[6], empty[6], q_full, q_empty, s_ready[2], p_ready[2], pv_done[2], o_free, met[4], drain;
    int64_t off[2][TOK][2];
    uint32_t counts[8][4];   // which tokens of a cached tile count
    uint32_t bad[4][3][4];   // of the last pairs: tokens of the first two cached tiles and of the drafted ones with bad values
    float shared[2][2][128]; // what a row's two threads tell one another
    uint32_t tmem;
};

// four 8-bit values as two pairs of bf16: sign, exponent and mantissa moved to bf16's places make the value times
// 2^-120; NaN (all of exponent and mantissa set) is put right by widen_nan
__device__ __forceinline__ void widen(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = __byte_perm(v, 0u, 0x1404), b = __byte_perm(v, 0u, 0x3424);  // bytes in the upper halves
    const __nv_bfloat162 up = __nv_bfloat162(__ushort_as_bfloat16(0x7b80), __ushort_as_bfloat16(0x7b80));  // 2^120
    const uint32_t x = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), y = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
    const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), up), q = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), up);
    lo = *reinterpret_cast<const uint32_t*>(&p);
    hi = *reinterpret_cast<const uint32_t*>(&q);
}
// the bytes that are NaN, in their uppermost bits
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ void widen_nan(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t nan = nan_bytes(v);
    if (nan & 0x80u) lo |= 0x00007fffu;
    if (nan & 0x8000u) lo |= 0x7fff0000u;
    if (nan & 0x800000u) hi |= 0x00007fffu;
    if (nan & 0x80000000u) hi |= 0x7fff0000u;
}

// The (sequence, block) pairs of a CTA's part of the list, one after another.
struct Pairs {
    Part P;
    int64_t pos;
    int n, hk, r0, begin, end, tiles;
    TreeRange R;
    template <int ROWS, int TOK> __device__ __forceinline__ bool next(const TreeArgs& A, int nb) {
        if (pos >= P.hi) return false;
        n = P.n;
        const int block = P.head * A.groups + P.group;
        hk = block / nb;
        r0 = (block - hk * nb) * ROWS;
        R = range_of(A, n);
        tiles = R.tiles(TOK);
        begin = P.at;
        end = int(min(int64_t(tiles), P.at + (P.hi - pos)));
        pos += end - begin;
        P.at = 0;
        if (++P.head == A.heads) P.head = 0, ++P.n;
        return true;
    }
};

template <typename C, int D, int NQ>
__global__ void __launch_bounds__(TreeTc<C, D, NQ>::T, 1) k_tree_tc(const TreeArgs A) {
    using L = TreeTc<C, D, NQ>;
    constexpr int TOK = L::TOK, SLOTS = L::SLOTS, NL = L::NL;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) TreeShared<TOK> sh;
    const gdn_tree_problem& p = A.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.Hq / p.Hkv, all_rows = p.T * G, nb = (all_rows + L::ROWS - 1) / L::ROWS;
    tc::pdl_launch_dependents();
    Pairs it;
    it.P = find_part<L::T>(A, TOK, 1);
    it.pos = it.P.lo;
    if (it.P.lo >= it.P.hi) return;
    const uint32_t q_at = (tc::smem_addr(raw) + 1023u) & ~1023u, ring = q_at + L::QB, stage = ring + SLOTS * L::SLOT;
    if (warp == 8) tc::tmem_alloc(&sh.tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            tc::mbar_init(&sh.full[i], L::NLW);
            tc::mbar_init(&sh.empty[i], 1);
        }
        tc::mbar_init(&sh.q_full, L::NLW);
        tc::mbar_init(&sh.q_empty, 1);
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&sh.s_ready[b], 1);
            tc::mbar_init(&sh.p_ready[b], NQ == 2 ? 4 : 8);
            tc::mbar_init(&sh.pv_done[b], 1);
        }
        tc::mbar_init(&sh.o_free, 8);
        for (int i = 0; i < 4; ++i) tc::mbar_init(&sh.met[i], 2);
        tc::mbar_init(&sh.drain, 1);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    bool ok = true;

    if (warp > 8) {  // ---- loads
        const int lt = tid - 288;
        // where piece u of this thread goes: row, piece of the row
        auto row_of = [&](int u) { return (lt + NL * u) / L::CPR; };
        auto piece_of = [&](int u) { return (lt + NL * u) % L::CPR; };
        auto swizzled = [&](uint32_t slot, int row, int pc) { return slot + (pc >> 3) * (TOK * 128) + row * 128 + (((pc & 7) ^ (row & 7)) << 4); };
        auto hand_over = [&](uint64_t* bar) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar);
        };
        // infinite and NaN values out of a piece that has just been read
        auto clean = [&](uint4& x, int row, uint32_t (*bad)[4], int which) {
            if (!(bad_pair(x.x) || bad_pair(x.y) || bad_pair(x.z) || bad_pair(x.w))) return false;
            x = make_uint4(clean_pair(x.x), clean_pair(x.y), clean_pair(x.z), clean_pair(x.w));
            atomicOr(&bad[which][row >> 5], 1u << (row & 31));
            return true;
        };
        int issued = 0, handed = 0, pair = -1, tile_count = -1;
        uint64_t codes = 0;  // of the groups on their way, oldest lowest: 4 bits, 1 + which tile of values to clean; 0: none; + 4: bf16 already; + 8: the pair's queries with them
        uint32_t bads = 0;   // their pairs' places in sh.bad, 2 bits each
        auto finish = [&]() {  // the oldest group
            const int n = handed++, code = int(codes & 15), which = (code & 3) - 1, slot = n % SLOTS;
            uint32_t(*bad)[4] = sh.bad[bads & 3];
            codes >>= 4;
            bads >>= 2;
            const uint32_t to = ring + slot * L::SLOT;
            if (L::E == 1 && !(code & 4)) {
                if (n >= SLOTS && ok) ok = warp_wait(&sh.empty[slot], (n / SLOTS - 1) & 1);
                if (!ok) return;
                // not unrolled further: the loading warps' code and the weights' share the instruction cache (8 times: 450
                // cycles to a piece)
#pragma unroll 2
                for (int u = 0; u < L::U; ++u) {
                    if (u * NL + lt >= L::PIECES) break;
                    const uint4 v = tc::lds128(stage + n % (L::STG ? L::STG : 1) * L::STGB + (u * NL + lt) * 16);
                    uint4 a, b;
                    widen(v.x, a.x, a.y);
                    widen(v.y, a.z, a.w);
                    widen(v.z, b.x, b.y);
                    widen(v.w, b.z, b.w);
                    const uint32_t nan = nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w);
                    if (nan) {
                        widen_nan(v.x, a.x, a.y);
                        widen_nan(v.y, a.z, a.w);
                        widen_nan(v.z, b.x, b.y);
                        widen_nan(v.w, b.z, b.w);
                    }
                    const int row = row_of(u), pc = piece_of(u);
                    tc::sts128(swizzled(to, row, 2 * pc), a);
                    tc::sts128(swizzled(to, row, 2 * pc + 1), b);
                }
            }
            if (which >= 0) {  // this thread's pieces, as it has just written them
                const int pieces = L::E == 1 && !(code & 4) ? L::CPR : D / 8, wide = L::E == 1 && !(code & 4) ? 2 : 1;
#pragma unroll 1
                for (int i = lt; i < TOK * pieces; i += NL)
#pragma unroll 1
                    for (int x = 0; x < wide; ++x) {
                        const int row = i / pieces;
                        const uint32_t at = swizzled(to, row, i % pieces * wide + x);
                        uint4 y = tc::lds128(at);
                        if (clean(y, row, bad, which)) tc::sts128(at, y);
                    }
            }
            if (code & 8) hand_over(&sh.q_full);
            hand_over(&sh.full[slot]);
        };
        auto push = [&](int code) {
            codes |= uint64_t(code) << (4 * (issued - handed));
            bads |= uint32_t(pair & 3) << (2 * (issued - handed));
            ++issued;
        };
        // One loop over all tiles of keys and of values, and one place where a tile is handed over and one where it is
        // requested: the code of both is long, and copies of it would not stay in the instruction cache.
        int page = -1, tile = 0, value = 1;
        bool more = true;
        it.end = 0;
        for (;;) {
            bool first = false, drafted = false;
            if ((value ^= 1) == 0) {
                if (++tile >= it.end) {
                    more = it.next<L::ROWS, TOK>(A, nb);
                    tile = it.begin;
                    if (more) {
                        first = true;
                        ++pair;
                    }
                }
                if (more) {
                    const int32_t* table = A.table + it.n * p.table_stride;
                    auto page_at = [&](int x) {  // of this thread's token
                        const int t = it.R.base + x * TOK + lt;
                        return lt < TOK && x < it.tiles - 1 && t < it.R.len && t >= it.R.first ? __ldg(table + A.page_div.of(t)) : -1;
                    };
                    if (first) {
                        page = page_at(tile);
                        if (lt < 12) sh.bad[pair & 3][lt >> 2][lt & 3] = 0;  // its last use was four pairs ago
                    }
                    ++tile_count;
                    if (tile < it.tiles - 1 && lt < TOK) {
                        const int t = it.R.base + tile * TOK + lt, in = t - A.page_div.of(t) * p.page_size;
                        const bool good = page >= 0 && page < p.num_pages;
                        sh.off[tile_count & 1][lt][0] = good ? page * p.k_page_stride + in * p.k_token_stride + it.hk * p.k_head_stride : -1;
                        sh.off[tile_count & 1][lt][1] = good ? page * p.v_page_stride + in * p.v_token_stride + it.hk * p.v_head_stride : -1;
                        const uint32_t votes = __ballot_sync(0xffffffffu, good);
                        if (lane == 0) sh.counts[tile_count & 7][lt >> 5] = votes;
                    }
                    if (tile + 1 < it.end) page = page_at(tile + 1);
                    tc::named_sync(1, NL);
                }
            }
            drafted = tile == it.tiles - 1;
            const bool queries = value == 1 && tile == it.begin;  // come with the pair's first values
            // How many tiles may be on their way: none at the end, or before drafted tokens' under 8 bits (copied to their
            // place at once); one before the queries of another pair, for their place is free only when the pair before has
            // its last tiles.
            int left = L::LAG;
            if (!more || (drafted && L::E == 1 && value == 0)) {
                left = 0;
                cp_wait<0>();
            } else if (queries && pair > 0) {
                left = 1;
                cp_wait<1>();
            } else {
                cp_wait<L::LAG>();
            }
#pragma unroll 1
            while (issued - handed > left) finish();
            if (!more) break;
            const int n = issued, slot = n % SLOTS, which = !value ? -1 : drafted ? 2 : p.window > 0 && tile < 2 ? tile : -1;
            if (queries && pair > 0 && ok) ok = warp_wait(&sh.q_empty, (pair - 1) & 1);
            if ((L::E == 2 || drafted) && n >= SLOTS && ok) ok = warp_wait(&sh.empty[slot], (n / SLOTS - 1) & 1);
            if (queries && ok) {
                constexpr int CPR = D / 8;
#pragma unroll 2
                for (int i = lt; i < L::ROWS * CPR; i += NL) {
                    const int row = i / CPR, pc = i % CPR, r = it.r0 + row, t = r / G, g = r - t * G;
                    const bool in = r < all_rows;
                    cp_async(q_at + (row >> 7) * (128 * D * 2) + (pc >> 3) * 16384 + (row & 127) * 128 + (((pc & 7) ^ (row & 7)) << 4),
                             static_cast<const __nv_bfloat16*>(A.q) + (in ? (int64_t(it.n) * p.T + t) * p.q_stride + int64_t(it.hk * G + g) * D + pc * 8 : 0), in);
                }
            }
            if (ok && drafted) {
                constexpr int CPR = D / 8;
                const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(value ? A.v_new : A.k_new) + int64_t(it.hk) * D;
                const int64_t stride = value ? p.v_new_stride : p.k_new_stride;
#pragma unroll 4
                for (int i = lt; i < TOK * CPR; i += NL) {
                    const int row = i / CPR, pc = i % CPR;
                    const bool in = row < p.T;
                    cp_async(swizzled(ring + slot * L::SLOT, row, pc), from + (in ? (int64_t(it.n) * p.T + row) * stride + pc * 8 : 0), in);
                }
            } else if (ok) {
                // the addresses first, the copies back to back
                const C* from = static_cast<const C*>(value ? A.v_cache : A.k_cache);
                int64_t off[L::U];
#pragma unroll
                for (int u = 0; u < L::U; ++u) off[u] = u * NL + lt < L::PIECES ? sh.off[tile_count & 1][row_of(u)][value] : -1;
#pragma unroll
                for (int u = 0; u < L::U; ++u) {
                    if (u * NL + lt >= L::PIECES) break;
                    const int row = row_of(u), pc = piece_of(u);
                    const uint32_t to = L::E == 1 ? stage + n % (L::STG ? L::STG : 1) * L::STGB + (u * NL + lt) * 16 : swizzled(ring + slot * L::SLOT, row, pc);
                    cp_async(to, from + (off[u] < 0 ? 0 : off[u] + pc * (16 / L::E)), off[u] >= 0);
                }
            }
            cp_commit();
            push((which >= 0 ? 1 + which : 0) | (drafted ? 4 : 0) | (queries ? 8 : 0));
        }
    } else if (warp == 8) {  // ---- products
        {
            const bool el = elected();
            const uint32_t tm = same(tmem);
            constexpr uint32_t IS = tc::make_idesc(128, TOK, 0, 0), IO = tc::make_idesc(128, D, 0, 1);
            int g = 0, pair = 0;  // tiles and pairs before
            while (ok && it.next<L::ROWS, TOK>(A, nb)) {
                const int nt = same(it.end - it.begin);
                auto slot_at = [&](int i, int value) { return ring + (2 * (g + i) + value) % SLOTS * L::SLOT; };
                auto full = [&](int i, int value) {
                    const int n = 2 * (g + i) + value;
                    return ok = ok && warp_wait(&sh.full[n % SLOTS], (n / SLOTS) & 1);
                };
                auto release = [&](int i, int value) {
                    if (el) tc::commit(&sh.empty[(2 * (g + i) + value) % SLOTS]);
                };
                auto scores = [&](int w, int i) {
                    if (!full(i, 0)) return;
                    tc::fence_after_sync();
                    const int buf = NQ == 2 ? w : (g + i) & 1;
                    const uint64_t a = desc_k<128>(q_at + w * (128 * D * 2), 0), b = desc_k<TOK>(slot_at(i, 0), 0);
                    if (el) {
#pragma unroll
                        for (int x = 0; x < D; x += 16) tc::mma_bf16(tm + L::S + buf * TOK, step_k<128>(a, x), step_k<TOK>(b, x), IS, x > 0);
                        tc::commit(&sh.s_ready[buf]);
                    }
                    if (w == NQ - 1) {
                        release(i, 0);
                        if (i == nt - 1 && el) tc::commit(&sh.q_empty);
                    }
                };
                auto values = [&](int w, int i) {
                    const int buf = NQ == 2 ? w : (g + i) & 1;
                    ok = ok && warp_wait(&sh.p_ready[buf], (NQ == 2 ? g + i : (g + i) >> 1) & 1);
                    if (i == 0 && w == 0 && pair > 0) ok = ok && warp_wait(&sh.o_free, (pair - 1) & 1);
                    if (!full(i, 1)) return;
                    tc::fence_after_sync();
                    const uint64_t b = desc_mn<TOK>(slot_at(i, 1), 0);
                    if (el) {
#pragma unroll
                        for (int x = 0; x < TOK; x += 16)
                            tc::mma_bf16_ta(tm + L::O + w * D, tm + L::S + buf * TOK + x / L::CW * L::CW + x % L::CW / 2, step_mn(b, x), IO, i > 0 || x > 0);
                        tc::commit(&sh.pv_done[buf]);
                    }
                    if (w == NQ - 1) release(i, 1);
                };
                ok = warp_wait(&sh.q_full, pair & 1);
                if (NQ == 2) {
                    for (int w = 0; w < NQ && ok; ++w) scores(w, 0);
                    for (int i = 0; i < nt && ok; ++i)
                        for (int w = 0; w < NQ && ok; ++w) {
                            values(w, i);
                            if (ok && i + 1 < nt) scores(w, i + 1);
                        }
                } else {
                    for (int i = 0; i < 2 && i < nt && ok; ++i) scores(0, i);
                    for (int i = 0; i < nt && ok; ++i) {
                        values(0, i);
                        if (ok && i + 2 < nt) scores(0, i + 2);
                    }
                }
                g += nt;
                ++pair;
            }
            if (!ok) {  // the products in flight end before tensor memory is freed
                if (el) tc::commit(&sh.drain);
                warp_wait(&sh.drain, 0);
            }
        }
    } else {  // ---- weights: thread to a row
        // A thread has a row: with two tiles of rows all of its columns, with one the half of its warpgroup; the row's two
        // threads then exchange maxima, and at the end sums.
        const int wg = warp >> 2, w = NQ == 2 ? wg : 0, half = NQ == 2 ? 0 : wg, lane_row = tid & 127, my_row = NQ == 2 ? tid : lane_row;
        const uint32_t mine = tmem + (uint32_t(warp & 3) << 21);
        constexpr int CW = L::CW, PIECE = CW < 64 ? CW : 64;
        int g = 0, pair = 0, met = 0;
        // The other half's value of the row.  A place is written again only after the next exchange, before which the
        // other thread has read it.
        auto exchange = [&](float x) {
            sh.shared[met & 1][half][lane_row] = x;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.met[warp & 3]);
            ok = ok && warp_wait(&sh.met[warp & 3], met & 1);
            return sh.shared[met++ & 1][half ^ 1][lane_row];
        };
        while (ok && it.next<L::ROWS, TOK>(A, nb)) {
            const int r = it.r0 + my_row, t = r / G, nt = it.end - it.begin;
            // what this row's drafted token attends to
            uint64_t sees = 0;
            int depth = -1;
            if (r < all_rows) {
                const int32_t* parents = A.parents + int64_t(it.n) * p.T;
                int at = t;
                while (at >= 0) {
                    ++depth;
                    if (p.window == 0 || depth < p.window) sees |= uint64_t(1) << at;
                    const int up = parents[at];
                    if (up < -1 || up >= at) {
                        sees = 0, depth = -1;
                        break;
                    }
                    at = up;
                }
            }
            // A row without a token goes along unmasked, for a warp with a masked row takes twice as long, and is dropped at the end.
            const bool live = depth >= 0;
            const int first = live ? first_cached(A, it.R, depth) : 0;
            if (!live) sees = ~uint64_t(0);
            const float ks = A.k_scale ? A.k_scale[it.hk] : 1.f, vs = A.v_scale ? A.v_scale[it.hk] : 1.f;
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < nt; ++i) {
                const int tile = it.begin + i, at_tile = g + i, buf = NQ == 2 ? w : at_tile & 1;
                const bool drafted = tile == it.tiles - 1;
                if (!(ok = warp_wait(&sh.s_ready[buf], (NQ == 2 ? at_tile : at_tile >> 1) & 1))) break;
                tc::fence_after_sync();
                const uint32_t at = mine + L::S + buf * TOK + half * CW;
                // which of 32 columns count
                auto see = [&](int x) {
                    const int y = half * (CW / 32) + x;
                    if (drafted) return y < 2 ? uint32_t(sees >> (32 * y)) : 0u;
                    const int skip = first - (it.R.base + tile * TOK + 32 * y);
                    return sh.counts[at_tile & 7][y] & (skip <= 0 ? 0xffffffffu : skip < 32 ? 0xffffffffu << skip : 0u);
                };
                uint32_t all = see(0);
#pragma unroll
                for (int x = 1; x < CW / 32; ++x) all &= see(x);
                const bool some_masked = __any_sync(0xffffffffu, all != 0xffffffffu);
                // a scale of 0 makes all scores alike: so does this one, and masked ones stay infinite
                float zs = p.scale * (drafted ? 1.f : ks) * LOG2E;
                if (zs == 0.f) zs = 1.17549435e-38f;
                const float vf = drafted ? 1.f : vs, none = zs < 0.f ? INFINITY : -INFINITY;
                float v[PIECE];
                auto read = [&](int x) {
#pragma unroll
                    for (int c = 0; c < PIECE; c += 32) tc::tmem_ld32(at + PIECE * x + c, v + c);
                    tc::tmem_ld_wait();
                    if (some_masked) {
#pragma unroll
                        for (int y = 0; y < PIECE; y += 32) {
                            const uint32_t counted = see((PIECE * x + y) / 32);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(counted >> c & 1)) v[y + c] = none;
                        }
                    }
                };
                float top = -INFINITY;
#pragma unroll 1
                for (int x = 0; x < CW / PIECE; ++x) {
                    read(x);
                    float e[4];
                    if (zs < 0.f) {  // a negative scale of the keys: the largest score is the least product's
#pragma unroll
                        for (int c = 0; c < PIECE; ++c) e[c & 3] = c < 4 ? -v[c] : fmaxf(e[c & 3], -v[c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < PIECE; ++c) e[c & 3] = c < 4 ? v[c] : fmaxf(e[c & 3], v[c]);
                    }
                    top = fmaxf(top, fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])));
                }
                if (NQ == 1) top = fmaxf(top, exchange(top));
                top = fmaxf(m, top == -INFINITY ? top : top * fabsf(zs));
                if (__any_sync(0xffffffffu, top > m + 8.f)) {
                    if (i > 0) {
                        const float f = top == -INFINITY ? 1.f : ex2(m - top);
                        if (!(ok = warp_wait(&sh.pv_done[NQ == 2 ? w : (at_tile - 1) & 1], (NQ == 2 ? at_tile - 1 : (at_tile - 1) >> 1) & 1))) break;
                        tc::fence_after_sync();
                        constexpr int OW = NQ == 2 ? D : D / 2;  // either warpgroup half of the accumulator's columns
#pragma unroll 1
                        for (int c = 0; c < OW; c += 32) {
                            float x[32];
                            tc::tmem_ld32(mine + L::O + w * D + half * OW + c, x);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] *= f;
                            tc::tmem_st32(mine + L::O + w * D + half * OW + c, x);
                        }
                        l *= f;
                    }
                    m = top;
                }
                const float sub = m == -INFINITY ? 0.f : m;
                const uint64_t zs2 = tc::dup2(zs), sub2 = tc::dup2(-sub), vf2 = tc::dup2(vf);
                uint64_t sum[2] = {0, 0};
#pragma unroll 1
                for (int x = 0; x < CW / PIECE; ++x) {
                    if (CW > PIECE) read(x);
#pragma unroll
                    for (int y = 0; y < PIECE; y += 32) {
                        float wts[16];
#pragma unroll
                        for (int c = y; c < y + 32; c += 2) {
                            float a, b;
                            tc::unpk2(tc::ffma2(tc::pk2(v[c], v[c + 1]), zs2, sub2), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[(c >> 1) & 1] = fadd2(sum[(c >> 1) & 1], tc::pk2(a, b));
                            tc::unpk2(tc::fmul2(tc::pk2(a, b), vf2), a, b);
                            wts[(c - y) / 2] = __uint_as_float(tc::pack_bf16(a, b));
                        }
                        // columns [c, c + 2) of the weights in place of the scores' column c / 2
                        tc::tmem_st16(at + (PIECE * x + y) / 2, wts);
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.p_ready[buf]);
                float a, b;
                tc::unpk2(fadd2(sum[0], sum[1]), a, b);
                l += a + b;
            }
            // With one tile of rows the scores run two tiles ahead and the last two products may both be open, or both done:
            // each has a barrier of its own, for a phase that another has followed can no longer be waited for.
            const int last = g + nt - 1;
            ok = ok && warp_wait(&sh.pv_done[NQ == 2 ? w : last & 1], (NQ == 2 ? last : last >> 1) & 1);
            if (!ok) break;
            tc::fence_after_sync();
            if (NQ == 1) {  // in one order for both
                const float other = exchange(l);
                l = half ? other + l : l + other;
                if (!ok) break;
            }
            const bool whole = it.begin == 0 && it.end == it.tiles, some = live && (l > 0.f || l != l);
            const float f = !whole ? 1.f : some ? 1.f / l : 0.f;
            const int64_t out = (int64_t(it.n) * p.T + t) * p.Hq + it.hk * G + (r - t * G), at = place_of(blockIdx.x, it.begin > 0, L::ROWS) + my_row;
            constexpr int OW = NQ == 2 ? D : D / 2;
            uint32_t any_bad = 0;
#pragma unroll
            for (int x = 0; x < 12; ++x) any_bad |= sh.bad[pair & 3][x >> 2][x & 3];
#pragma unroll 1
            for (int c = half * OW; c < (half + 1) * OW; c += 32) {
                float x[32];
                __syncwarp();
                tc::tmem_ld32(mine + L::O + w * D + c, x);
                tc::tmem_ld_wait();
                if (!some)
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0.f;
                if (any_bad && live)  // infinite and NaN values that this row sees
                    for (int b = 0; b < 3 * TOK; ++b) {
                        const int which = b / TOK, token = b % TOK, cached = it.R.base + which * TOK + token;
                        if (!(sh.bad[pair & 3][which][token >> 5] >> (token & 31) & 1)) continue;
                        if (which < 2 ? cached < first : !(sees >> token & 1)) continue;
                        const int page = which < 2 ? A.table[it.n * p.table_stride + A.page_div.of(cached)] : 0;
                        for (int e = 0; e < 32; ++e) {
                            float y;
                            if (which == 2)
                                y = to_f(static_cast<const __nv_bfloat16*>(A.v_new)[(int64_t(it.n) * p.T + token) * p.v_new_stride + int64_t(it.hk) * D + c + e]);
                            else
                                y = float(static_cast<const C*>(A.v_cache)[page * p.v_page_stride + (cached - A.page_div.of(cached) * p.page_size) * p.v_token_stride + it.hk * p.v_head_stride + c + e]) * vs;
                            if (!(fabsf(y) < INFINITY)) {
#pragma unroll
                                for (int z = 0; z < 32; ++z)
                                    if (z == e) x[z] += y;
                            }
                        }
                    }
                if (r >= all_rows) {
                } else if (whole) {
                    store_bf16x32(static_cast<__nv_bfloat16*>(A.o) + out * D + c, x, f, wide_aligned(A.o));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(A.part + at * D + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                }
            }
            if (r < all_rows && half == 0) {
                if (!whole)
                    A.part_ml[at] = live ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
                else if (A.lse)
                    A.lse[out] = some ? (m + log2f(l)) * LN2 : -INFINITY;
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.o_free);
            g += nt;
            ++pair;
        }
    }
    if (!ok) g_gave_up = 1;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

template <typename C, int D, int NQ>
cudaError_t tree_tc(const TreeArgs& A, const TreePlan& plan, cudaStream_t st) {
    using L = TreeTc<C, D, NQ>;
    cudaError_t e = smem_attr(k_tree_tc<C, D, NQ>, L::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin("tree_attn", st);
    k_tree_tc<C, D, NQ><<<plan.ctas, L::T, L::SMEM, st>>>(A);
    timing_end(st);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_tree_join<__nv_bfloat16, D>(A, plan, st);
}
template <typename C>
cudaError_t tree_tc_type(const TreeArgs& A, const TreePlan& plan, cudaStream_t st) {
    const bool two = plan.rows == 256;
    if (A.p.D == 64) return two ? tree_tc<C, 64, 2>(A, plan, st) : tree_tc<C, 64, 1>(A, plan, st);
    if (A.p.D == 128) return two ? tree_tc<C, 128, 2>(A, plan, st) : tree_tc<C, 128, 1>(A, plan, st);
    return tree_tc<C, 256, 1>(A, plan, st);
}

}  // namespace
}  // namespace gdn
