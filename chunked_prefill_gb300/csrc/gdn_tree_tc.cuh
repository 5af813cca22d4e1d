// Attention of drafted trees over a bf16 or 8-bit paged cache on the tensor cores (see gdn_tree.cu).
//
// A CTA has blocks of 128 rows (drafted token, query head), or of 256 as two tiles of 128 that share the loaded keys
// and values (more than 128 rows, up to 128 features), and walks over its part of the list of tiles of 128 cached tokens
// (64 with 256 features).  As in the attention over prompts: S = Q K^T into tensor memory, a warpgroup per tile of rows and
// a thread to a row makes weights of it in place, O += P V with P read from tensor memory, O rescaled only where a
// maximum has grown by more than 2^8.  A row is read twice from tensor memory, once for its maximum, in pieces of 64
// values: the registers are the helping warps' (a piece kept for its weights, with 168 of them: 628 us instead of 540 for 64 sequences of
// up to 16384 tokens, 8 bits).  With two tiles of rows the product begins with the first piece's weights.
// Pages lie anywhere, but their rows are at regular distances: TMA brings pieces of up to 16 tokens (the largest power of
// two that divides the page size), issued by the lanes of one warp, straight into the swizzled tiles that the tensor cores
// read; of 8-bit caches into a ring of their own, from where six warps widen them to bf16 (exactly).  A page number out of
// range is replaced by one past the last, which TMA reads as zeros.  Every piece is a request of its own, some 120 cycles of
// the warp that makes it, so pages whose size has no factor of 16 take longer, odd ones by far: 32 sequences, 400 MB of keys and
// values, 32 / 8 heads of 128, 16 drafted tokens, pages of 16 or 48, 24, 100, 5 or 1 tokens (pieces of 16, 8, 4, 1): bf16 109, 115,
// 143, 387 us; 8 bits, where one warp requests both sides, 206, 264, 382, 1108.  (Copied by cp.async, in 16-byte pieces by 128 to 224
// threads, 32 sequences of up to 8192 tokens took 190 us: a tile's addresses alone kept those threads busy.)
// Where some row masks a token that others see (drafted tokens, the edge of a window) infinite and NaN values are made
// zeros, for a weight of 0 would make NaN of them, and are added at the end to the rows that see them.
// Bound: HBM in the limit, up to some 128 rows to a kv-head with bf16; a tile's chain of requests, scores and weights keeps
// it from that: tree of 16 tokens, 32 sequences of up to 8192, 32 / 8 heads of 128: 127 us, 61 % of HBM's rate.  8 bits and
// 248 rows to a kv-head: the instructions of weights and widening (issue slots half used by 16 warps that wait for
// each other), 64 sequences of up to 16384: 544 us, 25 % of HBM's rate.
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
    // A piece takes the warp that requests it some 120 cycles (tree of 16, 32 sequences, bf16, by one warp: 158 us): keys and values of
    // bf16, whose rows are two pieces or more, by a warp each.
    static constexpr int NLW = E == 1 ? 1 : 2;           // loading warps
    static constexpr int NH = E == 1 ? 6 : 1;            // helping warps: widening; cleaning
    static constexpr int STG = E == 1 ? 3 : 0, STGB = TOK * (D < 128 ? 128 : D);  // 8-bit tiles on their way (a piece begins at 128 bytes)
    static constexpr int FIT = (225280 - QB - STG * STGB) / SLOT, SLOTS = FIT < 8 ? FIT : 8;
    static constexpr int SMEM = 1024 + QB + SLOTS * SLOT + STG * STGB;
    static constexpr int T = 256 + 32 + 32 * (NLW + NH);  // 8 warps of weights, then products, loads, helping ones
    static constexpr int CW = NQ == 2 ? TOK : TOK / 2;   // columns of a thread: with one tile of rows the two warpgroups share them
    static constexpr int PIECE = CW < 64 ? CW : 64;      // of which a thread holds so many at a time
    static constexpr int S = 0, O = 2 * TOK;             // tensor memory columns
    static_assert(SLOTS >= 3 && O + NQ * D <= 512, "");
};
constexpr int CLEAN = 8;  // tiles of values to be cleaned on their way at a time: each holds a place in the ring

struct TreeMaps {
    CUtensorMap k, v, k_new, v_new;
};

struct TreeShared {
    uint64_t p_half[2], full[8], empty[8], stage_full[4], stage_empty[4], issued[CLEAN], clean[CLEAN], q_full, q_empty, s_ready[2], p_ready[2], pv_done[2], o_free, met[4], drain;
    alignas(16) uint32_t counts[8][4];   // which tokens of a cached tile count
    // Of the last pairs (more than the ring holds): which had infinite or NaN values, and of the first two cached tiles and the
    // drafted tokens which tokens, as each helping warp found them.
    int bad_pair[8];
    uint32_t bad[8][3][6][4];
    float shared[2][2][128]; // what a row's two threads tell one another
    uint32_t tmem;
};

// four 8-bit values as two pairs of bf16, exactly, by way of fp16 and fp32 (bits moved to bf16's places and a product with
// 2^120 take a quarter more instructions, and NaN a test for itself)
__device__ __forceinline__ uint32_t widen_pair(uint16_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return tc::pack_bf16(f.x, f.y);
}
__device__ __forceinline__ void widen(uint32_t v, uint32_t& lo, uint32_t& hi) {
    lo = widen_pair(uint16_t(v));
    hi = widen_pair(uint16_t(v >> 16));
}
// the bytes that are NaN, in their uppermost bits
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ void zero_nan(uint32_t v, uint32_t& lo, uint32_t& hi) {
    const uint32_t nan = nan_bytes(v);
    if (nan & 0x80u) lo &= 0xffff0000u;
    if (nan & 0x8000u) lo &= 0xffffu;
    if (nan & 0x800000u) hi &= 0xffff0000u;
    if (nan & 0x80000000u) hi &= 0xffffu;
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

__device__ __forceinline__ void mark(uint32_t (&bad)[4], int row) {
#pragma unroll
    for (int w = 0; w < 4; ++w)
        if (row >> 5 == w) bad[w] |= 1u << (row & 31);
}
// By one of `parts` warps: of a swizzled tile of R rows x D bf16 values, rows outside [from, to) become zeros, and with
// `values` infinite and NaN values of the others too, their rows marked in `bad`.  As clean_tile.
template <int R, int D>
__device__ __forceinline__ void clean_rows(uint32_t tile, int from, int to, int part, int parts, bool values, uint32_t (&bad)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i0 = 8 * part; i0 < R * D / 256; i0 += 8 * parts) {  // 4 rows of 64 columns at a time
        const uint32_t at = tile + i0 * 512 + lane * 16;
        const int row0 = (i0 * 4 + (lane >> 3)) % R;
        uint32_t any = 0;
        if (values) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint4 v = tc::lds128(at + x * 512);
                any |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) | ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
            }
        }
        if (!(any & 0x80008000u) && row0 >= from && row0 + 28 < to) continue;
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
            const int row = row0 + 4 * x;
            const uint4 v = tc::lds128(at + x * 512);
            if (row < from || row >= to) {
                tc::sts128(at + x * 512, make_uint4(0u, 0u, 0u, 0u));
            } else if (values && (bad_pair(v.x) || bad_pair(v.y) || bad_pair(v.z) || bad_pair(v.w))) {
                tc::sts128(at + x * 512, make_uint4(clean_pair(v.x), clean_pair(v.y), clean_pair(v.z), clean_pair(v.w)));
                mark(bad, row);
            }
        }
    }
}

// log_rows: of the pieces of a page that are copied at a time, 2^log_rows rows
template <typename C, int D, int NQ>
__global__ void __launch_bounds__(TreeTc<C, D, NQ>::T, 1) k_tree_tc(const TreeArgs A, const __grid_constant__ TreeMaps M, int log_rows) {
    using L = TreeTc<C, D, NQ>;
    constexpr int TOK = L::TOK, SLOTS = L::SLOTS, NH = L::NH, STG = L::STG ? L::STG : 1;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) TreeShared sh;
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
            tc::mbar_init(&sh.full[i], L::E == 1 ? NH : 1);
            tc::mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&sh.stage_full[i], 1);
            tc::mbar_init(&sh.stage_empty[i], NH);
        }
        for (int i = 0; i < CLEAN; ++i) {
            tc::mbar_init(&sh.issued[i], 1);
            tc::mbar_init(&sh.clean[i], NH);
        }
        tc::mbar_init(&sh.q_full, 8);
        tc::mbar_init(&sh.q_empty, 1);
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&sh.s_ready[b], 1);
            tc::mbar_init(&sh.p_half[b], 4);
            tc::mbar_init(&sh.p_ready[b], NQ == 2 ? 4 : 8);
            tc::mbar_init(&sh.pv_done[b], 1);
        }
        tc::mbar_init(&sh.o_free, 8);
        for (int i = 0; i < 4; ++i) tc::mbar_init(&sh.met[i], 2);
        tc::mbar_init(&sh.drain, 1);
        tc::mbar_fence_init();
        for (int i = 0; i < 8; ++i) sh.bad_pair[i] = -1;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    bool ok = true;

    // Tile `tile` of the pair: where its tokens that count lie in it, whether its values are cleaned of infinities and NaN (and
    // which of sh.bad says of what: -1), and whether anything is to be done about them at all.
    auto bounds = [&](int tile, int& from, int& to, int& which) {
        const int t0 = it.R.base + tile * TOK;
        const bool drafted = tile == it.tiles - 1;
        from = drafted ? 0 : it.R.first - t0;
        to = drafted ? p.T : it.R.len - t0;
        which = drafted ? 2 : p.window > 0 && tile < 2 ? tile : -1;
        return which >= 0 || from > 0 || to < TOK;
    };

    if (warp > 8 && warp < 9 + L::NLW) {  // ---- loads
        const int mine = warp - 9;  // keys or values, where a warp has one of them
        const int log_pieces = (TOK == 128 ? 7 : 6) - log_rows, pieces = 1 << log_pieces;
        int cleaned = 0, tiles = 0;
        if (lane == 0) {
            prefetch_map(&M.k);
            prefetch_map(&M.v);
            prefetch_map(&M.k_new);
            prefetch_map(&M.v_new);
        }
        const int nowhere = int(p.num_pages > 0 ? p.num_pages : 1);
        const bool el = elected();
        while (ok && it.next<L::ROWS, TOK>(A, nb)) {
            const int32_t* table = A.table + it.n * p.table_stride;
            auto page_at = [&](int tile, int piece) {
                const int t = it.R.base + tile * TOK + (piece << log_rows);
                return piece < pieces && tile < it.tiles - 1 && t < it.R.len && t + (1 << log_rows) > it.R.first ? __ldg(table + A.page_div.of(t)) : -1;
            };
            const int hk = same(it.hk);
            int page[4], next[4];  // of this lane's pieces
#pragma unroll
            for (int x = 0; x < 4; ++x) next[x] = page_at(it.begin, lane + 32 * x);
            for (int tile = it.begin; tile < it.end && ok; ++tile, ++tiles) {
                const bool drafted = tile == it.tiles - 1;
#pragma unroll
                for (int x = 0; x < 4; ++x) page[x] = next[x];
                if (tile + 1 < it.end)
#pragma unroll
                    for (int x = 0; x < 4; ++x) next[x] = page_at(tile + 1, lane + 32 * x);
                if (!drafted) {
                    // which tokens count: a lane to a word of 32, which is 2 to 32 pieces of the 32 that one vote covers
                    const int per = 32 >> log_rows, first = lane * per;
                    uint32_t good = 0, word = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t votes = __ballot_sync(0xffffffffu, page[x] >= 0 && page[x] < p.num_pages);
                        if (first >> 5 == x) good = votes;
                    }
                    if (lane < TOK / 32) {
                        for (int y = 0; y < per; ++y)
                            if (good >> ((first + y) & 31) & 1) word |= ((1u << (1 << log_rows)) - 1) << (y << log_rows);
                        const int skip = it.R.first - (it.R.base + tile * TOK + lane * 32), left = it.R.len - (it.R.base + tile * TOK + lane * 32);
                        if (skip > 0) word &= skip < 32 ? 0xffffffffu << skip : 0u;
                        if (left < 32) word &= left > 0 ? 0xffffffffu >> (32 - left) : 0u;
                        if (mine == 0) sh.counts[tiles & 7][lane] = word;
                    }
                }
                __syncwarp();
                for (int value = mine; value < (L::NLW == 2 ? mine + 1 : 2) && ok; ++value) {
                    const int n = 2 * tiles + value, slot = n % SLOTS, st = n % STG;
                    const uint32_t to = ring + slot * L::SLOT;
                    uint64_t* bar = L::E == 1 ? &sh.stage_full[st] : &sh.full[slot];
                    if (L::E == 1 && n >= STG) ok = warp_wait(&sh.stage_empty[st], (n / STG - 1) & 1);
                    if ((L::E == 2 || drafted) && n >= SLOTS) ok = ok && warp_wait(&sh.empty[slot], (n / SLOTS - 1) & 1);
                    if (!ok) break;
                    if (el) tc::mbar_expect_tx(bar, drafted ? L::SLOT : TOK * D * L::E);
                    __syncwarp();
                    if (drafted) {
                        if (lane < D / 64) {
                            const int row = it.n * p.T;
                            tc::tma_load_4d(to + lane * (TOK * 128), value ? &M.v_new : &M.k_new, bar, lane * 64, it.hk, row, 0);
                            if (TOK == 128) tc::tma_load_4d(to + lane * (TOK * 128) + 64 * 128, value ? &M.v_new : &M.k_new, bar, lane * 64, it.hk, p.num_seqs * p.T, 0);  // zeros
                        }
                    } else {
                        // one piece after another by one lane: addresses that differ between the lanes of an instruction cost
                        // a turn of the warp each, 100 cycles (tree of 16, 32 sequences: 163 us)
                        const CUtensorMap* map = value ? &M.v : &M.k;
                        const uint32_t first = L::E == 1 ? stage + st * L::STGB : to, each = D << log_rows, step = L::E == 1 ? (each < 128 ? 128 : each) : 128u << log_rows;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if (32 * x >= pieces) break;
                            const int t = it.R.base + tile * TOK + ((lane + 32 * x) << log_rows), my_in = t - A.page_div.of(t) * p.page_size;
                            const int my_page = page[x] >= 0 && page[x] < p.num_pages ? page[x] : nowhere;
                            const int some = min(32, pieces - 32 * x);
#pragma unroll 1
                            for (int y = 0; y < some; ++y) {
                                const int pg = __shfl_sync(0xffffffffu, my_page, y), in = __shfl_sync(0xffffffffu, my_in, y);
                                const uint32_t at = first + (32 * x + y) * step;
                                if (el) {
                                    if (L::E == 1) {
                                        tc::tma_load_4d(at, map, bar, 0, hk, in, pg);
                                    } else {
#pragma unroll
                                        for (int c = 0; c < D / 64; ++c) tc::tma_load_4d(at + c * (TOK * 128), map, bar, c * 64, hk, in, pg);
                                    }
                                }
                            }
                        }
                    }
                    int from, till, which;
                    if (L::E == 2 && value && bounds(tile, from, till, which)) {
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&sh.issued[cleaned % CLEAN]);
                        ++cleaned;
                    }
                }
            }
        }
        if (!ok) {  // the copies in flight land before the CTA ends
            const int n = 2 * tiles + 2, ringed = L::E == 1 ? STG : SLOTS;
            for (int i = max(0, n - ringed); i < n; ++i) warp_wait(L::E == 1 ? &sh.stage_full[i % STG] : &sh.full[i % SLOTS], (i / ringed) & 1);
        }
    } else if (warp > 8) {  // ---- helping warps
        const int part = warp - 9 - L::NLW, lt = part * 32 + lane;
        int n = 0, cleaned = 0, pair = 0;
        while (ok && it.next<L::ROWS, TOK>(A, nb)) {
            for (int tile = it.begin; tile < it.end && ok; ++tile) {
                const bool drafted = tile == it.tiles - 1;
                int from, to, which;
                const bool some = bounds(tile, from, to, which);
                for (int value = 0; value < 2 && ok; ++value, ++n) {
                    const int slot = n % SLOTS, st = n % STG;
                    const uint32_t at = ring + slot * L::SLOT;
                    uint32_t bad[4] = {};
                    const bool here = value && some;
                    if (L::E == 1) {
                        ok = warp_wait(&sh.stage_full[st], (n / STG) & 1);
                        if (!drafted && n >= SLOTS) ok = ok && warp_wait(&sh.empty[slot], (n / SLOTS - 1) & 1);
                        if (!ok) break;
                        if (drafted) {
                            if (here) clean_rows<TOK, D>(at, from, to, part, NH, which >= 0, bad);
                        } else {
                            // A thread's pieces lie in one place of rows 24 (256 features: 12) apart: both addresses only grow.  (Rows of 64
                            // bytes in pieces of one row have 128 bytes each.)
                            constexpr int CPR = D / 16, STEP = 32 * NH / CPR;
                            static_assert(STEP * CPR == 32 * NH || L::E != 1, "");
                            const int row0 = lt / CPR, pc = lt % CPR, pitch = D == 64 && log_rows == 0 ? 128 : D;
                            uint32_t src = stage + st * L::STGB + row0 * pitch + pc * 16, dst = at + (2 * pc >> 3) * (TOK * 128) + row0 * 128;
                            // The second block of 64 columns takes its pieces' halves the other way round: 8 lanes then write distinct banks.
                            uint32_t lo = ((2 * pc & 7) ^ (row0 & 7)) << 4 ^ (pc & 4 ? 16 : 0), hi = lo ^ 16;
                            const uint32_t swap = pc & 4 ? 8 : 0;
                            // not unrolled further: these warps' code and the weights' share the instruction cache
#pragma unroll 2
                            for (int row = row0; row < TOK; row += STEP, src += STEP * pitch, dst += STEP * 128) {
                                const uint2 v0 = tc::lds64(src + swap), v1 = tc::lds64(src + (swap ^ 8));
                                const uint4 v = make_uint4(v0.x, v0.y, v1.x, v1.y);
                                uint4 a, b;
                                widen(v.x, a.x, a.y);
                                widen(v.y, a.z, a.w);
                                widen(v.z, b.x, b.y);
                                widen(v.w, b.z, b.w);
                                if (here && which >= 0 && (nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w))) {  // the only values without an end
                                    if (row >= from && row < to) mark(bad, row);
                                    zero_nan(v.x, a.x, a.y);
                                    zero_nan(v.y, a.z, a.w);
                                    zero_nan(v.z, b.x, b.y);
                                    zero_nan(v.w, b.z, b.w);
                                }
                                if (here && (row < from || row >= to)) a = b = make_uint4(0u, 0u, 0u, 0u);
                                tc::sts128(dst + lo, a);
                                tc::sts128(dst + hi, b);
                                if (STEP % 8) lo ^= (STEP % 8) << 4, hi ^= (STEP % 8) << 4;  // 4
                            }
                        }
                    } else if (here) {
                        ok = warp_wait(&sh.issued[cleaned % CLEAN], (cleaned / CLEAN) & 1);  // from then on the slot's barrier is in this tile's phase
                        ok = ok && warp_wait(&sh.full[slot], (n / SLOTS) & 1);
                        if (!ok) break;
                        clean_rows<TOK, D>(at, from, to, part, NH, which >= 0, bad);
                    }
                    if (here && which >= 0) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            bad[w] = __reduce_or_sync(0xffffffffu, bad[w]);
                            if (lane == 0) sh.bad[pair & 7][which][part][w] = bad[w];
                        }
                        if (lane == 0 && (bad[0] | bad[1] | bad[2] | bad[3])) sh.bad_pair[pair & 7] = pair;
                    }
                    if (L::E == 1 || here) {
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (L::E == 1) {
                                tc::mbar_arrive(&sh.full[slot]);
                                tc::mbar_arrive(&sh.stage_empty[st]);
                            } else {
                                tc::mbar_arrive(&sh.clean[cleaned % CLEAN]);
                            }
                        }
                        ++cleaned;
                    }
                }
            }
            ++pair;
        }
    } else if (warp == 8) {  // ---- products
        {
            const bool el = elected();
            const uint32_t tm = same(tmem);
            constexpr uint32_t IS = tc::make_idesc(128, TOK, 0, 0), IO = tc::make_idesc(128, D, 0, 1);
            int g = 0, pair = 0, cleaned = 0;  // tiles and pairs before, tiles of values cleaned
            while (ok && it.next<L::ROWS, TOK>(A, nb)) {
                const int nt = same(it.end - it.begin);
                auto slot_at = [&](int i, int value) { return ring + (2 * (g + i) + value) % SLOTS * L::SLOT; };
                auto full = [&](int i, int value) {
                    const int n = 2 * (g + i) + value;
                    return ok = ok && warp_spin(&sh.full[n % SLOTS], (n / SLOTS) & 1);
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
                    ok = ok && warp_spin(NQ == 2 ? &sh.p_half[buf] : &sh.p_ready[buf], (NQ == 2 ? g + i : (g + i) >> 1) & 1);
                    if (i == 0 && w == 0 && pair > 0) ok = ok && warp_spin(&sh.o_free, (pair - 1) & 1);
                    if (!full(i, 1)) return;
                    if (L::E == 2 && w == 0) {
                        int from, to, which;
                        if (bounds(it.begin + i, from, to, which)) {
                            ok = warp_spin(&sh.clean[cleaned % CLEAN], (cleaned / CLEAN) & 1);
                            ++cleaned;
                        }
                    }
                    if (!ok) return;
                    const uint64_t b = desc_mn<TOK>(slot_at(i, 1), 0);
                    constexpr int FIRST = NQ == 2 ? TOK / 2 : TOK;  // with two tiles of rows the weights come in two halves
                    auto product = [&](int from) {
                        tc::fence_after_sync();
                        if (el)
#pragma unroll
                            for (int x = 0; x < FIRST; x += 16)
                                tc::mma_bf16_ta(tm + L::O + w * D, tm + L::S + buf * TOK + (from + x) / L::PIECE * L::PIECE + (from + x) % L::PIECE / 2, step_mn(b, from + x), IO, i > 0 || from + x > 0);
                    };
                    product(0);
                    if (NQ == 2) {
                        if (!(ok = warp_spin(&sh.p_ready[buf], (g + i) & 1))) return;
                        product(FIRST);
                    }
                    if (el) tc::commit(&sh.pv_done[buf]);
                    if (w == NQ - 1) release(i, 1);
                };
                ok = warp_spin(&sh.q_full, pair & 1);
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
                warp_spin(&sh.drain, 0);
            }
        }
    } else {  // ---- weights: thread to a row
        // A thread has a row: with two tiles of rows all of its columns, with one the half of its warpgroup; the row's two
        // threads then exchange maxima, and at the end sums.
        const int wg = warp >> 2, w = NQ == 2 ? wg : 0, half = NQ == 2 ? 0 : wg, lane_row = tid & 127, my_row = NQ == 2 ? tid : lane_row;
        const uint32_t mine = tmem + (uint32_t(warp & 3) << 21);
        constexpr int CW = L::CW, PIECE = L::PIECE;
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
        // The queries of a pair, when the scores of the one before are made.
        auto load_queries = [&](const Pairs& x, int before) {
            if (before > 0) ok = ok && warp_wait(&sh.q_empty, (before - 1) & 1);
            constexpr int CPR = D / 8;
#pragma unroll 4
            for (int i = tid; i < L::ROWS * CPR && ok; i += 256) {
                const int row = i / CPR, pc = i % CPR, r = x.r0 + row, t = r / G;
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (r < all_rows) q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(A.q) + (int64_t(x.n) * p.T + t) * p.q_stride + int64_t(x.hk * G + r - t * G) * D + pc * 8);
                tc::sts128(q_at + (row >> 7) * (128 * D * 2) + (pc >> 3) * 16384 + (row & 127) * 128 + (((pc & 7) ^ (row & 7)) << 4), q);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.q_full);
        };
        Pairs ahead = it;
        ahead.next<L::ROWS, TOK>(A, nb);
        load_queries(ahead, 0);
        while (ok && it.next<L::ROWS, TOK>(A, nb)) {
            const int r = it.r0 + my_row, t = r / G, nt = it.end - it.begin;
            // what this row's drafted token attends to
            uint64_t sees = 0;
            int depth = -1;
            if (r < all_rows) read_token(A, it.n, t, sees, depth);
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
                const uint4 counted_all = *reinterpret_cast<const uint4*>(sh.counts[at_tile & 7]);
                const uint32_t all = TOK == 128 ? counted_all.x & counted_all.y & counted_all.z & counted_all.w : counted_all.x & counted_all.y;
                const bool some_masked = __any_sync(0xffffffffu, drafted || all != 0xffffffffu || first > it.R.base + tile * TOK);
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
                        // columns [c, c + 2) of a piece's weights in place of its scores' column c / 2
                        tc::tmem_st16(at + PIECE * x + y / 2, wts);
                    }
                    tc::tmem_st_wait();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(x + 1 < CW / PIECE ? &sh.p_half[buf] : &sh.p_ready[buf]);  // the product begins with the first half
                }
                float a, b;
                tc::unpk2(fadd2(sum[0], sum[1]), a, b);
                l += a + b;
            }
            if (ok && ahead.next<L::ROWS, TOK>(A, nb)) load_queries(ahead, pair + 1);
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
            const bool any_bad = sh.bad_pair[pair & 7] == pair;  // written before the last product
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
                        // of the tiles that this CTA has
                        if (which == 2 ? it.end < it.tiles : !(p.window > 0 && which >= it.begin && which < it.end && which < it.tiles - 1)) continue;
                        uint32_t bits = 0;
                        for (int h = 0; h < NH; ++h) bits |= sh.bad[pair & 7][which][h][token >> 5];
                        if (!(bits >> (token & 31) & 1)) continue;
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
    const gdn_tree_problem& p = A.p;
    int log_rows = 0;
    while (log_rows < 4 && p.page_size % (2 << log_rows) == 0) ++log_rows;
    TreeMaps m;
    const int64_t rows = int64_t(p.num_seqs) * p.T;
    const bool none = p.num_pages == 0 || !A.k_cache || !A.v_cache;  // read nowhere
    const void *k = none ? A.k_new : A.k_cache, *v = none ? A.v_new : A.v_cache;
    if (!make_pages_map(&m.k, k, L::E, D, none ? 1 : p.Hkv, none ? 1 : p.page_size, none ? 1 : p.num_pages, p.k_head_stride, p.k_token_stride, p.k_page_stride, 1 << log_rows) ||
        !make_pages_map(&m.v, v, L::E, D, none ? 1 : p.Hkv, none ? 1 : p.page_size, none ? 1 : p.num_pages, p.v_head_stride, p.v_token_stride, p.v_page_stride, 1 << log_rows) ||
        !make_pages_map(&m.k_new, A.k_new, 2, D, p.Hkv, int(rows), 1, D, p.k_new_stride, 0, 64) || !make_pages_map(&m.v_new, A.v_new, 2, D, p.Hkv, int(rows), 1, D, p.v_new_stride, 0, 64))
        return cudaErrorInvalidValue;
    cudaError_t e = smem_attr(k_tree_tc<C, D, NQ>, L::SMEM);
    if (e != cudaSuccess) return e;
    timing_begin("tree_attn", st);
    k_tree_tc<C, D, NQ><<<plan.ctas, L::T, L::SMEM, st>>>(A, m, log_rows);
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
