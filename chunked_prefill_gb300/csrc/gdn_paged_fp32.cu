// Attention over an fp32 paged cache, on the CUDA cores (see gdn_paged.cu).
//
// A warp takes 4 tokens at a time.  LPR = D / 8 lanes share a row, 8 features each (two pieces of 16 bytes, D / 2
// features apart), so that a lane group sums only over LPR lanes: a butterfly in which half of the values change
// lanes each time leaves every score of the 4 tokens and HB query heads in one lane (two with HB = 4), which works
// out its weight; the weights come back by one exchange each.  The groups of a warp (4 with 64 features, 2 with 128)
// keep softmax statistics of their own and meet only at the end.  Products are packed pairs of fp32.
// Rows go through a ring of STAGES steps in shared memory in which every lane copies (cp.async) the very pieces
// that it reads: no barrier, no bank conflict.  The page table is read 8 steps at a time and 8 steps ahead, by the
// lanes for one token each, which also work out where its rows begin: asked for one step ahead the table alone
// made pages of one token 20 to 50 % slower than larger ones.
// Bound: HBM up to some 8 query heads per kv-head, the arithmetic above (a pass over the cache for every 8).
// Measured, of the measured copy bandwidth: 16 sequences of up to 6103 tokens, 32 / 8 heads, 128 features, 62 us
// (5.7 TB/s, 0.85), of up to 12207, 32 / 4, 80 us (0.78); of up to 24414, 32 / 2, 136 us (0.46).  With a lane to
// D / 32 features of every row and 4 heads to a block instead, where the exchanges are half of the instructions,
// these took 73, 144 and 271 us.
#include "gdn_paged.cuh"

namespace gdn {
namespace {

constexpr int PT = 128;   // threads
constexpr int PW = PT / 32;
constexpr int PU = 4;     // tokens a warp takes at a time
constexpr int PTOK = 32;  // tokens to a tile of the list

template <int D, int HB> struct Fp32Tile {
    static constexpr int LPR = D / 8;                            // lanes to a row
    static constexpr int NG = 32 / LPR;                          // groups of lanes: rows side by side
    static constexpr int U = PU / NG;                            // rows of a group at a time
    static constexpr int NV = U * HB;                            // scores of a group at a time
    static constexpr int REP = LPR / NV;                         // lanes that get the same score
    static constexpr int CTAS = HB == 8 || D == 256 ? 2 : 4;     // per multiprocessor
    static constexpr int BYTES = 2 * PU * D * 4;                 // of a warp's step: keys, values
    static constexpr int FIT = 196608 / CTAS / (PW * BYTES), STAGES = FIT < 4 ? FIT : 4;  // more take more time (64 features: 6 of them 5 %)
    static constexpr int RINGS = STAGES * PW * BYTES, JOINED = (PW * NG + 1) * HB * D * 4;  // the groups' accumulators and their sum
    static constexpr int SMEM = RINGS > JOINED ? RINGS : JOINED;
    static_assert(REP >= 1 && STAGES >= 3, "");
};

// N values a lane, summed over 2 W lanes: lane l gets value l / REP of N = 2 W / REP.
template <int W, int N>
__device__ __forceinline__ float spread_sum(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int w = W;
#pragma unroll
    for (int n = N / 2; n > 0; n >>= 1, w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
#pragma unroll
    for (; w > 0; w >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
    return v[0];
}

template <int D, int HB>
__global__ void __launch_bounds__(PT, Fp32Tile<D, HB>::CTAS) k_paged_fp32(const PagedArgs A) {
    using L = Fp32Tile<D, HB>;
    constexpr int LPR = L::LPR, NG = L::NG, U = L::U, NV = L::NV, REP = L::REP, STAGES = L::STAGES;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float ml_s[PW * NG][HB][2];
    __shared__ float2 res_ml[HB];
    float* accs = reinterpret_cast<float*>(smem);  // [PW * NG][HB][D], then a cluster's [HB][D]
    float* res = accs + PW * NG * HB * D;
    const gdn_paged_problem& p = A.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane / LPR, sub = lane % LPR;
    const int G = p.Hq / p.Hkv, nb = (G + HB - 1) / HB;
    // this warp's ring: [stage][row of the group][key, value][piece][lane]
    const uint32_t mem = tc::smem_addr(smem) + warp * STAGES * L::BYTES + lane * 16;
    tc::pdl_launch_dependents();
    Part P = find_part<PT>(A, PTOK, 1);
    const Part P0 = P;
    if (A.cluster > 1 && tid < HB) res_ml[tid] = make_float2(-INFINITY, 0.f);
    for (int64_t pos = P.lo; pos < P.hi;) {
        const int n = P.n, block = P.head * A.groups + P.group, hk = block / nb, hb = (block % nb) * HB;
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

        constexpr int HOP = PW * PU;
        const int first = start + warp * PU;
        // Lane l looks after token l % 4 of step l / 4 of every 8: its page (asked for 8 steps ahead), then where
        // its rows begin.
        int page = 0, steps = 0;
        int64_t ko = 0, vo = 0;
        uint32_t valid8 = 0u;
        auto token = [&] { return first + (steps + (lane >> 2)) * HOP + (lane & (PU - 1)); };
        auto look = [&] {  // -1 where there is nothing to attend to
            const int t = token();
            page = t >= t0 && t < t1 ? table[A.page_div.of(t)] : -1;
        };
        look();
        // Requests the next step's rows (zeros where masked); returns which of its tokens count.
        auto issue = [&](uint32_t to) -> uint32_t {
            if (steps % 8 == 0) {
                const int t = token(), slot = t - A.page_div.of(t) * p.page_size;
                const bool in = page >= 0 && page < p.num_pages;
                valid8 = __ballot_sync(0xffffffffu, in);
                ko = in ? page * p.k_page_stride + slot * p.k_token_stride : 0;
                vo = in ? page * p.v_page_stride + slot * p.v_token_stride : 0;
                steps += 8;
                look();
                steps -= 8;
            }
            const int at = steps % 8 * PU;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = at + u * NG + grp;
                const float* k = kc + __shfl_sync(0xffffffffu, ko, row) + sub * 4;
                const float* v = vc + __shfl_sync(0xffffffffu, vo, row) + sub * 4;
                const bool in = valid8 >> row & 1;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    cp_async(to + ((u * 2 + 0) * 2 + c) * 512, k + c * (D / 2), in);
                    cp_async(to + ((u * 2 + 1) * 2 + c) * 512, v + c * (D / 2), in);
                }
            }
            ++steps;
            return valid8 >> at & ((1u << PU) - 1);
        };
        uint32_t masks = 0u;  // PU bits for each step in flight, oldest first
        static_assert(STAGES * PU <= 32, "a word of masks");
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            if (first + i * HOP < t1) masks |= issue(mem + i * L::BYTES) << (i * PU);
            cp_commit();
        }

        // pairs of features 4 sub + D / 2 (i / 2) + 2 (i % 2)
        uint64_t q[HB][4], acc[HB][4];
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float4 x = hb + h < G ? *reinterpret_cast<const float4*>(static_cast<const float*>(A.q) + n * p.q_stride + int64_t(hk * G + hb + h) * D + sub * 4 + c * (D / 2))
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                q[h][2 * c] = tc::pk2(x.x, x.y), q[h][2 * c + 1] = tc::pk2(x.z, x.w);
                acc[h][2 * c] = acc[h][2 * c + 1] = 0ull;
            }
        const float zs = p.scale * ks * LOG2E;
        // of this lane's head, (sub / REP) % HB; its token is u = sub / REP / HB of the group's U
        float m = -INFINITY, l = 0.f;
        const int mine = sub / REP / HB * NG + grp;
        int stage = 0;
        for (int t = first; t < t1; t += HOP) {
            cp_wait<STAGES - 2>();  // the lane's own copies: no barrier
            {
                const int next = t + (STAGES - 1) * HOP, to = stage == 0 ? STAGES - 1 : stage - 1;
                if (next < t1) masks |= issue(mem + to * L::BYTES) << ((STAGES - 1) * PU);
                cp_commit();
            }
            const uint32_t from = mem + stage * L::BYTES;
            float zv[NV];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint4 a = tc::lds128(from + (u * 2) * 2 * 512), b = tc::lds128(from + ((u * 2) * 2 + 1) * 512);
                const uint64_t k[4] = {uint64_t(a.y) << 32 | a.x, uint64_t(a.w) << 32 | a.z, uint64_t(b.y) << 32 | b.x, uint64_t(b.w) << 32 | b.z};
#pragma unroll
                for (int h = 0; h < HB; ++h) {
                    uint64_t z = tc::fmul2(q[h][0], k[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) z = tc::ffma2(q[h][i], k[i], z);
                    float lo, hi;
                    tc::unpk2(z, lo, hi);
                    zv[u * HB + h] = lo + hi;
                }
            }
            float z = spread_sum<LPR / 2>(zv) * zs;
            if (!(masks >> mine & 1)) z = -INFINITY;
            masks >>= PU;
            float top = z;
#pragma unroll
            for (int o = REP * HB; o < LPR; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (__any_sync(0xffffffffu, top > m)) {
                const float mn = fmaxf(m, top), c = mn == -INFINITY ? 1.f : ex2(m - mn);
                m = mn;
                l *= c;
#pragma unroll
                for (int h = 0; h < HB; ++h) {
                    const uint64_t ch = tc::dup2(__shfl_sync(0xffffffffu, c, h * REP, LPR));
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[h][i] = tc::fmul2(acc[h][i], ch);
                }
            }
            const float w = ex2(z - (m == -INFINITY ? 0.f : m));
            l += w;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint4 a = tc::lds128(from + (u * 2 + 1) * 2 * 512), b = tc::lds128(from + ((u * 2 + 1) * 2 + 1) * 512);
                const uint64_t v[4] = {uint64_t(a.y) << 32 | a.x, uint64_t(a.w) << 32 | a.z, uint64_t(b.y) << 32 | b.x, uint64_t(b.w) << 32 | b.z};
#pragma unroll
                for (int h = 0; h < HB; ++h) {
                    const uint64_t wu = tc::dup2(__shfl_sync(0xffffffffu, w, (u * HB + h) * REP, LPR));
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[h][i] = tc::ffma2(wu, v[i], acc[h][i]);
                }
            }
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }
#pragma unroll
        for (int o = REP * HB; o < LPR; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        cp_wait<0>();
        __syncthreads();  // the rings have been read
        const int part = warp * NG + grp;
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float4 x;
                tc::unpk2(acc[h][2 * c], x.x, x.y);
                tc::unpk2(acc[h][2 * c + 1], x.z, x.w);
                *reinterpret_cast<float4*>(accs + (part * HB + h) * D + sub * 4 + c * (D / 2)) = x;
            }
        if (sub < REP * HB && sub % REP == 0) {
            ml_s[part][sub / REP][0] = m;
            ml_s[part][sub / REP][1] = l;
        }
        __syncthreads();
        const int rows = min(HB, G - hb);
        for (int i = tid; i < rows * (D / 4); i += PT) {
            const int h = i / (D / 4), d = i % (D / 4) * 4;
            float M = -INFINITY, S = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int g = 0; g < PW * NG; ++g) M = fmaxf(M, ml_s[g][h][0]);
#pragma unroll
            for (int g = 0; g < PW * NG; ++g) {
                const float c = ml_s[g][h][0] == -INFINITY ? 0.f : ex2(ml_s[g][h][0] - M);
                const float4 x = *reinterpret_cast<const float4*>(accs + (g * HB + h) * D + d);
                S = fmaf(ml_s[g][h][1], c, S);
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
                *reinterpret_cast<float4*>(static_cast<float*>(A.o) + row * D + d) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
                if (A.lse && d == 0) A.lse[row] = some ? (M + log2f(S)) * LN2 : -INFINITY;
            } else {
                const int64_t at = place_of(blockIdx.x, began, HB) + h;
                *reinterpret_cast<float4*>(A.part + at * D + d) = a;
                if (d == 0) A.part_ml[at] = make_float2(M, S);
            }
        }
        __syncthreads();  // the shared arrays are read before the next pair writes them
    }
    if (A.cluster > 1) {
        const int block = P0.head * A.groups + P0.group, hb = (block % nb) * HB;
        join_cluster<float, D, PT>(A, tc::smem_addr(res), tc::smem_addr(res_ml), P0.n, block / nb, hb, min(HB, G - hb));
    }
}

template <int D, int HB> constexpr PagedShape fp32_shape() { return {PTOK, HB, 1, Fp32Tile<D, HB>::CTAS}; }

template <int D, int HB>
cudaError_t launch_fp32(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    constexpr int SMEM = Fp32Tile<D, HB>::SMEM;
    cudaError_t e = smem_attr(k_paged_fp32<D, HB>, SMEM);
    if (e != cudaSuccess) return e;
    timing_begin("paged_attn", st);
    e = launch_clusters(k_paged_fp32<D, HB>, A, plan.ctas, PT, SMEM, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
    return launch_join<float, D>(A, plan, fp32_shape<D, HB>(), st);
}

// Blocks of 8 query heads where more than 4 share a kv-head: a row of the cache is read once for them.
bool wide(int G) { return G > 4; }
template <int D> PagedShape shape(int G) { return wide(G) ? fp32_shape<D, 8>() : fp32_shape<D, 4>(); }
template <int D> cudaError_t launch(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    return wide(A.p.Hq / A.p.Hkv) ? launch_fp32<D, 8>(A, plan, st) : launch_fp32<D, 4>(A, plan, st);
}

}  // namespace

PagedShape paged_shape_fp32(int D, int G) { return D == 64 ? shape<64>(G) : D == 128 ? shape<128>(G) : shape<256>(G); }
cudaError_t launch_paged_fp32(const PagedArgs& A, const PagedPlan& plan, cudaStream_t st) {
    return A.p.D == 64 ? launch<64>(A, plan, st) : A.p.D == 128 ? launch<128>(A, plan, st) : launch<256>(A, plan, st);
}

}  // namespace gdn
