// Attention over prompts and its gradient on the CUDA cores, in fp32 throughout (see include/gdn.h): the tensor cores
// would round products to 10 bits.  Tiles of queries against tiles of keys in shared memory, a running softmax, 4 x 4
// values of a product in a thread's registers; the gradient in two passes, keys and queries, as with bf16.  Bound: the
// fp32 units' instructions and the reads of shared memory between them on long prompts (4 x 2048 tokens, 16 / 4 heads: forward
// 1.09, 2.21 and 4.51 ms with 64, 128 and 256 features, 31 TFLOP/s; gradient 4.2, 7.8 and 22.3 ms, 20, 22 and 15 TFLOP/s of the
// 10 D flops of one pass), latency on short ones (2 x 100 tokens, 8 / 2 heads, 64 features: 10 us a call).
#include "gdn_attn_simt.cuh"

namespace gdn {
namespace {

// ---- forward: a CTA has 16 MI queries of one head, their keys in tiles of 64
template <int D, int MI> constexpr int fwd_smem() { return ((16 * MI + 128) * (D + 4) + 16 * MI * 68) * 4; }

template <int D, int MI>
__global__ void __launch_bounds__(ST) k_prompt_fwd_simt(const PromptArgs A) {
    using T = float;
    constexpr int M = 16 * MI, B = 64, NJ = 4;
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + M * (D + 4), *V = K + B * (D + 4), *P = V + B * (D + 4);
    const gdn_prompt_problem& p = A.p;
    Seq s;
    int row;
    if (!find_tile<M>(p, false, gridDim.x - 1 - blockIdx.x, s, row)) return;  // of a sequence those with the most keys first
    const int h = blockIdx.y, j = h / (p.Hq / p.Hkv), rows = min(M, s.lq - row);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int k_end = s.rest ? 0 : min(s.lk, last_key(s, row + rows - 1) + 1), k_begin = k_end > 0 ? first_key(p, s, row) / B * B : 0;
    load_rows<M, D>(Q, static_cast<const T*>(A.q) + (int64_t(s.q0) + row) * p.q_stride + int64_t(h) * D, p.q_stride, rows);
    float acc[MI][D / 16] = {}, m[MI], l[MI] = {};
    int first[MI], last[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        m[i] = -INFINITY;
        first[i] = first_key(p, s, row + ty + 16 * i);
        last[i] = ty + 16 * i < rows ? last_key(s, row + ty + 16 * i) : -1;
    }
    const float zs = p.scale * LOG2E;
    for (int k0 = k_begin; k0 < k_end; k0 += B) {
        __syncthreads();
        const int keys = min(B, s.lk - k0);
        load_rows<B, D>(K, static_cast<const T*>(A.k) + (int64_t(s.k0) + k0) * p.k_stride + int64_t(j) * D, p.k_stride, keys);
        load_rows<B, D>(V, static_cast<const T*>(A.v) + (int64_t(s.k0) + k0) * p.v_stride + int64_t(j) * D, p.v_stride, keys);
        __syncthreads();
        float z[MI][NJ];
        mul_nt<MI, NJ, D>(z, Q, K);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int n = 0; n < NJ; ++n) {
                const int t = k0 + tx + 16 * n;
                z[i][n] = t >= first[i] && t <= last[i] ? z[i][n] * zs : -INFINITY;
            }
        softmax_step(z, m, l, acc, P);
        __syncthreads();
        const bool whole = rows == M && k0 + B - 1 <= last_key(s, row) && k0 >= first_key(p, s, row + M - 1);
        if (whole)
            mul_add<MI, D, false, false>(acc, B, P, B + 4, V, [](int, int) { return true; });
        else
            mul_add<MI, D, false, true>(acc, min(B, k_end - k0), P, B + 4, V, [&](int i, int n) { return k0 + n >= first[i] && k0 + n <= last[i]; });
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const float sum = row_sum(l[i]);
        if (ty + 16 * i >= rows) continue;
        const bool some = sum > 0.f || sum != sum;
        const float f = some ? 1.f / sum : 0.f;
        const int64_t at = (int64_t(s.q0) + row + ty + 16 * i) * p.Hq + h;
#pragma unroll
        for (int v = 0; v < D / 64; ++v)
            st4(static_cast<T*>(A.o) + at * D + 64 * v + 4 * tx, acc[i][4 * v] * f, acc[i][4 * v + 1] * f, acc[i][4 * v + 2] * f, acc[i][4 * v + 3] * f);
        if (A.lse && tx == 0) A.lse[at] = some ? (m[i] + log2f(sum)) * LN2 : -INFINITY;
    }
}

// ---- the queries' statistics for the gradient, for both types: bound by HBM, three rows read, 256-byte pieces
// of heads apart (8192 tokens, 32 heads of 128, bf16: 44 us, 4.6 TB/s): a block to 64 rows of a head, D / 8 lanes (fp32: D / 4) to a row, so that
// the statistics' rows are written whole
template <typename T, int D>
__global__ void __launch_bounds__(256) k_prompt_stat(const PromptArgs A) {
    constexpr int V = 16 / int(sizeof(T)), LPR = D / V < 32 ? D / V : 32, PER = D / V / LPR, R = 256 / LPR, U = 64 / R;  // rows at a time, times
    const gdn_prompt_problem& p = A.p;
    const int h = blockIdx.x % p.Hq, row0 = int(blockIdx.x / p.Hq) * 64, r = threadIdx.x / LPR, lane = threadIdx.x % LPR;
    // Everything is requested at once: the rows' lse, read when their sums were there, held the kernel at 3.8 TB/s.
    constexpr bool REST = sizeof(T) == 2;
    uint4 o[U * PER], g[U * PER], rest[REST ? U * PER : 1];
    float lse[U], dlse[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = row0 + r + R * u;
        const bool mine = lane == 0 && row < p.total_q;
        lse[u] = mine ? A.lse_in[int64_t(row) * p.Hq + h] : 0.f;
        dlse[u] = mine && A.dlse ? A.dlse[int64_t(row) * p.Hq + h] : 0.f;
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            const int64_t at = (int64_t(row) * p.Hq + h) * D + (x * LPR + lane) * V;
            const bool in = row < p.total_q;
            o[u * PER + x] = in ? *reinterpret_cast<const uint4*>(static_cast<const T*>(A.o_in) + at) : make_uint4(0u, 0u, 0u, 0u);
            g[u * PER + x] = in ? *reinterpret_cast<const uint4*>(static_cast<const T*>(A.dO) + at) : make_uint4(0u, 0u, 0u, 0u);
            if (REST) rest[u * PER + x] = in && A.rest_in ? *reinterpret_cast<const uint4*>(static_cast<const T*>(A.rest_in) + at) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            const T *a = reinterpret_cast<const T*>(&o[u * PER + x]), *b = reinterpret_cast<const T*>(&g[u * PER + x]);
#pragma unroll
            for (int e = 0; e < V; ++e) sum = fmaf(to_f(a[e]), to_f(b[e]), sum);
        }
        if (REST) {
#pragma unroll
            for (int x = 0; x < PER; ++x) {
                const T *a = reinterpret_cast<const T*>(&rest[u * PER + x]), *b = reinterpret_cast<const T*>(&g[u * PER + x]);
#pragma unroll
                for (int e = 0; e < V; ++e) sum = fmaf(to_f(a[e]), to_f(b[e]), sum);
            }
        }
#pragma unroll
        for (int w = LPR / 2; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        const int row = row0 + r + R * u;
        if (lane == 0 && row < p.total_q) A.stat[h * A.stat_rows + row] = make_float2(lse[u] * LOG2E, sum - dlse[u]);
    }
}

// ---- backward.  Tiles of B queries by B keys: P = softmax(z), S its gradient's product with it.
template <int D> struct Back {
    static constexpr int B = D == 256 ? 32 : 64, MI = B / 16;
    static constexpr int SMEM = (4 * B * (D + 4) + 2 * B * (B + 4)) * 4;
};

// P and S of the tile at (queries row .., keys k0 ..) into shared memory; `stat` of the thread's queries.
template <int D>
__device__ __forceinline__ void back_tile(const gdn_prompt_problem& p, const Seq& s, int row, int k0, const float2 (&stat)[Back<D>::MI], const float* Q, const float* K,
                                          const float* G, const float* V, float* P, float* S) {
    constexpr int B = Back<D>::B, MI = Back<D>::MI;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float z[MI][MI], dp[MI][MI];
    mul_nt<MI, MI, D>(z, Q, K);
    mul_nt<MI, MI, D>(dp, G, V);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = row + ty + 16 * i, first = first_key(p, s, r), last = r < s.lq ? last_key(s, r) : -1;
#pragma unroll
        for (int n = 0; n < MI; ++n) {
            const int t = k0 + tx + 16 * n;
            const bool in = t >= first && t <= last;
            const float w = in ? ex2(z[i][n] * (p.scale * LOG2E) - stat[i].x) : 0.f;
            P[(ty + 16 * i) * (B + 4) + tx + 16 * n] = w;
            S[(ty + 16 * i) * (B + 4) + tx + 16 * n] = in ? w * (dp[i][n] - stat[i].y) : 0.f;
        }
    }
}
template <int D>
__device__ __forceinline__ void load_stat(const PromptArgs& A, const Seq& s, int h, int row, float2 (&stat)[Back<D>::MI]) {
    const int ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < Back<D>::MI; ++i) {
        const int r = row + ty + 16 * i;
        stat[i] = r < s.lq ? A.stat[h * A.stat_rows + s.q0 + r] : make_float2(0.f, 0.f);
    }
}

// dk and dv of B keys of one kv-head: over the query heads that share it and their queries, in order
template <int D>
__global__ void __launch_bounds__(ST) k_prompt_dkv_simt(const PromptArgs A) {
    using T = float;
    constexpr int B = Back<D>::B, MI = Back<D>::MI;
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + B * (D + 4), *V = K + B * (D + 4), *G = V + B * (D + 4), *P = G + B * (D + 4), *S = P + B * (B + 4);
    const gdn_prompt_problem& p = A.p;
    Seq s;
    int k0;
    if (!find_tile<B>(p, true, blockIdx.x, s, k0)) return;  // the first keys have the most queries
    const int j = blockIdx.y, group = p.Hq / p.Hkv, keys = min(B, s.lk - k0), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_rows<B, D>(K, static_cast<const T*>(A.k) + (int64_t(s.k0) + k0) * p.k_stride + int64_t(j) * D, p.k_stride, keys);
    load_rows<B, D>(V, static_cast<const T*>(A.v) + (int64_t(s.k0) + k0) * p.v_stride + int64_t(j) * D, p.v_stride, keys);
    float dk[MI][D / 16] = {}, dv[MI][D / 16] = {};
    const int q_begin = first_query(s, k0) / B * B, q_end = s.rest ? 0 : last_query(p, s, k0 + keys - 1) + 1;
    for (int h = j * group; h < (j + 1) * group; ++h)
        for (int row = q_begin; row < q_end; row += B) {
            __syncthreads();
            const int rows = min(B, s.lq - row);
            load_rows<B, D>(Q, static_cast<const T*>(A.q) + (int64_t(s.q0) + row) * p.q_stride + int64_t(h) * D, p.q_stride, rows);
            load_rows<B, D>(G, static_cast<const T*>(A.dO) + ((int64_t(s.q0) + row) * p.Hq + h) * D, int64_t(p.Hq) * D, rows);
            float2 stat[MI];
            load_stat<D>(A, s, h, row, stat);
            __syncthreads();
            back_tile<D>(p, s, row, k0, stat, Q, K, G, V, P, S);
            __syncthreads();
            if (rows == B && keys == B && k0 + B - 1 <= last_key(s, row) && k0 >= first_key(p, s, row + B - 1)) {
                mul_add<MI, D, true, false>(dv, B, P, B + 4, G, [](int, int) { return true; });
                mul_add<MI, D, true, false>(dk, B, S, B + 4, Q, [](int, int) { return true; });
            } else {
                auto counts = [&](int i, int n) {
                    const int t = k0 + ty + 16 * i, r = row + n;
                    return r < s.lq && t >= first_key(p, s, r) && t <= last_key(s, r);
                };
                mul_add<MI, D, true, true>(dv, rows, P, B + 4, G, counts);
                mul_add<MI, D, true, true>(dk, rows, S, B + 4, Q, counts);
            }
        }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        if (ty + 16 * i >= keys) continue;
        const int64_t at = ((int64_t(s.k0) + k0 + ty + 16 * i) * p.Hkv + j) * D + 4 * tx;
#pragma unroll
        for (int v = 0; v < D / 64; ++v) {
            st4(static_cast<T*>(A.dk) + at + 64 * v, dk[i][4 * v] * p.scale, dk[i][4 * v + 1] * p.scale, dk[i][4 * v + 2] * p.scale, dk[i][4 * v + 3] * p.scale);
            st4(static_cast<T*>(A.dv) + at + 64 * v, dv[i][4 * v], dv[i][4 * v + 1], dv[i][4 * v + 2], dv[i][4 * v + 3]);
        }
    }
}

// dq of B queries of one head
template <int D>
__global__ void __launch_bounds__(ST) k_prompt_dq_simt(const PromptArgs A) {
    using T = float;
    constexpr int B = Back<D>::B, MI = Back<D>::MI;
    extern __shared__ __align__(16) float sm[];
    float *Q = sm, *K = Q + B * (D + 4), *V = K + B * (D + 4), *G = V + B * (D + 4), *P = G + B * (D + 4), *S = P + B * (B + 4);
    const gdn_prompt_problem& p = A.p;
    Seq s;
    int row;
    if (!find_tile<B>(p, false, gridDim.x - 1 - blockIdx.x, s, row)) return;
    const int h = blockIdx.y, j = h / (p.Hq / p.Hkv), rows = min(B, s.lq - row), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int k_end = s.rest ? 0 : min(s.lk, last_key(s, row + rows - 1) + 1), k_begin = k_end > 0 ? first_key(p, s, row) / B * B : 0;
    load_rows<B, D>(Q, static_cast<const T*>(A.q) + (int64_t(s.q0) + row) * p.q_stride + int64_t(h) * D, p.q_stride, rows);
    load_rows<B, D>(G, static_cast<const T*>(A.dO) + ((int64_t(s.q0) + row) * p.Hq + h) * D, int64_t(p.Hq) * D, rows);
    float2 stat[MI];
    load_stat<D>(A, s, h, row, stat);
    float dq[MI][D / 16] = {};
    for (int k0 = k_begin; k0 < k_end; k0 += B) {
        __syncthreads();
        const int keys = min(B, s.lk - k0);
        load_rows<B, D>(K, static_cast<const T*>(A.k) + (int64_t(s.k0) + k0) * p.k_stride + int64_t(j) * D, p.k_stride, keys);
        load_rows<B, D>(V, static_cast<const T*>(A.v) + (int64_t(s.k0) + k0) * p.v_stride + int64_t(j) * D, p.v_stride, keys);
        __syncthreads();
        back_tile<D>(p, s, row, k0, stat, Q, K, G, V, P, S);
        __syncthreads();
        if (rows == B && k0 + B - 1 <= last_key(s, row) && k0 >= first_key(p, s, row + B - 1))
            mul_add<MI, D, false, false>(dq, B, S, B + 4, K, [](int, int) { return true; });
        else
            mul_add<MI, D, false, true>(dq, keys, S, B + 4, K, [&](int i, int n) {
                const int r = row + ty + 16 * i;
                return r < s.lq && k0 + n >= first_key(p, s, r) && k0 + n <= last_key(s, r);
            });
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        if (ty + 16 * i >= rows) continue;
        const int64_t at = ((int64_t(s.q0) + row + ty + 16 * i) * p.Hq + h) * D + 4 * tx;
#pragma unroll
        for (int v = 0; v < D / 64; ++v)
            st4(static_cast<T*>(A.dq) + at + 64 * v, dq[i][4 * v] * p.scale, dq[i][4 * v + 1] * p.scale, dq[i][4 * v + 2] * p.scale, dq[i][4 * v + 3] * p.scale);
    }
}

cudaError_t launch(void (*kern)(const PromptArgs), const char* name, dim3 grid, int smem, const PromptArgs& A, cudaStream_t st) {
    if (grid.x == 0) return cudaSuccess;
    cudaError_t e = smem_attr(kern, smem);
    if (e != cudaSuccess) return e;
    timing_begin(name, st);
    kern<<<grid, ST, smem, st>>>(A);
    timing_end(st);
    return cudaGetLastError();
}
template <int D, int MI>
cudaError_t fwd_rows(const PromptArgs& A, cudaStream_t st) {
    return launch(k_prompt_fwd_simt<D, MI>, "prompt_attn_fwd", dim3(unsigned(tile_numbers(A.p, false, 16 * MI)), A.p.Hq), fwd_smem<D, MI>(), A, st);
}
// Fewer queries to a CTA as long as there is at most one CTA to a multiprocessor: 2 x 100 tokens, 8 / 2 heads, 64 features take
// 9 us with 16 queries, 14 with 64.
template <int D>
cudaError_t fwd(const PromptArgs& A, cudaStream_t st) {
    auto ctas = [&](int rows) { return (int64_t(A.p.total_q) / rows + A.p.num_seqs) * A.p.Hq; };
    const int sms = sm_count_cached();
    return ctas(16) <= sms ? fwd_rows<D, 1>(A, st) : ctas(32) <= sms ? fwd_rows<D, 2>(A, st) : fwd_rows<D, 4>(A, st);
}
template <int D>
cudaError_t bwd(const PromptArgs& A, cudaStream_t st) {
    cudaError_t e = A.p.total_q ? launch(k_prompt_dq_simt<D>, "prompt_attn_dq", dim3(unsigned(tile_numbers(A.p, false, Back<D>::B)), A.p.Hq), Back<D>::SMEM, A, st) : cudaSuccess;
    if (e != cudaSuccess || !A.p.total_k) return e;
    return launch(k_prompt_dkv_simt<D>, "prompt_attn_dkv", dim3(unsigned(tile_numbers(A.p, true, Back<D>::B)), A.p.Hkv), Back<D>::SMEM, A, st);
}

}  // namespace

size_t prompt_bwd_workspace(const gdn_prompt_problem& p) {
    const int parts = prompt_bwd_parts(p);
    return size_t((int64_t(p.total_q) + 127) / 128 * 128) * p.Hq * sizeof(float2) + (parts > 1 ? size_t(2) * parts * p.total_k * p.Hkv * p.D * sizeof(float) : 0);
}

cudaError_t launch_prompt_stat(const PromptArgs& A, cudaStream_t st) {
    const int64_t blocks = (int64_t(A.p.total_q) + 63) / 64 * A.p.Hq;
    if (blocks == 0) return cudaSuccess;
    timing_begin("prompt_attn_stat", st);
    auto go = [&](auto kern) { kern<<<unsigned(blocks), 256, 0, st>>>(A); };
    using B = __nv_bfloat16;
    if (A.p.dtype == GDN_FP32)
        A.p.D == 64 ? go(k_prompt_stat<float, 64>) : A.p.D == 128 ? go(k_prompt_stat<float, 128>) : go(k_prompt_stat<float, 256>);
    else
        A.p.D == 64 ? go(k_prompt_stat<B, 64>) : A.p.D == 128 ? go(k_prompt_stat<B, 128>) : go(k_prompt_stat<B, 256>);
    timing_end(st);
    return cudaGetLastError();
}
cudaError_t launch_prompt_fwd_simt(const PromptArgs& A, cudaStream_t st) { return A.p.D == 64 ? fwd<64>(A, st) : A.p.D == 128 ? fwd<128>(A, st) : fwd<256>(A, st); }
cudaError_t launch_prompt_bwd_simt(const PromptArgs& A, cudaStream_t st) { return A.p.D == 64 ? bwd<64>(A, st) : A.p.D == 128 ? bwd<128>(A, st) : bwd<256>(A, st); }

}  // namespace gdn
