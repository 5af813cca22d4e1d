// Recurrent step of the gated delta rule (include/gdn.h, gdn_recurrent_step): per sequence,
// v-head and token, for the state h [K][V]
//   u = beta (v - e^g h^T k),   h <- e^g h + k u^T,   o = scale h^T q.
// With a = h^T k and b = h^T q of the state before the token, o = scale (e^g b + <k, q> u): one
// pass over the state gives both sums, a second one (over registers) updates it, so a state is
// read from HBM once and written once however many tokens the sequence has.
//
// The columns of h are independent of one another, so a state is cut into 4 blocks of 32 columns, one to
// a CTA of 4 warps; a lane has one column and 32 of the rows in registers, as pairs of rows for the packed
// fp32 multiply-add, so that a token's sums need no exchange within a warp and one barrier (the warps' 4
// parts).  A token's q, k, v, gates and <k, q> are prepared by one warp, up to STEP_TOKENS tokens at a
// time, while the state is on its way.
// The decay of all but a sequence's last token stays a factor E of the whole state (the state is E h, u is
// added as u / E, a fast division within 2^-22), which spares a multiplication per value and token; E is
// multiplied out where it leaves [2^-20, 2^20], so that h and u / E keep within 2^20 of the state's own range, and
// with the last token, so that a single token rounds as the formula does.  (48 sequences of up to 6 tokens: 1.1e-7
// off 64 bits, the formula in fp32 tensor operations 1.6e-7.)
// Bound: HBM, 64 KB in and 64 KB out per (sequence, v-head).  Measured: 256 sequences x 64 v-heads, one
// token, bf16, 307 us (7.0 TB/s of states and rows, 1.05 of the copy bandwidth measured on the same GPUs);
// 32 x 24 from raw projections 18.5 us (floor 15.1: three waves of CTAs); 48 sequences of up to 6 tokens, 48
// v-heads, fp32, 56 us (floor 46.8: each token some 115 instructions a warp and one barrier; 58 with the decay
// multiplied into the state every token).  Not kept: two tokens to a barrier (66 us, registers spill), two columns
// and 16 rows a lane (58 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_common.cuh"
#include "gdn_decode.h"
#include "gdn_internal.h"
#include "tc05.cuh"

namespace gdn {
namespace {

constexpr int ST = 128;          // threads
constexpr int SC = 32;           // state columns per CTA
constexpr int SR = KD / 4;       // rows of the state per thread
constexpr int STEP_TOKENS = 8;   // tokens prepared at a time
constexpr float LEAST = 1.f / (1 << 20);  // of the factor E

// 4 consecutive values
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float dot4(float4 a, float4 b) { return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w))); }

template <typename Op>
__global__ void __launch_bounds__(ST, 8) k_step(const StepArgs A) {
    const gdn_step_problem& p = A.p;
    __shared__ __align__(16) float sk[STEP_TOKENS][KD], sq[STEP_TOKENS][KD];
    __shared__ float sv[STEP_TOKENS][SC], red[2][4][2][SC];
    __shared__ float4 gate[STEP_TOKENS];  // e^g, beta, <k, q>
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t item = int64_t(blockIdx.x) / (VD / SC);
    const int col = int(blockIdx.x % (VD / SC)) * SC + lane;
    const int s = int(item / p.Hv), j = int(item % p.Hv), hq = j / (p.Hv / p.Hqk);

    int t0, t1;
    if (p.cu_seqlens) {
        t0 = max(0, min(p.cu_seqlens[s], p.total_tokens));
        t1 = max(t0, min(p.cu_seqlens[s + 1], p.total_tokens));
    } else {
        const int per = p.total_tokens / p.num_seqs;
        t0 = s * per;
        t1 = t0 + per;
    }
    Op* o = static_cast<Op*>(A.o) + int64_t(j) * VD + col;
    if (p.clear_rest) {  // the first sequence's and the last one's CTAs, where there is such a token at all
        if (s == 0)
            for (int t = warp; t < t0; t += 4) o[int64_t(t) * p.Hv * VD] = from_f<Op>(0.f);
        if (s == p.num_seqs - 1)
            for (int t = t1 + warp; t < p.total_tokens; t += 4) o[int64_t(t) * p.Hv * VD] = from_f<Op>(0.f);
    }
    const int64_t slot = p.slots ? p.slots[s] : s;
    if (slot < 0 || slot >= p.num_slots) {
        for (int t = t0 + warp; t < t1; t += 4) o[int64_t(t) * p.Hv * VD] = from_f<Op>(0.f);
        return;
    }

    const int64_t base = (slot * p.Hv + j) * (int64_t(KD) * VD) + int64_t(warp) * SR * VD + col;
    uint64_t h[SR / 2];  // pairs of rows
    if (A.state_in) {
        const float* in = A.state_in + base;
        float x[SR];
#pragma unroll
        for (int i = 0; i < SR; ++i) x[i] = in[i * VD];
#pragma unroll
        for (int i = 0; i < SR / 2; ++i) h[i] = tc::pk2(x[2 * i], x[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < SR / 2; ++i) h[i] = 0ull;
    }

    if (A.state_in && tid == 0 && blockIdx.x % (VD / SC) == 0) {
        // the state of the item one multiprocessor's worth of CTAs on is asked into L2 (3 to 6 % less
        // time at 768 to 12288 states; two on: as much at few tokens, 7 % more at 16384 states)
        const int64_t next = item + A.ahead;
        if (next < int64_t(p.num_seqs) * p.Hv) {
            const int s2 = int(next / p.Hv), j2 = int(next % p.Hv);
            const int64_t slot2 = p.slots ? p.slots[s2] : s2;
            if (slot2 >= 0 && slot2 < p.num_slots)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(A.state_in + (slot2 * p.Hv + j2) * (int64_t(KD) * VD)),
                             "r"(KD * VD * 4)
                             : "memory");
        }
    }
    float E = 1.f;  // the state is E h
    for (int c0 = t0; c0 < t1; c0 += STEP_TOKENS) {
        const int n = min(STEP_TOKENS, t1 - c0);
        if (c0 > t0) __syncthreads();  // the last tokens have been read
        for (int i = warp; i < n; i += 4) {  // a warp prepares a token
            const int64_t t = c0 + i;
            float4 q = load4(static_cast<const Op*>(A.q) + t * p.q_stride + hq * KD + 4 * lane);
            float4 k = load4(static_cast<const Op*>(A.k) + t * p.k_stride + hq * KD + 4 * lane);
            float g = A.g[t * p.g_stride + j], beta = A.beta[t * p.beta_stride + j];
            const float v = to_f(static_cast<const Op*>(A.v)[t * p.v_stride + int64_t(j) * VD + col]);
            float kq = dot4(k, q), qq = 0.f, kk = 0.f;
            if (A.A_log) qq = dot4(q, q), kk = dot4(k, k);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) {
                kq += __shfl_xor_sync(0xffffffffu, kq, m);
                if (A.A_log) {
                    qq += __shfl_xor_sync(0xffffffffu, qq, m);
                    kk += __shfl_xor_sync(0xffffffffu, kk, m);
                }
            }
            if (A.A_log) {
                const float iq = rsqrtf(qq + PRO_EPS), ik = rsqrtf(kk + PRO_EPS);
                q.x *= iq, q.y *= iq, q.z *= iq, q.w *= iq;
                k.x *= ik, k.y *= ik, k.z *= ik, k.w *= ik;
                kq *= iq * ik;
                g = -expf(A.A_log[j]) * softplus_f(g + A.dt_bias[j]);
                beta = sigmoid_f(beta);
            }
            *reinterpret_cast<float4*>(&sq[i][4 * lane]) = q;
            *reinterpret_cast<float4*>(&sk[i][4 * lane]) = k;
            sv[i][lane] = v;
            if (lane == 0) gate[i] = make_float4(expf(g), beta, kq, 0.f);
        }
        __syncthreads();
        for (int i = 0; i < n; ++i) {
            const ulonglong2* k2 = reinterpret_cast<const ulonglong2*>(&sk[i][warp * SR]);
            const ulonglong2* q2 = reinterpret_cast<const ulonglong2*>(&sq[i][warp * SR]);
            uint64_t a2 = 0ull, b2 = 0ull, a3 = 0ull, b3 = 0ull;
#pragma unroll
            for (int x = 0; x < SR / 4; ++x) {
                const ulonglong2 kx = k2[x], qx = q2[x];
                a2 = tc::ffma2(h[2 * x], kx.x, a2);
                b2 = tc::ffma2(h[2 * x], qx.x, b2);
                a3 = tc::ffma2(h[2 * x + 1], kx.y, a3);
                b3 = tc::ffma2(h[2 * x + 1], qx.y, b3);
            }
            float a[4], b[4];
            tc::unpk2(a2, a[0], a[1]);
            tc::unpk2(a3, a[2], a[3]);
            tc::unpk2(b2, b[0], b[1]);
            tc::unpk2(b3, b[2], b[3]);
            red[i & 1][warp][0][lane] = (a[0] + a[1]) + (a[2] + a[3]);
            red[i & 1][warp][1][lane] = (b[0] + b[1]) + (b[2] + b[3]);
            __syncthreads();  // a warp is at most one token ahead of the others' reads: two buffers
            const float4 gt = gate[i];
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                sa += red[i & 1][w][0][lane];
                sb += red[i & 1][w][1][lane];
            }
            const float decay = E * gt.x, u = gt.y * (sv[i][lane] - decay * sa);
            if (warp == (i & 3)) o[int64_t(c0 + i) * p.Hv * VD] = from_f<Op>(p.scale * fmaf(gt.z, u, decay * sb));
            if (c0 + i + 1 < t1 && decay >= LEAST && decay <= 1.f / LEAST) {
                E = decay;
                const uint64_t u2 = tc::dup2(__fdividef(u, decay));
#pragma unroll
                for (int x = 0; x < SR / 4; ++x) {
                    const ulonglong2 kx = k2[x];
                    h[2 * x] = tc::ffma2(kx.x, u2, h[2 * x]);
                    h[2 * x + 1] = tc::ffma2(kx.y, u2, h[2 * x + 1]);
                }
            } else {
                E = 1.f;
                const uint64_t u2 = tc::dup2(u), e2 = tc::dup2(decay);
#pragma unroll
                for (int x = 0; x < SR / 4; ++x) {
                    const ulonglong2 kx = k2[x];
                    h[2 * x] = tc::ffma2(kx.x, u2, tc::fmul2(e2, h[2 * x]));
                    h[2 * x + 1] = tc::ffma2(kx.y, u2, tc::fmul2(e2, h[2 * x + 1]));
                }
            }
        }
    }
    if (A.state_out && (t1 > t0 || A.state_out != A.state_in)) {
        float* out = A.state_out + base;
#pragma unroll
        for (int i = 0; i < SR / 2; ++i) {
            float x, y;
            tc::unpk2(h[i], x, y);
            out[2 * i * VD] = x;
            out[(2 * i + 1) * VD] = y;
        }
    }
}

}  // namespace

cudaError_t launch_step(const StepArgs& A, cudaStream_t st) {
    const int64_t blocks = int64_t(A.p.num_seqs) * A.p.Hv * (VD / SC);
    StepArgs B = A;
    B.ahead = sm_count_cached();
    timing_begin("recurrent_step", st);
    if (A.p.dtype == GDN_BF16)
        k_step<__nv_bfloat16><<<unsigned(blocks), ST, 0, st>>>(B);
    else
        k_step<float><<<unsigned(blocks), ST, 0, st>>>(B);
    timing_end(st);
    return cudaGetLastError();
}

}  // namespace gdn
