// Recurrent step of the gated delta rule (include/gdn.h, gdn_recurrent_step): per sequence,
// v-head and token, for the state h [K][V]
//   u = beta (v - e^g h^T k),   h <- e^g h + k u^T,   o = scale h^T q.
// With a = h^T k and b = h^T q of the state before the token, o = scale (e^g b + <k, q> u): one
// pass over the state gives both sums, a second one (over registers) updates it, so a state is
// read from HBM once and written once however many tokens the sequence has.
//
// The columns of h are independent of one another, so a state is cut into 4 blocks of 32
// columns, one to a CTA of 128 threads that keeps its 16 KB in registers (8 float4 a thread).
// The sums over K run over a thread's 8 rows, the 4 row lanes of a warp and the 4 warps.
// Bound: HBM, 64 KB in and 64 KB out per (sequence, v-head).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_common.cuh"
#include "gdn_decode.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int ST = 128;       // threads
constexpr int SC = 32;        // state columns per CTA
constexpr int SR = KD / 16;   // rows of the state per thread

__device__ __forceinline__ float sum_rows(float v) {  // over the 4 row lanes of a warp
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

template <typename Op>
__global__ void __launch_bounds__(ST) k_step(const StepArgs A) {
    const gdn_step_problem& p = A.p;
    __shared__ float sq[KD], sk[KD], nrm[2][4];
    __shared__ float4 red[2][4][SC / 4];
    __shared__ float red_kq[4];
    const int tid = threadIdx.x, warp = tid >> 5, c4 = tid & 7, r = tid >> 3;
    const int64_t item = int64_t(blockIdx.x) / (VD / SC);
    const int col = int(blockIdx.x % (VD / SC)) * SC + 4 * c4;
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
    Op* o = static_cast<Op*>(A.o);
    const int64_t slot = p.slots ? p.slots[s] : s;
    if (slot < 0 || slot >= p.num_slots) {
        for (int t = t0 + r; t < t1; t += 16) {
            Op* to = o + (int64_t(t) * p.Hv + j) * VD + col;
            st2(to, 0.f, 0.f);
            st2(to + 2, 0.f, 0.f);
        }
        return;
    }

    const int64_t base = (slot * p.Hv + j) * (int64_t(KD) * VD) + col;
    float4 h[SR];
#pragma unroll
    for (int i = 0; i < SR; ++i)
        h[i] = A.state_in ? *reinterpret_cast<const float4*>(A.state_in + base + int64_t(r + 16 * i) * VD)
                          : make_float4(0.f, 0.f, 0.f, 0.f);

    const float decay = A.A_log ? -expf(A.A_log[j]) : 0.f, bias = A.A_log ? A.dt_bias[j] : 0.f;
    for (int t = t0; t < t1; ++t) {
        float xq = to_f(static_cast<const Op*>(A.q)[t * p.q_stride + hq * KD + tid]);
        float xk = to_f(static_cast<const Op*>(A.k)[t * p.k_stride + hq * KD + tid]);
        float g = A.g[t * p.g_stride + j], beta = A.beta[t * p.beta_stride + j];
        const Op* vt = static_cast<const Op*>(A.v) + t * p.v_stride + int64_t(j) * VD + col;
        const float v4[4] = {to_f(vt[0]), to_f(vt[1]), to_f(vt[2]), to_f(vt[3])};
        float iq = 1.f, ik = 1.f;
        __syncthreads();  // the last token's reads of the shared arrays are done
        sq[tid] = xq;
        sk[tid] = xk;
        if (A.A_log) {
            float nq = xq * xq, nk = xk * xk;
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) {
                nq += __shfl_xor_sync(0xffffffffu, nq, m);
                nk += __shfl_xor_sync(0xffffffffu, nk, m);
            }
            if ((tid & 31) == 0) {
                nrm[0][warp] = nq;
                nrm[1][warp] = nk;
            }
            g = decay * softplus_f(g + bias);
            beta = sigmoid_f(beta);
        }
        __syncthreads();
        if (A.A_log) {
            iq = rsqrtf(nrm[0][0] + nrm[0][1] + nrm[0][2] + nrm[0][3] + PRO_EPS);
            ik = rsqrtf(nrm[1][0] + nrm[1][1] + nrm[1][2] + nrm[1][3] + PRO_EPS);
        }
        float a[4] = {}, b[4] = {}, kq = 0.f, kr[SR];
#pragma unroll
        for (int i = 0; i < SR; ++i) {
            kr[i] = sk[r + 16 * i] * ik;
            const float qr = sq[r + 16 * i] * iq;
            a[0] = fmaf(h[i].x, kr[i], a[0]);
            a[1] = fmaf(h[i].y, kr[i], a[1]);
            a[2] = fmaf(h[i].z, kr[i], a[2]);
            a[3] = fmaf(h[i].w, kr[i], a[3]);
            b[0] = fmaf(h[i].x, qr, b[0]);
            b[1] = fmaf(h[i].y, qr, b[1]);
            b[2] = fmaf(h[i].z, qr, b[2]);
            b[3] = fmaf(h[i].w, qr, b[3]);
            kq = fmaf(kr[i], qr, kq);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = sum_rows(a[e]);
            b[e] = sum_rows(b[e]);
        }
        kq = sum_rows(kq);
        if ((tid & 31) < 8) {
            red[0][warp][c4] = make_float4(a[0], a[1], a[2], a[3]);
            red[1][warp][c4] = make_float4(b[0], b[1], b[2], b[3]);
            red_kq[warp] = kq;
        }
        __syncthreads();
        float sa[4] = {}, sb[4] = {};
        kq = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 x = red[0][w][c4], y = red[1][w][c4];
            sa[0] += x.x; sa[1] += x.y; sa[2] += x.z; sa[3] += x.w;
            sb[0] += y.x; sb[1] += y.y; sb[2] += y.z; sb[3] += y.w;
            kq += red_kq[w];
        }
        const float eg = expf(g);
        float u[4], out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u[e] = beta * (v4[e] - eg * sa[e]);
            out[e] = p.scale * fmaf(kq, u[e], eg * sb[e]);
        }
        if (r == 0) {
            Op* to = o + (int64_t(t) * p.Hv + j) * VD + col;
            st2(to, out[0], out[1]);
            st2(to + 2, out[2], out[3]);
        }
#pragma unroll
        for (int i = 0; i < SR; ++i) {
            h[i].x = fmaf(kr[i], u[0], eg * h[i].x);
            h[i].y = fmaf(kr[i], u[1], eg * h[i].y);
            h[i].z = fmaf(kr[i], u[2], eg * h[i].z);
            h[i].w = fmaf(kr[i], u[3], eg * h[i].w);
        }
    }
    if (A.state_out && (t1 > t0 || A.state_out != A.state_in)) {
#pragma unroll
        for (int i = 0; i < SR; ++i)
            *reinterpret_cast<float4*>(A.state_out + base + int64_t(r + 16 * i) * VD) = h[i];
    }
}

}  // namespace

cudaError_t launch_step(const StepArgs& A, cudaStream_t st) {
    const int64_t blocks = int64_t(A.p.num_seqs) * A.p.Hv * (VD / SC);
    timing_begin("recurrent_step", st);
    if (A.p.dtype == GDN_BF16)
        k_step<__nv_bfloat16><<<unsigned(blocks), ST, 0, st>>>(A);
    else
        k_step<float><<<unsigned(blocks), ST, 0, st>>>(A);
    timing_end(st);
    return cudaGetLastError();
}

}  // namespace gdn
