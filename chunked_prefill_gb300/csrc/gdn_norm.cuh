// The RMS norm's kernels and launches for one type of rows (see gdn_norm.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <map>
#include <mutex>
#include <tuple>

#include "gdn_common.cuh"
#include "gdn_decode.h"
#include "gdn_internal.h"
#include "tc05.cuh"

namespace gdn {
namespace {

constexpr float F8_MAX = 448.f;
constexpr float F8_TINY = 1.17549435e-38f;  // 2^-126
constexpr int ROWS_T = 256;                 // threads of a CTA of the lane-group kernels
constexpr int LOOP_T = 512;                 // threads of the looping kernels
// Threads of a CTA at most, so that a row's values fit the registers that many threads leave each.
constexpr int max_threads(int vec, int nv, int lpr, bool backward) {
    return lpr ? ROWS_T : vec == 1 ? (nv == 16 ? 512 : 256) : (backward || nv >= 2) ? 512 : 1024;
}

// the larger of two values, NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// 1 / x to 2^-23 of itself
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool MAX> __device__ __forceinline__ float join(float a, float b) { return MAX ? max_nan(a, b) : a + b; }

template <bool MAX, int LANES>
__device__ __forceinline__ float lane_red(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = join<MAX>(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// Over the threads of a row; a CTA's rows go through `red` (32 floats, not used again before every
// thread has read it: callers alternate between two).
template <bool MAX, int LPR>
__device__ __forceinline__ float row_red(float v, float* red) {
    if constexpr (LPR > 0) {
        return lane_red<MAX, LPR>(v);
    } else {
        v = lane_red<MAX, 32>(v);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        return lane_red<MAX, 32>(lane < warps ? red[lane] : 0.f);
    }
}

__device__ __forceinline__ int64_t wide_mul(uint32_t a, int64_t b) { return int64_t(uint64_t(a) * uint32_t(b)); }

// VEC consecutive values as they lie in memory.
template <typename T, int VEC> struct Vec {
    T v[VEC];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (sizeof(T) * VEC == 16)
            *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (sizeof(T) * VEC == 8)
            *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
        else if constexpr (sizeof(T) * VEC == 32) {
            reinterpret_cast<uint4*>(v)[0] = reinterpret_cast<const uint4*>(p)[0];
            reinterpret_cast<uint4*>(v)[1] = reinterpret_cast<const uint4*>(p)[1];
        } else
            v[0] = p[0];
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (sizeof(T) * VEC == 16)
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
        else
            p[0] = v[0];
    }
    __device__ __forceinline__ float at(int i) const { return to_f(v[i]); }
};

// The values of a row's piece that starts at value `off` of the row.  `left`: values of the tensor from the
// row's start on.  A piece that reaches into a neighbouring row is read whole (the row before it is there, the
// one after it where `left` says so); whatever is written there meanwhile does not matter, for the values
// outside [0, dim) are masked by mask_piece (apart, so that a load need not be waited for where it is asked for).
template <bool SHIFT, typename T, int VEC>
__device__ __forceinline__ void load_piece(Vec<T, VEC>& v, const T* row, int off, int dim, int64_t left) {
    if (!SHIFT || off + VEC <= left) {
        v.load(row + off);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v.v[e] = unsigned(off + e) < unsigned(dim) ? row[off + e] : from_f<T>(0.f);
    }
}
template <bool SHIFT, typename T, int VEC>
__device__ __forceinline__ void mask_piece(Vec<T, VEC>& v, int off, int dim) {
    if (SHIFT && (off < 0 || off + VEC > dim)) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (unsigned(off + e) >= unsigned(dim)) v.v[e] = from_f<T>(0.f);
    }
}
template <bool SHIFT, typename T, int VEC>
__device__ __forceinline__ void store_piece(const Vec<T, VEC>& v, T* row, int off, int dim) {
    if (!SHIFT || (off >= 0 && off + VEC <= dim)) {
        v.store(row + off);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (unsigned(off + e) < unsigned(dim)) row[off + e] = v.v[e];
    }
}

template <int VEC>
__device__ __forceinline__ void load_weight(const gdn_norm_problem& p, const void* w, int i, float (&out)[VEC]) {
    if (p.weight_dtype == GDN_BF16) {
        Vec<__nv_bfloat16, VEC> x;
        x.load(static_cast<const __nv_bfloat16*>(w) + i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = x.at(e) + p.weight_offset;
    } else {
        Vec<float, VEC> x;
        x.load(static_cast<const float*>(w) + i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = x.at(e) + p.weight_offset;
    }
}

// The weights (with their offset) of a piece, zeros outside the row.
template <bool SHIFT, int VEC>
__device__ __forceinline__ void weight_piece(const gdn_norm_problem& p, const void* w, int off, float (&out)[VEC]) {
    if constexpr (!SHIFT) {
        load_weight<VEC>(p, w, off, out);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float one[1] = {0.f};
            if (unsigned(off + e) < unsigned(p.dim)) load_weight<1>(p, w, off + e, one);
            out[e] = one[0];
        }
    }
}

// y * inv in 8 bits, round to nearest even (|y inv| <= 448 up to rounding; NaN stays NaN).  inv = rcp(scale), once
// for a piece of a row: within 2^-22 of the quotient; a division per value would be many more instructions where
// the issue slots are 75 % busy.
template <int VEC>
__device__ __forceinline__ void store8(uint8_t* p, const float (&y)[VEC], float inv) {
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(y[0] * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int e = 0; e < VEC / 4; ++e) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * e] * inv, y[4 * e + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * e + 2] * inv, y[4 * e + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            w[e] = lo | (hi << 16);
        }
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

// mag / 448 as a product (a division takes the same time and lies within 2^-24 instead of 2^-23 of it, but torch's
// own division of a GPU tensor by 448 is this product: 40 M values in groups of 128 agree with torch's to 2.4e-4 of
// their norm, with a division to 3.9e-4, and both are 0.026 off the exact values, the 8 bits' own rounding).
__device__ __forceinline__ float scale_of(float mag) { return max_nan(mag * (1.f / F8_MAX), F8_TINY); }

// OUT8: 0 dtype out; 1 one scale per row; 2 groups of 2^n <= 32 lanes' vectors; 3 other groups
// (magnitudes by shared-memory maxima, whose order does not matter).
template <typename T, int VEC, int NV, int LPR, bool SHIFT, int OUT8>
__global__ void __launch_bounds__(max_threads(VEC, NV, LPR, false), LPR == 0 && VEC > 1 && NV == 2 && !SHIFT ? 4 : 1) k_norm_fwd(const NormArgs A) {
    const gdn_norm_problem& p = A.p;
    __shared__ float red[2][32];
    extern __shared__ uint32_t mags[];  // OUT8 == 3: per group of the CTA's row(s)
    const int tid = threadIdx.x, step = LPR ? LPR : blockDim.x, at0 = LPR ? tid % step : tid;
    const int per = LPR ? int(blockDim.x) / step : 1, mine = LPR ? tid / step : 0;  // rows per CTA, and this thread's
    const uint32_t row = blockIdx.x * per + mine;  // rows, strides and dim are below 2^31, products of two 64 bits
    const int a0 = SHIFT ? int(row * uint32_t(p.dim) & (VEC - 1)) : 0, nvec = SHIFT ? (a0 + p.dim + VEC - 1) / VEC : p.dim / VEC;
    const bool live = row < uint32_t(p.rows);
    const T* x = static_cast<const T*>(A.x) + wide_mul(row, p.x_stride);
    const T* res = static_cast<const T*>(A.residual) + wide_mul(row, p.residual_stride);
    const int64_t left = wide_mul(uint32_t(p.rows) - row, p.dim);

    Vec<T, VEC> xv[NV], rv[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int j = at0 + k * step;
        if (live && j < nvec) {
            load_piece<SHIFT>(xv[k], x, j * VEC - a0, p.dim, left);
            if (A.residual) load_piece<SHIFT>(rv[k], res, j * VEC - a0, p.dim, left);
        }
    }
    float s[NV][VEC], ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const bool in = live && at0 + k * step < nvec;
        if (in) {
            mask_piece<SHIFT>(xv[k], (at0 + k * step) * VEC - a0, p.dim);
            if (A.residual) mask_piece<SHIFT>(rv[k], (at0 + k * step) * VEC - a0, p.dim);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s[k][e] = in ? (A.residual ? xv[k].at(e) + rv[k].at(e) : xv[k].at(e)) : 0.f;
            ss = fmaf(s[k][e], s[k][e], ss);
        }
    }
    if (A.sum) {
        T* sum = static_cast<T*>(A.sum) + wide_mul(row, p.dim);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = at0 + k * step;
            if (live && j < nvec) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) xv[k].v[e] = from_f<T>(s[k][e]);
                store_piece<SHIFT>(xv[k], sum, j * VEC - a0, p.dim);
            }
        }
    }
    const float r = rsqrtf(row_red<false, LPR>(ss, red[0]) * A.inv_dim + p.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int j = at0 + k * step;
        if (j < nvec) {
            float w[VEC];
            weight_piece<SHIFT, VEC>(p, A.weight, j * VEC - a0, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[k][e] = s[k][e] * r * w[e];
        }
    }
    if constexpr (OUT8 == 0) {
        T* y = static_cast<T*>(A.y) + wide_mul(row, p.dim);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = at0 + k * step;
            if (live && j < nvec) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) xv[k].v[e] = from_f<T>(s[k][e]);
                store_piece<SHIFT>(xv[k], y, j * VEC - a0, p.dim);
            }
        }
    } else {
        uint8_t* y = static_cast<uint8_t*>(A.y) + wide_mul(row, p.dim);
        float mag[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            mag[k] = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) mag[k] = max_nan(mag[k], fabsf(s[k][e]));
        }
        const int groups = p.group ? p.dim / p.group : 1;
        float* scales = A.y_scale + wide_mul(row, groups);
        if constexpr (OUT8 == 1) {
#pragma unroll
            for (int k = 1; k < NV; ++k) mag[0] = max_nan(mag[0], mag[k]);
            const float sc = scale_of(row_red<true, LPR>(mag[0], red[1]));
            if (live && at0 == 0) scales[0] = sc;
            const float inv = rcp(sc);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (live && at0 + k * step < nvec) {
                    const int off = (at0 + k * step) * VEC - a0;
                    if (!SHIFT || (off >= 0 && off + VEC <= p.dim)) {
                        store8<VEC>(y + off, s[k], inv);
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float one[1] = {s[k][e]};
                            if (unsigned(off + e) < unsigned(p.dim)) store8<1>(y + off + e, one, inv);
                        }
                    }
                }
        } else if constexpr (OUT8 == 2) {
            const int lanes = p.group / VEC, shift = __ffs(lanes) - 1;  // 2^shift lanes hold a group, at a multiple of 2^shift
            for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < NV; ++k) mag[k] = max_nan(mag[k], __shfl_xor_sync(0xffffffffu, mag[k], o));
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = at0 + k * step;
                if (live && j < nvec) {
                    const float sc = scale_of(mag[k]);
                    if ((j & (lanes - 1)) == 0) scales[j >> shift] = sc;
                    store8<VEC>(y + int64_t(j) * VEC, s[k], rcp(sc));
                }
            }
        } else {
            uint32_t* m = mags + mine * groups;
            for (int g = at0; g < groups; g += step) m[g] = 0u;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = at0 + k * step;
                if (j < nvec) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) atomicMax(m + (j * VEC + e) / p.group, __float_as_uint(fabsf(s[k][e])));
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = at0 + k * step;
                if (live && j < nvec) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int i = j * VEC + e, g = i / p.group;
                        const float sc = scale_of(__uint_as_float(m[g])), one[1] = {s[k][e]};
                        if (i % p.group == 0) scales[g] = sc;
                        store8<1>(y + i, one, rcp(sc));
                    }
                }
            }
        }
    }
}

// The backward asks for the next row before it reduces the present one: into registers, or, RINGED, into a ring of
// RING rows in shared memory, each thread copying and reading its own pieces (no barrier), which takes a third
// fewer registers.  That pays for rows of a CTA with SHIFT (30000 rows of 1001: 48 us instead of 57) and where
// two CTAs fit a multiprocessor instead of one (16384 of 5120: 103 us instead of 126), not elsewhere (65536 of
// 1000: 100 us instead of 88).
constexpr int RING = 3;
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {  // the rest of the 16 is 0
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// With SHIFT the CTAs' rows are 8 k apart, so that a0 is the same for all of a thread's rows and its columns
// stay its own.
template <typename T, int VEC, int NV, int LPR, bool SHIFT, bool RINGED>
__global__ void __launch_bounds__(max_threads(VEC, NV, LPR, true)) k_norm_bwd(const NormArgs A) {
    const gdn_norm_problem& p = A.p;
    __shared__ float red[2][2][32];
    const int tid = threadIdx.x, step = LPR ? LPR : blockDim.x, at0 = LPR ? tid % step : tid;
    const int per = LPR ? int(blockDim.x) / step : 1, mine = LPR ? tid / step : 0;
    const uint32_t first = blockIdx.x * per + mine;
    const int a0 = SHIFT ? int(first * uint32_t(p.dim) & (VEC - 1)) : 0, nvec = SHIFT ? (a0 + p.dim + VEC - 1) / VEC : p.dim / VEC;
    tc::pdl_launch_dependents();
    constexpr bool KEEP = NV * VEC < 32;  // the weights stay in registers (else: read again, from L1)
    float w[KEEP ? NV : 1][VEC], dw[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[k][e] = 0.f;
        if (KEEP && at0 + k * step < nvec) weight_piece<SHIFT, VEC>(p, A.weight, (at0 + k * step) * VEC - a0, w[KEEP ? k : 0]);
    }
    const float inv_dim = A.inv_dim;
    int turn = 0;
    constexpr bool AHEAD = !RINGED && (NV * VEC < 16 || (VEC == 8 && NV == 2));
    extern __shared__ __align__(16) unsigned char dyn[];
    const uint32_t ring = RINGED ? tc::smem_addr(dyn) + tid * 16 : 0, slot = blockDim.x * 16;
    Vec<T, VEC> xn[RINGED ? 1 : NV], dn[RINGED ? 1 : NV], sn[RINGED ? 1 : NV];
    const uint32_t hop = gridDim.x * per, rows = uint32_t(p.rows);
    auto fetch = [&](uint32_t row) {
        if (RINGED || row >= rows) return;
        const T* x = static_cast<const T*>(A.x) + wide_mul(row, p.x_stride);
        const T* dy = static_cast<const T*>(A.dy) + wide_mul(row, p.dy_stride);
        const T* ds = static_cast<const T*>(A.dsum) + wide_mul(row, p.dsum_stride);
        const int64_t left = wide_mul(rows - row, p.dim);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = at0 + k * step;
            if (j < nvec) {
                load_piece<SHIFT>(xn[RINGED ? 0 : k], x, j * VEC - a0, p.dim, left);
                load_piece<SHIFT>(dn[RINGED ? 0 : k], dy, j * VEC - a0, p.dim, left);
                if (A.dsum) load_piece<SHIFT>(sn[RINGED ? 0 : k], ds, j * VEC - a0, p.dim, left);
            }
        }
    };
    // the pieces of a row into the ring's place `at`
    auto copy = [&](uint32_t row, int at) {
        if (row < rows) {
            const T* x = static_cast<const T*>(A.x) + wide_mul(row, p.x_stride);
            const T* dy = static_cast<const T*>(A.dy) + wide_mul(row, p.dy_stride);
            const T* ds = static_cast<const T*>(A.dsum) + wide_mul(row, p.dsum_stride);
            const int64_t left = wide_mul(rows - row, p.dim);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = at0 + k * step, off = j * VEC - a0;
                const int64_t there = (left - off) * int64_t(sizeof(T));
                const int bytes = !SHIFT || there >= 16 ? 16 : int(there);
                const uint32_t to = ring + (at * 3 * NV + k) * slot;
                if (j < nvec) {
                    copy16(to, x + off, bytes);
                    copy16(to + NV * slot, dy + off, bytes);
                    if (A.dsum) copy16(to + 2 * NV * slot, ds + off, bytes);
                }
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    int place = 0;
    if (RINGED) {
#pragma unroll
        for (int i = 0; i < RING - 1; ++i) copy(first + i * hop, i);
    }
    if (AHEAD) fetch(first);
    // every lane of a warp takes part in the shuffles of every turn
    for (uint32_t row0 = blockIdx.x * per; row0 < rows; row0 += hop, turn ^= 1) {
        const uint32_t row = row0 + mine;
        const bool live = row < rows;
        Vec<T, VEC> xv[NV], dv[NV], sv[NV];
        if constexpr (RINGED) {
            asm volatile("cp.async.wait_group %0;\n" ::"n"(RING - 2) : "memory");
            copy(row + (RING - 1) * hop, place == 0 ? RING - 1 : place - 1);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const uint32_t from = ring + (place * 3 * NV + k) * slot;
                if (live && at0 + k * step < nvec) {
                    *reinterpret_cast<uint4*>(xv[k].v) = tc::lds128(from);
                    *reinterpret_cast<uint4*>(dv[k].v) = tc::lds128(from + NV * slot);
                    if (A.dsum) *reinterpret_cast<uint4*>(sv[k].v) = tc::lds128(from + 2 * NV * slot);
                }
            }
            place = place + 1 == RING ? 0 : place + 1;
        } else {
            if (!AHEAD) fetch(row);
#pragma unroll
            for (int k = 0; k < NV; ++k) xv[k] = xn[k], dv[k] = dn[k], sv[k] = sn[k];
            if (AHEAD) fetch(row + hop);
        }
        float ss = 0.f, c = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!(live && at0 + k * step < nvec)) continue;
            mask_piece<SHIFT>(xv[k], (at0 + k * step) * VEC - a0, p.dim);
            mask_piece<SHIFT>(dv[k], (at0 + k * step) * VEC - a0, p.dim);
            if (!KEEP) weight_piece<SHIFT, VEC>(p, A.weight, (at0 + k * step) * VEC - a0, w[0]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                ss = fmaf(xv[k].at(e), xv[k].at(e), ss);
                c = fmaf(w[KEEP ? k : 0][e] * dv[k].at(e), xv[k].at(e), c);
            }
        }
        if constexpr (LPR > 0) {
            ss = lane_red<false, LPR>(ss);
            c = lane_red<false, LPR>(c);
        } else {  // both sums behind one barrier
            ss = lane_red<false, 32>(ss);
            c = lane_red<false, 32>(c);
            const int lane = tid & 31, warps = blockDim.x >> 5;
            if (lane == 0) {
                red[turn][0][tid >> 5] = ss;
                red[turn][1][tid >> 5] = c;
            }
            __syncthreads();
            ss = lane_red<false, 32>(lane < warps ? red[turn][0][lane] : 0.f);
            c = lane_red<false, 32>(lane < warps ? red[turn][1][lane] : 0.f);
        }
        const float r = rsqrtf(ss * inv_dim + p.eps);
        c *= r * inv_dim;
        T* dx = static_cast<T*>(A.dx) + wide_mul(row, p.dim);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = at0 + k * step;
            if (live && j < nvec) {
                if (!KEEP) weight_piece<SHIFT, VEC>(p, A.weight, j * VEC - a0, w[0]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float n = xv[k].at(e) * r, d = dv[k].at(e);
                    dw[k][e] = fmaf(d, n, dw[k][e]);
                    xv[k].v[e] = from_f<T>(fmaf(r, w[KEEP ? k : 0][e] * d - n * c, A.dsum ? sv[k].at(e) : 0.f));
                }
                store_piece<SHIFT>(xv[k], dx, j * VEC - a0, p.dim);
            }
        }
    }
    float* part = A.part + int64_t(blockIdx.x) * p.dim;
    if constexpr (LPR > 0) {  // the CTA's rows' shares, in row order
        float* share = reinterpret_cast<float*>(dyn);  // [per][dim]
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = at0 + k * step;
            if (j < nvec)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (!SHIFT || unsigned(j * VEC - a0 + e) < unsigned(p.dim)) share[mine * p.dim + j * VEC - a0 + e] = dw[k][e];
        }
        __syncthreads();
        for (int i = tid; i < p.dim; i += blockDim.x) {
            float t = 0.f;
            for (int g = 0; g < per; ++g) t += share[g * p.dim + i];
            part[i] = t;
        }
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int j = at0 + k * step;
            if (j < nvec)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (!SHIFT || unsigned(j * VEC - a0 + e) < unsigned(p.dim)) part[j * VEC - a0 + e] = dw[k][e];
        }
    }
}

// ---- rows too long for the registers: value by value, a row read again (from L2) per phase
__device__ __forceinline__ float weight_at(const NormArgs& A, int i) {
    float w[1];
    load_weight<1>(A.p, A.weight, i, w);
    return w[0];
}

template <typename T>
__global__ void __launch_bounds__(LOOP_T) k_norm_fwd_loop(const NormArgs A) {
    const gdn_norm_problem& p = A.p;
    __shared__ float red[2][32];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(A.x) + row * p.x_stride;
    const T* res = A.residual ? static_cast<const T*>(A.residual) + row * p.residual_stride : nullptr;
    auto at = [&](int i) { return res ? to_f(x[i]) + to_f(res[i]) : to_f(x[i]); };
    float ss = 0.f;
    for (int i = threadIdx.x; i < p.dim; i += LOOP_T) ss = fmaf(at(i), at(i), ss);
    const float r = rsqrtf(row_red<false, 0>(ss, red[0]) * A.inv_dim + p.eps);
    auto y_at = [&](int i) { return at(i) * r * weight_at(A, i); };
    if (p.out_dtype == GDN_E4M3) {
        const int group = p.group ? p.group : p.dim, groups = p.dim / group;
        for (int g = 0; g < groups; ++g) {
            float m = 0.f;
            for (int i = threadIdx.x; i < group; i += LOOP_T) m = max_nan(m, fabsf(y_at(g * group + i)));
            __syncthreads();  // the last group's maxima have been read
            const float sc = scale_of(row_red<true, 0>(m, red[1]));
            if (threadIdx.x == 0) A.y_scale[row * groups + g] = sc;
            for (int i = threadIdx.x; i < group; i += LOOP_T) {
                const float one[1] = {y_at(g * group + i)};
                store8<1>(static_cast<uint8_t*>(A.y) + row * p.dim + g * group + i, one, rcp(sc));
            }
        }
        __syncthreads();  // sum may be x or residual, which other threads have read above
    }
    for (int i = threadIdx.x; i < p.dim; i += LOOP_T) {
        const float v = at(i), y = y_at(i);
        if (A.sum) static_cast<T*>(A.sum)[row * p.dim + i] = from_f<T>(v);
        if (p.out_dtype != GDN_E4M3) static_cast<T*>(A.y)[row * p.dim + i] = from_f<T>(y);
    }
}

template <typename T>
__global__ void __launch_bounds__(LOOP_T) k_norm_bwd_loop(const NormArgs A) {
    tc::pdl_launch_dependents();
    const gdn_norm_problem& p = A.p;
    __shared__ float red[2][32];
    float* part = A.part + int64_t(blockIdx.x) * p.dim;
    for (int i = threadIdx.x; i < p.dim; i += LOOP_T) part[i] = 0.f;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(A.x) + row * p.x_stride;
        const T* dy = static_cast<const T*>(A.dy) + row * p.dy_stride;
        const T* ds = A.dsum ? static_cast<const T*>(A.dsum) + row * p.dsum_stride : nullptr;
        float ss = 0.f, c = 0.f;
        for (int i = threadIdx.x; i < p.dim; i += LOOP_T) {
            const float v = to_f(x[i]);
            ss = fmaf(v, v, ss);
            c = fmaf(weight_at(A, i) * to_f(dy[i]), v, c);
        }
        const float r = rsqrtf(row_red<false, 0>(ss, red[0]) * A.inv_dim + p.eps);
        c = row_red<false, 0>(c, red[1]) * r * A.inv_dim;
        for (int i = threadIdx.x; i < p.dim; i += LOOP_T) {
            const float n = to_f(x[i]) * r, d = to_f(dy[i]), add = ds ? to_f(ds[i]) : 0.f;
            part[i] = fmaf(d, n, part[i]);
            static_cast<T*>(A.dx)[row * p.dim + i] = from_f<T>(fmaf(r, weight_at(A, i) * d - n * c, add));
        }
        __syncthreads();
    }
}

// How a problem's rows are laid over threads.
struct Layout {
    int vec, nv, lpr, threads;  // lpr 0: a CTA per row; vec 0: the looping kernels
    bool shift;
    int per() const { return lpr ? threads / lpr : 1; }
};
Layout layout_of(int64_t rows, int dim, int vec, bool shift, bool backward) {
    Layout L{vec, 1, 0, ROWS_T, shift};
    const bool wide = vec > 1;
    const int n = shift ? (dim + 2 * vec - 2) / vec : dim / vec;  // pieces of a row at most
    if (n <= 32) {
        L.lpr = n <= 8 ? 8 : n <= 16 ? 16 : 32;
        return L;
    }
    // a warp per row: two pieces of 16 bytes a lane, up to 16 values otherwise
    if (n <= (wide ? 64 : 512)) {
        L.lpr = 32;
        for (L.nv = 2; n > 32 * L.nv; L.nv *= 2) {}
        return L;
    }
    // a CTA per row: two pieces a thread while its threads hold the row so, else more.  Rows that leave
    // multiprocessors free take one, for the shorter way through the kernel (16 rows of 2048: 2.5 us
    // instead of 2.9; 8191 rows of 5120: 62 us instead of 53).
    const bool few = rows <= sm_count_cached();
    for (L.nv = !wide ? 8 : few ? 1 : 2; L.nv <= (wide ? 4 : 16); L.nv *= 2) {
        L.threads = ((n + L.nv - 1) / L.nv + 31) / 32 * 32;
        if (L.threads <= max_threads(L.vec, L.nv, 0, backward)) return L;
    }
    L.vec = 0;
    L.shift = false;
    L.threads = LOOP_T;
    return L;
}

int full_vec(int dtype) { return dtype == GDN_BF16 ? 8 : 4; }

// CTAs of a kernel that a multiprocessor holds (looked up once per kernel, device and launch shape).
int resident(const void* kern, int threads, size_t smem) {
    static std::mutex mu;
    static std::map<std::tuple<const void*, int, int, size_t>, int> known;
    int dev = 0, n = 1;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    std::lock_guard<std::mutex> lock(mu);
    auto& r = known[{kern, dev, threads, smem}];
    if (r == 0) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) == cudaSuccess && n > 0 ? n : 1;
    return r;
}

template <int OUT8, typename T, int VEC, int NV, int LPR, bool SHIFT>
cudaError_t fwd_launch(const NormArgs& A, const Layout& L, cudaStream_t st) {
    const int64_t blocks = (A.p.rows + L.per() - 1) / L.per();
    const size_t smem = OUT8 == 3 ? size_t(L.per()) * (A.p.dim / A.p.group) * 4 : 0;
    if (smem > 40 * 1024) {  // (set once, so to the most that the kernel is launched with: a group to a value)
        const cudaError_t e = smem_attr(k_norm_fwd<T, VEC, NV, LPR, SHIFT, OUT8>, max_threads(VEC, NV, LPR, false) * NV * VEC * 4);
        if (e != cudaSuccess) return e;
    }
    k_norm_fwd<T, VEC, NV, LPR, SHIFT, OUT8><<<unsigned(blocks), L.threads, smem, st>>>(A);
    return cudaGetLastError();
}
template <typename T, int VEC, int NV, int LPR, bool SHIFT>
cudaError_t fwd_out(const NormArgs& A, const Layout& L, cudaStream_t st) {
    if (A.p.out_dtype != GDN_E4M3) return fwd_launch<0, T, VEC, NV, LPR, SHIFT>(A, L, st);
    if (A.p.group == 0 || A.p.group == A.p.dim) return fwd_launch<1, T, VEC, NV, LPR, SHIFT>(A, L, st);
    if constexpr (SHIFT) {
        return cudaErrorNotSupported;  // groups of rows that lie off 16-byte pieces go value by value
    } else {
        const int lanes = A.p.group % VEC ? 0 : A.p.group / VEC;
        const int whole = LPR ? LPR : 32;
        if (lanes > 0 && lanes <= whole && (lanes & (lanes - 1)) == 0) return fwd_launch<2, T, VEC, NV, LPR, SHIFT>(A, L, st);
        return fwd_launch<3, T, VEC, NV, LPR, SHIFT>(A, L, st);
    }
}

template <typename T, int VEC, int NV, int LPR, bool SHIFT, bool RINGED>
cudaError_t bwd_launch(const NormArgs& A, const Layout& L, int& parts, cudaStream_t st) {
    const size_t smem = LPR ? size_t(L.per()) * A.p.dim * 4 : RINGED ? size_t(RING) * 3 * NV * L.threads * 16 : 0;
    if (smem > 40 * 1024) {  // (set once, so to the most that the kernel is launched with)
        const cudaError_t e = smem_attr(k_norm_bwd<T, VEC, NV, LPR, SHIFT, RINGED>, RING * 3 * NV * max_threads(VEC, NV, LPR, true) * 16);
        if (e != cudaSuccess) return e;
    }
    const int fit = resident(reinterpret_cast<const void*>(k_norm_bwd<T, VEC, NV, LPR, SHIFT, RINGED>), L.threads, smem) * sm_count_cached();
    if (parts > fit) parts = fit;  // one wave: the rows are dealt out to the CTAs in turn
    // four rows to a CTA at least where the multiprocessors have one each: a CTA's share of dweight costs as much
    // as a row or two (2003 rows of 1024: 10.1 us instead of 11.7)
    const int64_t quarter = A.p.rows / 4, sms = sm_count_cached();
    if (parts > quarter && parts > sms) parts = int(quarter > sms ? quarter : sms);
    if (SHIFT) parts = parts > 8 ? parts / 8 * 8 : 8;
    k_norm_bwd<T, VEC, NV, LPR, SHIFT, RINGED><<<parts, L.threads, smem, st>>>(A);
    return cudaGetLastError();
}

template <typename T, int VEC, int NV, int LPR, bool SHIFT>
cudaError_t bwd_out(const NormArgs& A, const Layout& L, int& parts, cudaStream_t st) {
    constexpr bool CAN = LPR == 0 && VEC > 1 && NV <= 2;
    if constexpr (CAN && SHIFT) {
        return bwd_launch<T, VEC, NV, LPR, SHIFT, true>(A, L, parts, st);
    } else if constexpr (CAN && NV == 2 && sizeof(T) == 2) {
        if (L.threads > 256 && L.threads <= 384) return bwd_launch<T, VEC, NV, LPR, SHIFT, true>(A, L, parts, st);
        return bwd_launch<T, VEC, NV, LPR, SHIFT, false>(A, L, parts, st);
    } else {
        return bwd_launch<T, VEC, NV, LPR, SHIFT, false>(A, L, parts, st);
    }
}

// Calls f<VEC, NV, LPR, SHIFT> for the layout.  (The forward takes SHIFT for rows of more than 512 values alone,
// which are more than 64 pieces: a CTA each.)
#define NORM_CTA(F, T, FULL, SHIFT, ...)                                           \
    do {                                                                            \
        if (L.nv == 1) return F<T, FULL, 1, 0, SHIFT>(__VA_ARGS__);                 \
        if (L.nv == 2) return F<T, FULL, 2, 0, SHIFT>(__VA_ARGS__);                 \
        return F<T, FULL, 4, 0, SHIFT>(__VA_ARGS__);                                \
    } while (0)
#define NORM_WIDE(F, T, FULL, SHIFT, ...)                                          \
    do {                                                                            \
        if (L.lpr == 8) return F<T, FULL, 1, 8, SHIFT>(__VA_ARGS__);                \
        if (L.lpr == 16) return F<T, FULL, 1, 16, SHIFT>(__VA_ARGS__);              \
        if (L.lpr == 32 && L.nv == 1) return F<T, FULL, 1, 32, SHIFT>(__VA_ARGS__); \
        if (L.lpr == 32) return F<T, FULL, 2, 32, SHIFT>(__VA_ARGS__);              \
        NORM_CTA(F, T, FULL, SHIFT, __VA_ARGS__);                                   \
    } while (0)
#define NORM_LAYOUTS(F, T, FULL, SHIFTED, ...)                                     \
    do {                                                                            \
        if (L.shift) SHIFTED(F, T, FULL, true, __VA_ARGS__);                        \
        if (L.vec > 1) NORM_WIDE(F, T, FULL, false, __VA_ARGS__);                   \
        if (L.lpr == 8) return F<T, 1, 1, 8, false>(__VA_ARGS__);                   \
        if (L.lpr == 16) return F<T, 1, 1, 16, false>(__VA_ARGS__);                 \
        if (L.lpr == 32 && L.nv <= 2) return F<T, 1, 2, 32, false>(__VA_ARGS__);    \
        if (L.lpr == 32 && L.nv <= 8) return F<T, 1, 8, 32, false>(__VA_ARGS__);    \
        if (L.lpr == 32) return F<T, 1, 16, 32, false>(__VA_ARGS__);                \
        if (L.nv == 8) return F<T, 1, 8, 0, false>(__VA_ARGS__);                    \
        return F<T, 1, 16, 0, false>(__VA_ARGS__);                                  \
    } while (0)

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T>
cudaError_t fwd_type(const NormArgs& A, cudaStream_t st) {
    const gdn_norm_problem& p = A.p;
    const int full = full_vec(p.dtype);
    const bool rows16 = on16(A.x) && on16(A.residual) && on16(A.sum) && on16(A.y);
    const bool vectors = rows16 && on16(A.weight) && p.dim % full == 0 && p.x_stride % full == 0 && p.residual_stride % full == 0;
    const bool groups = p.out_dtype == GDN_E4M3 && p.group != 0 && p.group != p.dim;
    // short rows are quicker value by value, a warp to a row (38544 rows of 235: 15.1 us instead of 17.8; 30000
    // of 1001: 72 instead of 40)
    const bool shift = p.dim > 512 && !vectors && rows16 && !groups && p.x_stride == p.dim && (!A.residual || p.residual_stride == p.dim);
    const Layout L = layout_of(p.rows, p.dim, vectors || shift ? full : 1, shift, false);
    if (L.vec == 0) {
        k_norm_fwd_loop<T><<<unsigned(p.rows), LOOP_T, 0, st>>>(A);
        return cudaGetLastError();
    }
    NORM_LAYOUTS(fwd_out, T, (sizeof(T) == 2 ? 8 : 4), NORM_CTA, A, L, st);
}

int parts_of(const gdn_norm_problem& p, const Layout& L) {
    const int64_t groups = (p.rows + L.per() - 1) / L.per();
    int64_t most = int64_t(sm_count_cached()) * (2048 / L.threads);
    if (groups < most) most = groups;
    return int(most > 0 ? most : 1);
}

template <typename T>
cudaError_t bwd_type(const NormArgs& A, int& parts, cudaStream_t st) {
    const gdn_norm_problem& p = A.p;
    const int full = full_vec(p.dtype);
    const bool rows16 = on16(A.x) && on16(A.dy) && on16(A.dsum) && on16(A.dx);
    const bool vectors = rows16 && on16(A.weight) && p.dim % full == 0 && p.x_stride % full == 0 && p.dy_stride % full == 0 && p.dsum_stride % full == 0;
    const bool shift = !vectors && rows16 && p.x_stride == p.dim && p.dy_stride == p.dim && (!A.dsum || p.dsum_stride == p.dim);
    const Layout L = layout_of(p.rows, p.dim, vectors || shift ? full : 1, shift, true);
    parts = parts_of(p, L);
    if (L.vec == 0) {
        k_norm_bwd_loop<T><<<parts, LOOP_T, 0, st>>>(A);
        return cudaGetLastError();
    }
    NORM_LAYOUTS(bwd_out, T, (sizeof(T) == 2 ? 8 : 4), NORM_WIDE, A, L, parts, st);
}

}  // namespace
}  // namespace gdn
