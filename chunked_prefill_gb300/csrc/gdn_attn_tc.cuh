// What the tensor-core (tcgen05) kernels of attention share.
#pragma once
#include <cuda.h>

#include "gdn_attn.cuh"

namespace gdn {
namespace {

// Every wait of these kernels is bounded (2 s): one that gives up sets this, and the CTA winds down.
__device__ int g_gave_up;

// Whether one gave up since the last time; -1 where that cannot be asked.
inline int take_gave_up() {
    int x = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&x, g_gave_up, sizeof(x)) != cudaSuccess) return -1;
    if (x && cudaMemcpyToSymbol(g_gave_up, &zero, sizeof(zero)) != cudaSuccess) return -1;
    return x;
}

// A wait that gives up after 4e9 cycles (2 s).
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t phase) {
    if (tc::mbar_try_wait(bar, phase)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i)
            if (tc::mbar_try_wait(bar, phase)) return true;
        if (clock64() - t0 > 4000000000ll) return false;
    }
}
// by a whole warp
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, bounded_wait(bar, phase)); }

// 32 lanes x 32 columns from v[0 .. 31]
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
        "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// 32 bytes to global memory (32-byte aligned)
__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 16 fp32 values as bf16 to global memory; a 16-byte aligned address
__device__ __forceinline__ void store_bf16x16(__nv_bfloat16* p, const float* x, float f) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = tc::pack_bf16(x[2 * i] * f, x[2 * i + 1] * f);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Operands of 128-byte swizzled tiles of R rows (see tc05.cuh): the K-major step of 16 columns at c, and the
// MN-major step of 16 rows at r.
template <int R> __device__ __forceinline__ uint64_t desc_k(uint32_t tile, int c) { return tc::make_desc(tile + (c >> 6) * (R * 128) + (c & 63) * 2, 0, 1024); }
template <int R> __device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int r) { return tc::make_desc(tile + r * 128, R * 128, 1024); }

__device__ __forceinline__ bool bad_pair(uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ uint32_t clean_pair(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}
// By one warp: of a swizzled tile of 128 rows x COLS bf16 values, rows [valid, 128) become zeros, and infinite and
// NaN values of the others too; returns which rows (bits) had any, the same in every lane.
template <int COLS>
__device__ __forceinline__ void clean_tile(uint32_t tile, int valid, uint32_t (&bad)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int part = 0; part < COLS / 64; ++part) {
        const uint32_t base = tile + part * 16384 + lane * 16;
#pragma unroll 4
        for (int i = 0; i < 32; ++i) {  // 4 rows at a time
            const uint32_t at = base + i * 512;
            const int row = i * 4 + (lane >> 3);
            uint4 x = tc::lds128(at);
            if (row >= valid) {
                if (x.x | x.y | x.z | x.w) tc::sts128(at, make_uint4(0u, 0u, 0u, 0u));
            } else if (bad_pair(x.x) || bad_pair(x.y) || bad_pair(x.z) || bad_pair(x.w)) {
                tc::sts128(at, make_uint4(clean_pair(x.x), clean_pair(x.y), clean_pair(x.z), clean_pair(x.w)));
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (row >> 5 == w) bad[w] |= 1u << (row & 31);
            }
        }
    }
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bad[w] |= __shfl_xor_sync(0xffffffffu, bad[w], o);
}

}  // namespace
}  // namespace gdn
