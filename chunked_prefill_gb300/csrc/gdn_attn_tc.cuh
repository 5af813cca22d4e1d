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

// A wait that gives up after `limit` cycles (4e9: 2 s).
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t phase, long long limit = 4000000000ll) {
    if (tc::mbar_try_wait(bar, phase)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i)
            if (tc::mbar_try_wait(bar, phase)) return true;
        if (clock64() - t0 > limit) return false;
    }
}
// The same without suspending the thread, whose waking is on the critical path.
__device__ __forceinline__ bool bounded_spin(uint64_t* bar, uint32_t phase) {
    if (tc::mbar_test(bar, phase)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (tc::mbar_test(bar, phase)) return true;
        if (clock64() - t0 > 4000000000ll) return false;
    }
}
// by a whole warp
__device__ __forceinline__ bool warp_spin(uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, bounded_spin(bar, phase)); }
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, bounded_wait(bar, phase)); }

// Of the failure report's test: a wait for a barrier at which nothing arrives.
__global__ void __launch_bounds__(32) k_wait_out(long long limit) {
    __shared__ uint64_t bar;
    if (threadIdx.x > 0) return;
    tc::mbar_init(&bar, 1);
    tc::mbar_fence_init();
    if (!bounded_wait(&bar, 0, limit)) g_gave_up = 1;
}
inline cudaError_t launch_wait_out(int32_t limit_us, cudaStream_t st) {
    k_wait_out<<<1, 32, 0, st>>>(2000ll * limit_us);
    return cudaGetLastError();
}

// The thread of a warp that issues its products.  The warp runs their loop as a whole and on values that the compiler
// sees to be the same in all lanes (broadcast by same()), so that descriptors and addresses stay in uniform registers:
// where one lane ran it alone every product took several moves into them, 120 to 140 cycles for 128 x 128 x 16 instead
// of the tensor cores' 64.
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int same(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t same(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Registers of a thread from here on, by all warps of a warpgroup.  What they add up to stays within what the block
// was launched with.
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// the largest of N values; NaN is passed over
template <int N>
__device__ __forceinline__ float max_of(const float* v) {
    float t[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int c = 4; c + 8 <= N; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = max3(t[e], v[c + e], v[c + 4 + e]);
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = fmaxf(t[e], v[N - 4 + e]);
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Of 32 columns the bits of [lo, hi].  Masks are made of these words, with one test to a column, in half of the code that two
// comparisons take: it runs once or twice for a tile of queries and comes from far away each time (128 columns: 4000 cycles for a masked
// tile, 1200 for others).
__device__ __forceinline__ uint32_t span_of(int lo, int hi) {
    return (lo <= 0 ? 0xffffffffu : lo < 32 ? 0xffffffffu << lo : 0u) & (hi >= 31 ? 0xffffffffu : hi >= 0 ? 0xffffffffu >> (31 - hi) : 0u);
}
// 32 bytes to global memory (32-byte aligned)
__device__ __forceinline__ void stg256(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// 32 fp32 values as bf16 to global memory, 16-byte aligned, or 32-byte aligned (wide): whole sectors a store
__device__ __forceinline__ void store_bf16x32(__nv_bfloat16* p, const float* x, float f, bool wide) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = tc::pack_bf16(x[2 * i] * f, x[2 * i + 1] * f);
    if (wide) {
        stg256(p, w);
        stg256(p + 16, w + 8);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(p + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}
__device__ __forceinline__ bool wide_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }
__device__ __forceinline__ void prefetch_map(const void* m) { asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory"); }

// Operands of 128-byte swizzled tiles of R rows (see tc05.cuh): the K-major step of 16 columns at c, and the
// MN-major step of 16 rows at r.
template <int R> __device__ __forceinline__ uint64_t desc_k(uint32_t tile, int c) { return tc::make_desc(tile + (c >> 6) * (R * 128) + (c & 63) * 2, 0, 1024); }
template <int R> __device__ __forceinline__ uint64_t desc_mn(uint32_t tile, int r) { return tc::make_desc(tile + r * 128, R * 128, 1024); }
// The same for a step further in, from the tile's first: addresses are the lowest field, in units of 16 bytes.
template <int R> __device__ __forceinline__ uint64_t step_k(uint64_t first, int c) { return first + (((c >> 6) * (R * 128) + (c & 63) * 2) >> 4); }
__device__ __forceinline__ uint64_t step_mn(uint64_t first, int r) { return first + (r * 128 >> 4); }

__device__ __forceinline__ bool bad_pair(uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ uint32_t clean_pair(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}
// By one warp: of rows [64 half, 64 half + 64) of a swizzled tile of 128 rows x COLS bf16 values, those from `valid` on
// become zeros, and infinite and NaN values of the others too; sets the bits of rows (of the 64) that had any, the
// same in every lane.  8 pieces of 16 bytes a lane are looked at together: an exponent of all ones carries into the bit above.
template <int COLS>
__device__ __forceinline__ void clean_tile(uint32_t tile, int valid, int half, uint32_t (&bad)[2]) {
    const int lane = threadIdx.x & 31, row0 = 64 * half + (lane >> 3);
#pragma unroll 1
    for (int part = 0; part < COLS / 64; ++part)
#pragma unroll 1
        for (int i = 0; i < 16; i += 8) {  // 4 rows a piece
            const uint32_t at = tile + part * 16384 + half * 8192 + i * 512 + lane * 16;
            uint32_t any = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint4 v = tc::lds128(at + x * 512);
                any |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) | ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
            }
            any &= 0x80008000u;
            if (!any && row0 + 4 * (i + 7) < valid) continue;
#pragma unroll 1
            for (int x = 0; x < 8; ++x) {
                const int row = row0 + 4 * (i + x);
                const uint4 v = tc::lds128(at + x * 512);
                if (row >= valid) {
                    tc::sts128(at + x * 512, make_uint4(0u, 0u, 0u, 0u));
                } else if (bad_pair(v.x) || bad_pair(v.y) || bad_pair(v.z) || bad_pair(v.w)) {
                    tc::sts128(at + x * 512, make_uint4(clean_pair(v.x), clean_pair(v.y), clean_pair(v.z), clean_pair(v.w)));
                    bad[(row & 63) >> 5] |= 1u << (row & 31);
                }
            }
        }
    if (__any_sync(0xffffffffu, (bad[0] | bad[1]) != 0u)) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) bad[w] |= __shfl_xor_sync(0xffffffffu, bad[w], o);
    }
}

}  // namespace
}  // namespace gdn
