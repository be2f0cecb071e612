// sv_rotate.cuh -- what the appending kernels share: exact angles of far positions, two fp32 operations
// per instruction, and how the elements of a rotated pair lie in the threads.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace svc {

// inv_freq / (2 pi) as a 64-bit binary fraction of a turn, modulo 1.
__device__ __forceinline__ uint64_t turns_of(float f) {
    const uint64_t inv2pi = 0x28BE60DB9391054Aull;   // round(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f);
    const int ex = (u >> 23) & 0xff;
    const uint64_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int sh = 150 - (ex ? ex : 1);              // f = m 2^-sh
    const uint64_t lo = m * inv2pi, hi = __umul64hi(m, inv2pi);
    uint64_t t;
    if (sh <= 0) t = sh > -64 ? lo << -sh : 0;
    else if (sh < 64) t = (lo >> sh) | (hi << (64 - sh));
    else t = sh < 128 ? hi >> (sh - 64) : 0;
    return (u >> 31) ? 0 - t : t;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

// How the two elements of a pair come together: as neighbours; in one thread, which holds 4 elements
// of each half (rotary_dim a multiple of 8); or through shared memory, at any distance.
enum { PAIR_NEXT, PAIR_HALVES, PAIR_ANY };

}  // namespace svc
