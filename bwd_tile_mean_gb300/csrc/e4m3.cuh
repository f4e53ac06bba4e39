// e4m3.cuh -- the 8-bit cache's numbers: e4m3 bytes with a power of two per
// block of 16 tokens and key/value head. Internal.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace vsa {

// Two e4m3 bytes (the lower 16 bits) as fp16: exact.
__device__ __forceinline__ uint32_t half2_of(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    return h;
}
__device__ __forceinline__ float2 float2_of(uint32_t two) {
    const uint32_t h = half2_of(two);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// Two floats as e4m3 bytes, to nearest (ties to even); beyond 448 as 448, NaN as NaN.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// 2^e, -126 <= e <= 127
__device__ __forceinline__ float power_of(int e) { return __int_as_float((e + 127) << 23); }
// The least power of two from 2^-126 on with top <= 448 times it (448 = 1.75 * 2^8): top = 1.m 2^n gives 2^(n - 8), or
// the next one where 1.m is above 1.75.
__device__ __forceinline__ float scale_of(float top) {
    const uint32_t u = __float_as_uint(top);
    const int field = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
    return __uint_as_float((uint32_t)(field > 1 ? field : 1) << 23);
}

}  // namespace vsa
