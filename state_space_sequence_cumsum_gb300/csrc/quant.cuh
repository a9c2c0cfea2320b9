// Values in 8-bit floats with a power-of-two scale, as k_block_quantize.cu
// defines them.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace ssd {

// Bits of the scale and of its inverse for the largest magnitude's bits: with
// amax = 1.f * 2^k, e = k - TOP + (f > 1.75), TOP = 8 or 15.
template <bool kE5M2> __device__ __forceinline__ void scale_of(uint32_t amax, float &scale, float &inverse)
{
    constexpr int top = kE5M2 ? 15 : 8;
    // the biased exponent of amax, one more where its fraction is over 0.75
    const int k = (int)((amax + 0x1fffffu) >> 23);
    const int e = max(k - top, 9);  // biased; 2^-118
    const bool bad = amax >= 0x7f800000u;
    scale = __uint_as_float(bad ? 0x7fffffffu : (uint32_t)e << 23);
    inverse = __uint_as_float(bad ? 0x7fffffffu : (uint32_t)(254 - e) << 23);
}

// Four values to four bytes, the first in the low one.
template <bool kE5M2> __device__ __forceinline__ uint32_t to_bytes(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    if (kE5M2) {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    return (uint32_t)lo | (uint32_t)hi << 16;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace ssd
