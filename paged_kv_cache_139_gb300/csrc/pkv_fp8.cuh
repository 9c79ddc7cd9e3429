// The 8-bit cache: e4m3 values with a power-of-two scale per (block, kv head)
// for keys and one for values, in [num_blocks][kv heads rounded up to even][2]
// fp32 (key, value).  A block's scales are one 8-byte load per kv head, and
// its record is a multiple of 16 bytes, so block copies move it as they move
// the block.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

constexpr int kMinScaleExp = -60;      // the smallest block scale is 2^-60

__host__ __device__ constexpr int scale_heads(int num_kv_heads) { return num_kv_heads + (num_kv_heads & 1); }

// The smallest power of two s >= 2^-60 with amax <= 448 s (448, the largest
// e4m3 value, is 1.75 * 2^8): with amax = m * 2^e, 2^(e - 8) while m <= 1.75,
// else 2^(e - 7).  A power of two costs e4m3 no precision, makes x / s exact
// and re-rounds a value under a larger scale without loss, but for what
// becomes subnormal.  amax must be finite and not negative.
__device__ __forceinline__ float pow2_scale(float amax) {
    const unsigned b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < kMinScaleExp ? kMinScaleExp : e;
    return __uint_as_float((unsigned)(e + 127) << 23);
}

// Four fp32 to four e4m3 (x in the low byte): round to nearest even,
// magnitudes above 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float x, float y, float z, float w) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y), "f"(x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(w), "f"(z));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The two e4m3 values in the low / high half of w as two fp16 (exact; the
// lower byte in the low half).
__device__ __forceinline__ uint32_t e4m3x2_lo(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t e4m3x2_hi(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(w));
    return d;
}

}  // namespace pkv
