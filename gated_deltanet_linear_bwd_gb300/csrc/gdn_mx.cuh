// gdn_mx.cuh -- microscaled (MX) blocks on the device: the exponent of a block,
// its elements, and where a scale byte lives.
#pragma once

#include <stdint.h>

namespace gdn {
namespace mx {

// Offset of the scale byte of (row, block): tiles of 128 rows x 4 blocks, `ktiles`
// of them to a row of tiles.
__host__ __device__ __forceinline__ long long scale_offset(long long row, int block, int ktiles) {
    return ((row >> 7) * ktiles + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
           (block & 3);
}

// Scale byte of a block whose largest magnitude has the bits `amax` (sign
// cleared): the least exponent e with amax 2^-e <= 448 = 1.75 2^8 (e4m3) or 6 =
// 1.5 2^2 (e2m1), straight from the fp32 fields.  NaN and infinities, whose bits
// compare above every number's, give 255.
template <bool FP4>
__device__ __forceinline__ int scale_byte(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255;
    const int e = (int)(amax >> 23);
    const bool up = (amax & 0x7fffffu) > (FP4 ? 0x400000u : 0x600000u);
    return max(0, e - (FP4 ? 2 : 8) + (up ? 1 : 0));
}
// 2^(127 - byte), the factor from values to elements (0 for a NaN block, whose
// elements are then zeros).
__device__ __forceinline__ float scale_factor(int byte) {
    return byte == 255 ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);
}

// Four e4m3 elements, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n"
        ".reg .b16 lo, hi;\n"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        "mov.b32 %0, {lo, hi};\n"
        "}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// Eight e2m1 elements, the first in the low half of the low byte.
__device__ __forceinline__ uint32_t e2m1x8(float v0, float v1, float v2, float v3, float v4, float v5, float v6,
                                           float v7) {
    uint32_t r;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}\n"
        : "=r"(r)
        : "f"(v0), "f"(v1), "f"(v2), "f"(v3), "f"(v4), "f"(v5), "f"(v6), "f"(v7));
    return r;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

}  // namespace mx
}  // namespace gdn
