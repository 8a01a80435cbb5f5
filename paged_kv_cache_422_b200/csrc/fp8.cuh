// The 8-bit KV cache: e4m3 codes with one power-of-two scale per (slot, KV head).
//
// A row x of head_dim values is held as codes c_d and one scale byte b (an exponent with
// bias 127): x_d ~ c_d * 2^(b - 127).  With amax the largest finite magnitude of the row,
// b - 127 = max(-118, ceil(log2(amax / 448))), so that no finite value saturates.  A power
// of two keeps the relative precision of the floating-point codes that any other scale
// would give, and makes reading back exact: a code has 4 significant bits, so c * 2^e is a
// bf16 value (and an fp16 value before the scale).  -118 is the smallest exponent for which
// every code, subnormals included, is still a multiple of the smallest bf16 magnitude.
#pragma once

#include "common.cuh"

namespace nvpa {

constexpr int kMinScaleByte = 9;     // 2^-118
constexpr uint32_t kE4m3Nan = 0x7f;

// The scale byte of a row whose largest finite magnitude has the bf16 bits `amax`:
// 448 = 1.75 * 2^8, so the exponent is that of amax less 8, and one more when the fraction
// is above 0.75 (0x60 of 0x80): adding 0x1f carries into the exponent exactly then.
__host__ __device__ __forceinline__ int scale_byte(uint32_t amax) {
    const int b = (int)((amax + 31u) >> 7) - 8;
    return b > kMinScaleByte ? b : kMinScaleByte;
}

// 2^(b - 127) as float (b in [1, 254])
__device__ __forceinline__ float scale_value(uint32_t b) { return __uint_as_float(b << 23); }

// Two float32 values rounded (nearest-even) to e4m3, lo in the low byte.  NaN becomes 0x7f.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The e4m3 pairs in the low and high halves of w, widened exactly to packed fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

}  // namespace nvpa
