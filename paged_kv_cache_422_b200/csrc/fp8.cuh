// The 8-bit KV cache: e4m3 codes with one power-of-two scale per (slot, KV head).
//
// A row x of head_dim values is held as codes c_d and one scale byte b (an exponent with
// bias 127): x_d ~ c_d * 2^(b - 127).  With amax the largest finite magnitude of the row,
// b - 127 = max(-118, ceil(log2(amax / 448))), so that no finite value saturates.  A power
// of two keeps the relative precision of the floating-point codes that any other scale
// would give, and makes reading back exact: a code has 4 significant bits, so c * 2^e is a
// bf16 value (and an fp16 value before the scale).  From -118 on that holds for every code,
// subnormals included: codes are multiples of 2^-9, their values of 2^-127, 2^6 above the
// smallest bf16 magnitude; rows below 448 * 2^-118 lose relative precision instead.
#pragma once

#include <cuda_fp16.h>

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

// A row's scale 2^(byte - 127) for widening its codes to bf16.  The products are exact (4
// significant bits), so the upper halves of their float32 forms are their bf16 forms.  A scale
// that is an fp16 value (2^-24 .. 2^15: rows of magnitude up to 2^-16 .. 2^24) goes through the
// mixed-precision FMA, which widens and scales in one instruction: 4.3 ns per warp and 32-bit
// word against 6.2 for conversion, multiplication and packing.  (The addend is -0, which keeps
// the sign of a zero.)
struct RowScale {
    uint16_t half;    // 0: outside fp16
    float value;
};
__device__ __forceinline__ RowScale row_scale(uint32_t byte) {
    RowScale r;
    r.value = scale_value(byte);
    r.half = byte > 142 || byte < 103 ? 0 : (uint16_t)(byte >= 113 ? (byte - 112) << 10 : 1u << (byte - 103));
    return r;
}
__device__ __forceinline__ uint32_t scale_half2(uint32_t h2, uint16_t f) {
    float x, y;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "fma.rn.f32.f16 %0, a, %3, %4;\n\tfma.rn.f32.f16 %1, b, %3, %4;\n\t}"
        : "=f"(x), "=f"(y) : "r"(h2), "h"(f), "f"(-0.f));
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}

// 16 codes times the scale as bf16; f from row_scale().half.
__device__ __forceinline__ void widen16(const uint4& u, uint16_t f, uint4& lo, uint4& hi) {
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e4m3x4_to_half2(in[i], w[2 * i], w[2 * i + 1]);
        w[2 * i] = scale_half2(w[2 * i], f);
        w[2 * i + 1] = scale_half2(w[2 * i + 1], f);
    }
    lo = make_uint4(w[0], w[1], w[2], w[3]);
    hi = make_uint4(w[4], w[5], w[6], w[7]);
}
// The same for any scale.
__device__ __forceinline__ void widen16_any(const uint4& u, float f, uint4& lo, uint4& hi) {
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
        e4m3x4_to_half2(in[i], h[0], h[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 x = __half22float2(*reinterpret_cast<__half2*>(&h[k]));
            w[2 * i + k] = pack_bf16x2(x.x * f, x.y * f);
        }
    }
    lo = make_uint4(w[0], w[1], w[2], w[3]);
    hi = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace nvpa
