// fp8.cuh -- the row format of the 8-bit paged cache.
//
// A row (one token, one KV head) of d bf16 values x is held as d e4m3 codes c
// and one exponent s, x ~ c * 2^s, with s the smallest integer for which
// max|x| <= 448 * 2^s over the row's finite values (448 = 1.75 * 2^8 is e4m3's
// largest value), held within [kScaleMin, kScaleMax].  A power of two costs a
// floating format no precision (only the bottom of its range moves), scaling
// by it is exact, and c * 2^s is exact in bf16, so reading back adds no
// rounding and the attention kernel may apply the scale wherever it likes.
// The bounds keep the spread of scales within one sequence below 2^97, so that
// sums over a sequence can be kept in units of any of its rows in fp32.
#pragma once

#include <cstdint>

namespace treeattn {

// Scale bytes hold s + 127 (e8m0): s in [-56, 40].
constexpr int kScaleByteMin = 127 - 56;
constexpr int kScaleByteMax = 127 + 40;

// 2^(byte - 127) and its inverse, for bytes in [1, 253].
__device__ __forceinline__ float scale_of(int byte) { return __int_as_float(byte << 23); }
__device__ __forceinline__ float inv_scale_of(int byte) {
    return __int_as_float((254 - byte) << 23);
}

// Scale byte of a row whose largest finite |x| has the bf16 bits `amax`
// (0 for a row without finite non-zero values): with |x| = (1 + m/128) * 2^e,
// s = e - 8, one more when 1 + m/128 exceeds 1.75.
__device__ __forceinline__ int scale_byte(uint32_t amax) {
    const int b = static_cast<int>(amax >> 7) - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
    return b < kScaleByteMin ? kScaleByteMin : (b > kScaleByteMax ? kScaleByteMax : b);
}

// Two fp32 values to e4m3 codes (low byte: lo), to nearest even, beyond +-448
// (infinities too) saturated, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes as fp16 pairs (exact): the low code in the low half.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}

// Four codes as two fp16 pairs.
__device__ __forceinline__ void f16x2_of_e4m3x4(uint32_t codes, uint32_t& h0, uint32_t& h1) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(codes));
}

}  // namespace treeattn
