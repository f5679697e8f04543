// The 8-bit row format of activation checkpoints: every 32 consecutive values
// of a row share one power-of-two step 2^e, and each value is a whole multiple
// of it, int8 in [-127, 127]:
//     e = the smallest integer with max|v| <= 127 * 2^e, at least -126
//     code = v / 2^e rounded to nearest even;  scale byte = e + 127
// (127: half of all magnitudes a symmetric int8 can hold are used at worst,
// and the rounding is off by at most 2^e / 2 <= max|v| / 127). The step is a
// power of two so that v / 2^e is exact before the one rounding and a value
// read back, 7 significant bits times 2^e, is exact in bf16 as in float32:
// what a kernel multiplies is what the format holds. A block with an infinity
// or a NaN gets scale byte 255 and reads back as NaN, whatever
// its codes.
//
// A buffer of `rows` rows of n values: the codes [rows, n32] (n32 = n rounded
// up to 32; the padding's codes are 0), rounded up to 256 bytes, then the
// scale bytes [rows, n32 / 32], rounded up to 256 bytes.
#pragma once

#include "moe_device.h"

namespace moe {

constexpr int kRows8Block = 32;

inline size_t rows8_align(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int64_t rows8_stride(int64_t n) { return (n + kRows8Block - 1) / kRows8Block * kRows8Block; }
// byte offset of the scale bytes, and the whole buffer's size
inline size_t rows8_scales_at(int64_t rows, int64_t n) {
    return rows8_align(static_cast<size_t>(rows) * static_cast<size_t>(rows8_stride(n)));
}
inline size_t rows8_bytes(int64_t rows, int64_t n) {
    return rows8_scales_at(rows, n) +
           rows8_align(static_cast<size_t>(rows) * static_cast<size_t>(rows8_stride(n) / kRows8Block));
}

// scale byte of a block whose largest magnitude is amax (>= 0; NaN counts as
// the largest): with amax = 1.m * 2^q, 127 = 1.984375 * 2^6, so e = q - 6, one
// more where 1.m > 1.984375
__device__ __forceinline__ uint32_t rows8_scale(uint32_t amax_bits) {
    const int q = static_cast<int>(amax_bits >> 23);
    const int b = q - 6 + ((amax_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return q == 255 ? 255u : static_cast<uint32_t>(b < 1 ? 1 : b);
}
// 2^-e, by which a value is multiplied before its rounding (0 for a block
// that is not finite); e >= -126 and e <= 121
__device__ __forceinline__ float rows8_inverse(uint32_t scale) {
    return scale == 255u ? 0.0f : __uint_as_float((254u - scale) << 23);
}
// 2^e, or NaN
__device__ __forceinline__ float rows8_step(uint32_t scale) {
    return scale == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(scale << 23);
}
// Four codes as the bytes of a word. v * inverse is exact, so adding 1.5 * 2^23
// (whose last bit is worth 1) in one fused step rounds it to the nearest whole
// number, ties to even, and leaves it in two's complement in the low byte.
__device__ __forceinline__ uint32_t rows8_code4(float a, float b, float c, float d, float inverse) {
    const uint32_t qa = __float_as_uint(__builtin_fmaf(a, inverse, 12582912.0f));
    const uint32_t qb = __float_as_uint(__builtin_fmaf(b, inverse, 12582912.0f));
    const uint32_t qc = __float_as_uint(__builtin_fmaf(c, inverse, 12582912.0f));
    const uint32_t qd = __float_as_uint(__builtin_fmaf(d, inverse, 12582912.0f));
    // v_perm_b32: bytes 0..3 of the second operand, 4..7 of the first
    const uint32_t ab = __builtin_amdgcn_perm(qb, qa, 0x0c0c0400u), cd = __builtin_amdgcn_perm(qd, qc, 0x04000c0cu);
    return ab | cd;
}
__device__ __forceinline__ float rows8_value(uint32_t word, int i, float step) {
    return static_cast<float>(static_cast<int8_t>((word >> (8 * i)) & 0xffu)) * step;
}
// |v| as bits, which order as the magnitudes do, a NaN above an infinity
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace moe
