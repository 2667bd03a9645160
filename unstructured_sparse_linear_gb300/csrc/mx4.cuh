// Microscaled 4-bit values on the device. A code is E2M1: sign, two exponent bits (bias 1), one mantissa bit, so
// 0, .5, 1, 1.5, 2, 3, 4 or 6; a scale byte b is 2^(b - 127), 255 is NaN.
#pragma once

#include <type_traits>

#include "common.cuh"

// Codes, scales and X are read by plain loads: these kernels begin while the one before them in the stream may still be
// writing those arrays, and read-only loads (ld.global.nc, __ldg) promise that nobody does as long as a kernel runs.

namespace spops {
namespace mx4 {

// 2^(b - 127) in fp32 (b = 0: the subnormal 2^-127; 255: NaN).
__device__ __forceinline__ float scale_f32(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}

// A code times 2^(b - 127) in fp32: exact, or infinite. The code's exponent and mantissa bits are those of a
// subnormal number that is 2^126 times smaller.
__device__ __forceinline__ float value_f32(uint32_t code, float scale) {
    return __uint_as_float((code & 7u) << 22 | (code & 8u) << 28) * 0x1p126f * scale;
}

// Scales that fp16 holds exactly, 2^-24 to 2^15: decode8 multiplies with them as fp16 numbers. Others (and NaN) go by way
// of decode8_any.
__device__ __forceinline__ bool plain(uint32_t b) { return b - 103u <= 39u; }
// The scale of a plain byte as fp16, in both halves.
__device__ __forceinline__ uint32_t factor2(uint32_t b) {
    const uint32_t h = b >= 113u ? (b - 112u) << 10 : 1u << (b - 103u);
    return h | h << 16;
}

// Two codes (byte i of w) as two fp16 values, the first in the low half.
template <int I>
__device__ __forceinline__ uint32_t pair_f16(uint32_t w) {
    uint32_t r;
    if constexpr (I == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Two codes times a plain scale. fp16: one product, correctly rounded. bf16: products of fp16 numbers with fp32 results, which
// are exact, and their upper halves, which hold all of them. (Cycles of a scheduler for eight values, measured: 13.7 and
// 21.7; placing the bits with shifts and masks and one product took 32.)
template <typename T, int I>
__device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t factor) {
    const uint32_t h = pair_f16<I>(w);
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 r = __hmul2_rn(reinterpret_cast<const __half2&>(h), reinterpret_cast<const __half2&>(factor));
        return reinterpret_cast<const uint32_t&>(r);
    } else {
        float lo, hi;  // (plus -0, which keeps a zero's sign)
        asm("{\n\t.reg .b16 a, b, f, g;\n\tmov.b32 {a, b}, %2;\n\tmov.b32 {f, g}, %3;\n\t"
            "fma.rn.f32.f16 %0, a, f, 0f80000000;\n\tfma.rn.f32.f16 %1, b, f, 0f80000000;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(h), "r"(factor));
        return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    }
}

// Eight codes (the first in the lowest bits) as eight 16-bit values, two a word, for a plain scale.
template <typename T>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t factor, uint32_t (&o)[4]) {
    o[0] = pair<T, 0>(w, factor);
    o[1] = pair<T, 1>(w, factor);
    o[2] = pair<T, 2>(w, factor);
    o[3] = pair<T, 3>(w, factor);
}

// The same for any scale, by way of fp32.
template <typename T>
__device__ __forceinline__ void decode8_any(uint32_t w, uint32_t b, uint32_t (&o)[4]) {
    const float s = scale_f32(b);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = value_f32(w >> (4 * j), s);
    const uint4 v = Elt<T>::pack(f);
    o[0] = v.x;
    o[1] = v.y;
    o[2] = v.z;
    o[3] = v.w;
}

// The least magnitude but zero of bf16 numbers, eight of them two a word, as a bit pattern; beyond all of them where there is none.
__device__ __forceinline__ int least8(const uint4& v) {
    const uint32_t a = 0x7fff7fffu;  // (a signed half less 32767 + 1: zeros become the largest)
    const uint32_t m = __vmins2(__vmins2((v.x & a) + a, (v.y & a) + a), __vmins2((v.z & a) + a, (v.w & a) + a));
    return min((int)m >> 16, (int)(m << 16) >> 16) + 32769;
}

}  // namespace mx4
}  // namespace spops
