// Microscaled 4-bit values on the device. A code is E2M1: sign, two exponent bits (bias 1), one mantissa bit, so
// 0, .5, 1, 1.5, 2, 3, 4 or 6; a scale byte b is 2^(b - 127), 255 is NaN.
#pragma once

#include <type_traits>

#include "common.cuh"

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

// The factor that decode8 multiplies with (both halves), for b <= kPlain: the codes' bits are placed as those of a
// number 2^126 (bf16) or 2^14 (fp16) times smaller, mostly subnormal, and one multiplication gives the value,
// correctly rounded (the type's products keep subnormals).
constexpr uint32_t kPlain = 128;
template <typename T>
__device__ __forceinline__ uint32_t factor2(uint32_t b) {
    if constexpr (std::is_same<T, __half>::value) {
        const int e = (int)b - 113;  // 2^e; below 2^-24 every value rounds to zero
        const uint32_t h = e >= -14 ? (uint32_t)(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
        return h | h << 16;
    } else {
        const uint32_t h = (b + 126) << 7;
        return h | h << 16;
    }
}

template <typename T>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 r = __hmul2_rn(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b));
        return reinterpret_cast<const uint32_t&>(r);
    } else {
        const __nv_bfloat162 r =
            __hmul2_rn(reinterpret_cast<const __nv_bfloat162&>(a), reinterpret_cast<const __nv_bfloat162&>(b));
        return reinterpret_cast<const uint32_t&>(r);
    }
}

// Eight codes (the first in the lowest bits) as eight 16-bit values, two a word.
template <typename T>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t factor, uint32_t (&o)[4]) {
    constexpr int up = std::is_same<T, __half>::value ? 9 : 6;  // to the lowest exponent and highest mantissa bits
    constexpr uint32_t mag = 0x00070007u << up;
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // codes j and j + 4
        const int by = up - 4 * j;
        const uint32_t m = (by >= 0 ? w << (by & 31) : w >> (-by & 31)) & mag;
        r[j] = mul2<T>(((w << (12 - 4 * j)) & 0x80008000u) | m, factor);
    }
    o[0] = __byte_perm(r[0], r[1], 0x5410);
    o[1] = __byte_perm(r[2], r[3], 0x5410);
    o[2] = __byte_perm(r[0], r[1], 0x7632);
    o[3] = __byte_perm(r[2], r[3], 0x7632);
}

// The same for scales above kPlain (values from 2 on, infinities and NaN), by way of fp32.
template <typename T>
__device__ __forceinline__ void decode8_large(uint32_t w, uint32_t b, uint32_t (&o)[4]) {
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

}  // namespace mx4
}  // namespace spops
