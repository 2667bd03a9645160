// Microscaled 4-bit weights: conversion from and to fp32, fp16 and bf16, and the choice between the products'
// kernels.
//
// A block of 32 consecutive values of a row shares the scale 2^e, e = floor(log2 max|x|) - 2 (the exponent of the largest
// value less that of 4, the grid's last power of two), and each value is rounded to the nearest of 0, .5, 1, 1.5, 2, 3,
// 4, 6 times it (ties to the even mantissa, beyond 6 to 6).
//
// All kernels stream: four lanes share a block, a lane has eight values (16 bytes of a 16-bit type, 4 bytes of codes; from
// codes to fp32 four values), and a warp several steps of 256 values, loaded before any is used. The flat kernels take
// matrices of whole blocks without gaps between the rows, on 16-byte boundaries, as one long row, without any bounds but the
// end: 11008 x 4096 bf16 to 4 bits 22.6 us, back 18.7. Bound by HBM, to 4 bits also by what a warp issues. By rows 39 and 35 (a
// division per step of 256 values), rows that do not begin on 16-byte boundaries value by value: 11008 x 4100 44 and 129.
#include "internal.h"
#include "mx4.cuh"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;  // of 256 values a warp
constexpr int kMx4FewTokens = 8;
constexpr int64_t kMx4FewValues = 1 << 24, kMx4OneValues = 1 << 26;  // of the weight

// Rows as both kernels walk them: in steps of 256 values. A matrix of whole blocks in contiguous rows is one row.
struct Walk {
    int64_t rows, cols, steps, blocks;  // steps and blocks of a row
};
inline Walk make_walk(int64_t rows, int64_t cols, int64_t ld) {
    Walk w{rows, cols, 0, 0};
    if (rows == 1 || (cols % kMx4Block == 0 && ld == cols)) w = {1, rows * cols, 0, 0};
    w.blocks = mx4_blocks(w.cols);
    w.steps = (w.blocks + 7) / 8;
    return w;
}

// Up to eight values from p on as fp32 (zeros behind the last). whole: all eight, on a 16-byte boundary.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* p, int n, bool vec) {
    Raw<T> r;
    if (vec && n >= 8) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = ld_v4(reinterpret_cast<const char*>(p) + 16 * i);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : Elt<T>::from_f(0.f);
        memcpy(&r, e, sizeof(r));
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw<T>& r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) Elt<T>::unpack(r.v[i], f + i * Elt<T>::kVec);
}

// The largest magnitude of eight values as an fp32 bit pattern (16-bit patterns are ordered as their values are).
template <typename T>
__device__ __forceinline__ uint32_t largest8(const Raw<T>& r) {
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            m = max(max(m, max(r.v[i].x & 0x7fffffffu, r.v[i].y & 0x7fffffffu)), max(r.v[i].z & 0x7fffffffu, r.v[i].w & 0x7fffffffu));
        return m;
    } else {
        const uint32_t a = 0x7fff7fffu;
        uint32_t m = __vmaxu2(__vmaxu2(r.v[0].x & a, r.v[0].y & a), __vmaxu2(r.v[0].z & a, r.v[0].w & a));
        m = max(m >> 16, m & 0xffffu);
        const uint16_t h = (uint16_t)m;
        return __float_as_uint(Elt<T>::to_f(reinterpret_cast<const T&>(h)));
    }
}

// Eight values as eight codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t encode8(const float (&f)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

// A lane's eight values (of four lanes' block) as codes, and the block's scale.
template <typename T>
__device__ __forceinline__ uint32_t convert8(const Raw<T>& raw, uint32_t& b) {
    uint32_t m = largest8(raw);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // the exponent field less 2; a block that holds an infinity or a NaN (field 255) is NaN
    b = m >= 0x7f800000u ? 255u : (uint32_t)max(0, (int)(m >> 23) - 2);
    const float inv = __uint_as_float((254u - b) << 23);  // 2^(127 - b), b <= 252
    float f[8];
    widen8(raw, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= inv;
    const uint32_t c = encode8(f);
    return b == 255u ? 0u : c;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_quantize_flat_kernel(const T* X, int64_t eights, uint32_t* codes,
                                                                     uint8_t* scales) {
    constexpr int kUnroll = sizeof(T) == 2 ? 4 : 2;
    pdl_trigger();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * kThreads;
    const int lane = threadIdx.x & 31;
    // (a warp's first eight decides, so that its lanes stay together; eights is a multiple of 4)
    for (int64_t e0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; e0 - lane < eights; e0 += kUnroll * step) {
        Raw<T> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            raw[u] = Raw<T>{};
            if (e0 + u * step < eights) raw[u] = load8(X + (e0 + u * step) * 8, 8, true);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            uint32_t b;
            const uint32_t c = convert8(raw[u], b);
            if (e0 + u * step < eights) {
                codes[e0 + u * step] = c;
                if ((lane & 3) == 0) scales[(e0 + u * step) >> 2] = (uint8_t)b;
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const T* X, int64_t ldx, Walk w, bool vec, uint32_t* codes,
                                                                uint8_t* scales) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t items = w.rows * w.steps;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    for (int64_t i0 = first; i0 < items; i0 += kSteps * warps) {
        Raw<T> raw[kSteps];
        int64_t at[kSteps];  // the lane's eight values among all of them, in eights
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int64_t i = i0 + u * warps;
            at[u] = -1;
            if (i < items) {
                const int64_t row = w.rows == 1 ? 0 : i / w.steps, eight = (i - row * w.steps) * 32 + lane;
                if (eight < w.blocks * 4) {
                    const int64_t left = w.cols - eight * 8;
                    raw[u] = load8(X + row * ldx + eight * 8, (int)min64(left, 8), vec);
                    at[u] = row * w.blocks * 4 + eight;
                }
            }
            if (at[u] < 0) raw[u] = Raw<T>{};
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            uint32_t b;
            const uint32_t c = convert8(raw[u], b);
            if (at[u] >= 0) {
                codes[at[u]] = c;
                if ((lane & 3) == 0) scales[at[u] >> 2] = (uint8_t)b;
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint32_t* codes, const uint8_t* scales, Walk w, T* Y,
                                                                  int64_t ldy, bool vec) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t items = w.rows * w.steps;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    for (int64_t i0 = first; i0 < items; i0 += kSteps * warps) {
        uint32_t c[kSteps], b[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int64_t i = i0 + u * warps;
            c[u] = b[u] = 0;
            if (i < items) {
                const int64_t row = w.rows == 1 ? 0 : i / w.steps, eight = (i - row * w.steps) * 32 + lane;
                if (eight < w.blocks * 4) {
                    c[u] = codes[row * w.blocks * 4 + eight];
                    b[u] = scales[row * w.blocks + (eight >> 2)];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int64_t i = i0 + u * warps;
            if (i >= items) break;
            const int64_t row = w.rows == 1 ? 0 : i / w.steps, eight = (i - row * w.steps) * 32 + lane;
            const int n = (int)min64(w.cols - eight * 8, 8);
            if (n <= 0) continue;
            const float s = mx4::scale_f32(b[u]);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = mx4::value_f32(c[u] >> (4 * e), s);
            T* to = Y + row * ldy + eight * 8;
            if (vec && n == 8) {
#pragma unroll
                for (int e = 0; e < (int)sizeof(T) / 2; ++e)
                    reinterpret_cast<uint4*>(to)[e] = Elt<T>::pack(f + e * Elt<T>::kVec);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) to[e] = Elt<T>::from_f(f[e]);
            }
        }
    }
}

// kVals: of a lane and step, 16 bytes of Y.
template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_flat_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                       int64_t pieces, T* Y) {
    constexpr int kVals = Elt<T>::kVec, kUnroll = 4;
    using Code = typename std::conditional<kVals == 8, uint32_t, uint16_t>::type;
    pdl_trigger();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t p0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; p0 < pieces; p0 += kUnroll * step) {
        uint32_t c[kUnroll], b[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t p = p0 + u * step;
            c[u] = p < pieces ? reinterpret_cast<const Code*>(codes)[p] : 0;
            b[u] = p < pieces ? scales[p / (kMx4Block / kVals)] : 127;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t p = p0 + u * step;
            if (p >= pieces) break;
            uint4 v;
            if constexpr (kVals == 8) {
                uint32_t o[4];
                if (mx4::plain(b[u])) mx4::decode8<T>(c[u], mx4::factor2(b[u]), o);
                else mx4::decode8_any<T>(c[u], b[u], o);
                v = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                const float s = mx4::scale_f32(b[u]);
                v = make_uint4(__float_as_uint(mx4::value_f32(c[u], s)), __float_as_uint(mx4::value_f32(c[u] >> 4, s)),
                               __float_as_uint(mx4::value_f32(c[u] >> 8, s)), __float_as_uint(mx4::value_f32(c[u] >> 12, s)));
            }
            reinterpret_cast<uint4*>(Y)[p] = v;
        }
    }
}

// Rows, zeros behind the last column.
template <typename T>
__global__ void __launch_bounds__(kThreads) mx4_copy_kernel(const T* from, int64_t ldf, T* to, int64_t ldt, int64_t rows,
                                                            int64_t cols, int64_t cols_to) {
    pdl_trigger();
    pdl_wait();
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
        for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < cols_to; c += (int64_t)gridDim.x * kThreads)
            to[r * ldt + c] = c < cols ? from[r * ldf + c] : (T)0;
}

// fp32 as the sum of three bf16 parts, rounded towards zero but for the last: 8 bits each, all 24 of a number from 2^-110 on. Below,
// the last part ends at bf16's least number, 2^-133: off by 2^-134 at most (parts times a power of two of their own would need
// accumulators of their own, or a factor per token behind the product). part: columns of a part. Infinities and NaN are their first part, beside zeros.
__global__ void __launch_bounds__(kThreads) mx4_split_kernel(const float* from, int64_t ldf, uint16_t* to, int64_t rows,
                                                             int64_t cols, int64_t part) {
    pdl_trigger();
    pdl_wait();
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
        for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < part; c += (int64_t)gridDim.x * kThreads) {
            const float x = c < cols ? from[r * ldf + c] : 0.f;
            const bool finite = fabsf(x) <= 3.402823466e38f;
            const float a = finite ? __uint_as_float(__float_as_uint(x) & 0xffff0000u) : x;
            const float y = finite ? x - a : 0.f, b = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
            const float parts[3] = {a, b, y - b};
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const __nv_bfloat16 h = __float2bfloat16_rn(parts[i]);
                to[r * 3 * part + i * part + c] = reinterpret_cast<const uint16_t&>(h);
            }
        }
}

dim3 copy_grid(int64_t rows, int64_t cols) {
    return dim3((unsigned)min64((cols + kThreads - 1) / kThreads, 1024), (unsigned)min64(rows, 4096));
}
cudaError_t copy_rows(const void* from, int64_t ldf, void* to, int64_t ldt, int64_t rows, int64_t cols, int64_t cols_to,
                      int64_t es, cudaStream_t s) {
    count_launches(1);
    if (es == 4)
        return launch_pdl(mx4_copy_kernel<float>, copy_grid(rows, cols_to), dim3(kThreads), 0, s, static_cast<const float*>(from), ldf,
                          static_cast<float*>(to), ldt, rows, cols, cols_to);
    return launch_pdl(mx4_copy_kernel<uint16_t>, copy_grid(rows, cols_to), dim3(kThreads), 0, s,
                      static_cast<const uint16_t*>(from), ldf, static_cast<uint16_t*>(to), ldt, rows, cols, cols_to);
}

unsigned walk_grid(const Walk& w) {
    const int64_t items = w.rows * w.steps, per = (int64_t)(kThreads / 32) * kSteps;
    return (unsigned)max64(1, min64((items + per - 1) / per, (int64_t)device_props().sm_count * 8));
}

// CTAs of a flat kernel: eight an SM, fewer where its threads would have nothing.
unsigned flat_grid(int64_t pieces, int unroll) {
    const int64_t per = (int64_t)kThreads * unroll;
    return (unsigned)max64(1, min64((pieces + per - 1) / per, (int64_t)device_props().sm_count * 8));
}

template <typename T>
cudaError_t quantize(const void* X, int64_t ldx, int32_t rows, int32_t cols, uint8_t* codes, uint8_t* scales,
                     cudaStream_t s) {
    const Walk w = make_walk(rows, cols, ldx);
    const bool vec = reinterpret_cast<uintptr_t>(X) % 16 == 0 && (w.rows == 1 || ldx * (int64_t)sizeof(T) % 16 == 0);
    count_launches(1);
    if (w.rows == 1 && w.cols % kMx4Block == 0 && vec)
        return launch_pdl(mx4_quantize_flat_kernel<T>, dim3(flat_grid(w.cols / 8, sizeof(T) == 2 ? 4 : 2)), dim3(kThreads), 0, s,
                          static_cast<const T*>(X), w.cols / 8, reinterpret_cast<uint32_t*>(codes), scales);
    return launch_pdl(mx4_quantize_kernel<T>, dim3(walk_grid(w)), dim3(kThreads), 0, s, static_cast<const T*>(X), ldx, w,
                      vec, reinterpret_cast<uint32_t*>(codes), scales);
}

template <typename T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t cols, void* Y, int64_t ldy,
                       cudaStream_t s) {
    const Walk w = make_walk(rows, cols, ldy);
    const bool vec = reinterpret_cast<uintptr_t>(Y) % 16 == 0 && (w.rows == 1 || ldy * (int64_t)sizeof(T) % 16 == 0);
    count_launches(1);
    if (w.rows == 1 && w.cols % kMx4Block == 0 && vec)
        return launch_pdl(mx4_dequantize_flat_kernel<T>, dim3(flat_grid(w.cols / Elt<T>::kVec, 4)), dim3(kThreads), 0, s, codes, scales,
                          w.cols / Elt<T>::kVec, static_cast<T*>(Y));
    return launch_pdl(mx4_dequantize_kernel<T>, dim3(walk_grid(w)), dim3(kThreads), 0, s,
                      reinterpret_cast<const uint32_t*>(codes), scales, w, static_cast<T*>(Y), ldy, vec);
}

}  // namespace

cudaError_t launch_mx4_quantize(int dt, const void* X, int64_t ldx, int32_t rows, int32_t cols, uint8_t* codes,
                                uint8_t* scales, cudaStream_t s) {
    if (dt == kF32) return quantize<float>(X, ldx, rows, cols, codes, scales, s);
    if (dt == kF16) return quantize<__half>(X, ldx, rows, cols, codes, scales, s);
    return quantize<__nv_bfloat16>(X, ldx, rows, cols, codes, scales, s);
}

cudaError_t launch_mx4_dequantize(int dt, const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t cols,
                                  void* Y, int64_t ldy, cudaStream_t s) {
    if (dt == kF32) return dequantize<float>(codes, scales, rows, cols, Y, ldy, s);
    if (dt == kF16) return dequantize<__half>(codes, scales, rows, cols, Y, ldy, s);
    return dequantize<__nv_bfloat16>(codes, scales, rows, cols, Y, ldy, s);
}

// The kernels without tensor-core tiles, forward, us as these kernels / the tiles. 1 token: 4096 x 4096 6.3 / 8.5, fp16 5.1 /
// 7.4, 11008 x 4096 12.2 / 13.4, fp16 10.9 / 11.3, 8192 x 8192 16.3 / 14.9, fp16 13.6 / 12.7. 8: 4096 x 4096 8.6 / 8.6, fp16
// 6.8 / 7.5, 1536 x 384 3.8 / 4.8, but 6144 x 4096 13.6 / 10.0, fp16 10.0 / 8.7, 8192 x 8192 25.4 / 15.0. They take any rows.
// The number of values decides, which is right for weights about as wide as long. The tiles need features, of which each 256 are
// a pair's and at most four splits: 8 tokens of 1024 x 16384 8.8 / 13.4, and just above the limit 1024 x 32768 would be 14.7
// and is 22.0, 512 x 65536 25.8 and 38; 16384 x 1024 is 8.6 and would be 6.9.
static bool mx4_few(int dt, bool back, const Mx4Args& a) {
    if (back || dt == kF32 || a.tokens > kMx4FewTokens) return false;
    const int64_t values = (int64_t)a.rows * a.cols;
    return (a.tokens == 1 ? values < kMx4OneValues : values <= kMx4FewValues) || !mx4_tile_rows(a.X, a.ldx, a.cols, 2) ||
           !mx4_tile_rows(a.Y, a.ldy, a.rows, 2);
}

bool mx4_needs_copies(int dt, bool back, const Mx4Args& a) {
    if (a.rows == 0 || a.cols == 0 || mx4_few(dt, back, a)) return false;
    const int64_t in = back ? a.rows : a.cols, out = back ? a.cols : a.rows, es = (int64_t)dtype_size(dt);
    return dt == kF32 || !mx4_tile_rows(a.X, a.ldx, in, es) || !mx4_tile_rows(a.Y, a.ldy, out, es);
}

cudaError_t launch_mx4_product(int dt, bool back, const Mx4Args& a, void* workspace, cudaStream_t s) {
    const int64_t in = back ? a.rows : a.cols, out = back ? a.cols : a.rows, es = (int64_t)dtype_size(dt);
    if (in == 0)  // nothing to sum
        return cudaMemset2DAsync(a.Y, (size_t)(a.ldy * es), 0, (size_t)(out * es), (size_t)a.tokens, s);
    if (mx4_few(dt, back, a)) return a.tokens == 1 ? launch_mx4_vec(dt, a, s) : launch_mx4_rows(dt, a, s);
    Mx4Args t = a;
    cudaError_t e = cudaSuccess;
    char* ws = static_cast<char*>(workspace);
    if (dt == kF32) {
        const int64_t part = mx4_split_cols(in) / 3;
        t.X = ws;
        t.ldx = 3 * part;
        count_launches(1);
        e = launch_pdl(mx4_split_kernel, copy_grid(a.tokens, part), dim3(kThreads), 0, s, static_cast<const float*>(a.X), a.ldx,
                       reinterpret_cast<uint16_t*>(ws), (int64_t)a.tokens, in, part);
        ws += mx4_x_bytes(a.tokens, in, es);
    } else if (!mx4_tile_rows(a.X, a.ldx, in, es)) {
        t.X = ws;
        t.ldx = (in + 7) / 8 * 8;
        e = copy_rows(a.X, a.ldx, ws, t.ldx, a.tokens, in, t.ldx, es, s);
        ws += mx4_x_bytes(a.tokens, in, es);
    }
    const bool own = mx4_tile_rows(a.Y, a.ldy, out, es);
    if (!own) {
        t.Y = ws;
        t.ldy = (out * es + 15) / 16 * 16 / es;
    }
    if (e == cudaSuccess) e = back ? launch_mx4_backward(dt, t, s) : launch_mx4_forward(dt, t, s);
    if (e == cudaSuccess && !own) e = copy_rows(t.Y, t.ldy, a.Y, a.ldy, a.tokens, out, out, es, s);
    return e;
}

}  // namespace spops
