// X W^T for a microscaled 4-bit weight and up to eight tokens (fp16 / bf16, any alignment of X and Y).
//
// mx4_rows_kernel: a warp has 16 features, the eight tokens and a share of the contraction, and multiplies on the warp-wide tensor
// instruction in fp16: the codes become fp16 numbers by conversion (exact, without their scale), a block of 32 is two
// products into sums of its own, which are then added times the block's scale in fp32. So decoding costs 8 conversions
// for 16 x 32 values, whatever X's type. bf16 X is staged as fp16 numbers times a power of two for each 32 of them, which is
// exact where none but zeros lies below 2^-31 of the largest (looking for that takes 0.5 us of the times below); other blocks of
// a token are multiplied value by value in fp32.
// The codes come by asynchronous copies into rings of the warp's own, X through registers, a phase of the contraction ahead. A
// CTA's warps have two groups of 16 features and share the contraction by four, a cluster's CTAs share it once more; partial
// sums are added in one order. Bound by the first loads and by the latency of 130 instructions a block (a third of them for
// staging X) that depend on each other, with 3.4 warps a scheduler: it issues in 43 % of the cycles, integer pipe 34 %.
// 8 tokens, 4096 x 4096: 8.6 us (tcgen05 tiles 8.6), fp16 6.8 (7.5); 11008 x 4096 22.7 (13.5).
#include <type_traits>

#include "internal.h"
#include "mx4.cuh"
#include "mx4.h"
#include "tc.cuh"

namespace spops {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRing = 3;  // phases of codes in a warp's ring
constexpr int kShare = 8;  // blocks of a warp and phase: 128 bytes of a row's codes
// A warp's share of a phase in shared memory: 16 rows of codes 144 bytes apart (four banks, so that the reads of a word of
// 8 rows x 4 lanes meet no conflict), then 16 rows of scales.
constexpr uint32_t kCodesRow = kShare * 16 + 16, kCodes = 16 * kCodesRow, kSlot = kCodes + 16 * kShare;

// A phase is kBlocks blocks of the contraction; X's rows are 64 bytes apart modulo 128, so that the fragments' reads meet no
// bank conflict.
constexpr int kTokens = 8, kWk = 4, kWf = kWarps / kWk, kBlocks = kWk * kShare;
constexpr uint32_t kRow = kBlocks * 64 + 64, kX = kTokens * kRow, kXe = kTokens * kBlocks * 4;
constexpr int kLoads = kTokens * kBlocks * 4 / kThreads;  // of 16 bytes of X a thread and phase
constexpr uint32_t kSmem = 2 * (kX + kXe) + kWarps * kRing * kSlot;
static_assert(kSmem >= kWarps * kTokens * 16 * 4, "the partial sums fit");
constexpr int kPerSm = 2;

struct RowsArgs {
    Mx4Args a;
    int64_t blocks;
    int32_t phases, vec, scales4;  // scales4: whole aligned words of scales
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// A scale with which a block's sums can be multiplied as they are: its values are their codes times it in X's type too
// (fp16), and times X's own power of two, 2^-60 to 2^113, it is a normal number (bf16).
template <typename T>
__device__ __forceinline__ bool simple(uint32_t b) {
    return std::is_same<T, __half>::value ? b - 104u <= 36u : b - 61u <= 80u;
}

// The other scales: a word's values in X's type as fp16 numbers, to be multiplied with rare_factor. fp16: the values
// themselves and 1 (NaN for a scale that is NaN); bf16: the codes, infinite where the value is, and the scale.
template <typename T>
__device__ __noinline__ uint4 decode_rare(uint32_t w, uint32_t b) {
    const float s = mx4::scale_f32(b);
    constexpr bool f16 = std::is_same<T, __half>::value;
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float v = mx4::value_f32(w >> (8 * i + 4 * e), 1.f), x = Elt<T>::to_f(Elt<T>::from_f(v * s));
            y[e] = (f16 && b != 255) || (!f16 && isinf(x)) ? x : v;
        }
        r[i] = Elt<__half>::p2(y[0], y[1]);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
template <typename T>
__device__ __forceinline__ float rare_factor(uint32_t b) {
    return std::is_same<T, __half>::value && b != 255 ? 1.f : mx4::scale_f32(b);
}

// A block's products with n values of a token, added to two features' sums: value by value, as X's type has them. c0, c1: the
// features' codes in shared memory.
template <typename T>
__device__ __noinline__ float2 add_values(const T* x, int n, uint32_t c0, uint32_t c1, uint32_t b0, uint32_t b1, float2 acc) {
    const float s0 = mx4::scale_f32(b0), s1 = mx4::scale_f32(b1);
    uint32_t w0 = 0, w1 = 0;
    for (int i = 0; i < n; ++i, w0 >>= 4, w1 >>= 4) {
        if (i % 8 == 0) {
            w0 = lds_u32(c0 + i / 2);
            w1 = lds_u32(c1 + i / 2);
        }
        const float v = Elt<T>::to_f(x[i]);
        acc.x = fmaf(Elt<T>::to_f(Elt<T>::from_f(mx4::value_f32(w0, s0))), v, acc.x);
        acc.y = fmaf(Elt<T>::to_f(Elt<T>::from_f(mx4::value_f32(w1, s1))), v, acc.y);
    }
    return acc;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm) mx4_rows_kernel(const RowsArgs g) {
    constexpr bool kF16 = std::is_same<T, __half>::value;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const uint32_t sbase = smem_u32(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = lane >> 2, t = lane & 3;
    const int C = (int)cluster_size(), crank = (int)cluster_rank();
    const int wi = warp % kWf, wj = warp / kWf;
    const int64_t f0 = (int64_t)(blockIdx.x / C) * kWf * 16;  // the CTA's features
    const int tokens = g.a.tokens;
    const int p0 = (int)((int64_t)g.phases * crank / C), phases = (int)((int64_t)g.phases * (crank + 1) / C) - p0;
    const uint32_t xe_at = sbase + 2 * kX;
    const uint32_t ring = sbase + 2 * (kX + kXe) + warp * (kRing * kSlot);
    pdl_trigger();
    pdl_wait();

    // A lane's copies of a phase: 16 bytes of codes of rows lane / 8 + 4 j, four bytes of scales of row lane / 2. Rows behind
    // the last are the last again (their sums are not written).
    const int64_t row0 = f0 + wi * 16, last = g.a.rows - 1;
    const int64_t share0 = (int64_t)p0 * kBlocks + wj * kShare;  // the warp's first block
    const uint8_t* codes[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        codes[j] = g.a.codes + (min64(row0 + (lane >> 3) + 4 * j, last) * g.blocks + share0 + (lane & 7)) * 16;
    const uint8_t* scales = g.a.scales + min64(row0 + (lane >> 1), last) * g.blocks + share0 + 4 * (lane & 1);
    const uint32_t codes_to = ring + (lane >> 3) * kCodesRow + (lane & 7) * 16, scales_to = ring + kCodes + lane * 4;
    int load_slot = 0;
    int64_t load_left = g.blocks - share0;  // blocks from the phase's first on
    auto load_codes = [&](int p) {
        if (p < phases) {
            const uint32_t slot = load_slot * kSlot;
            const uint32_t there = (lane & 7) < load_left ? 16 : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                tc::cp_async16(codes_to + slot + 4 * j * kCodesRow, there ? codes[j] : g.a.codes, there);
                codes[j] += kBlocks * 16;
            }
            if (g.scales4) {
                const uint32_t in = 4 * (lane & 1) < load_left ? 4 : 0;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(scales_to + slot),
                             "l"(in ? scales : g.a.scales), "r"(in)
                             : "memory");
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t b = 4 * (lane & 1) + e < load_left ? scales[e] : 0;
                    asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales_to + slot + e), "r"(b) : "memory");
                }
            }
            scales += kBlocks;
            load_left -= kBlocks;
            load_slot = load_slot + 1 == kRing ? 0 : load_slot + 1;
        }
        tc::cp_async_commit();
    };

    // X: 16 bytes a load, four lanes a block
    const T* X = static_cast<const T*>(g.a.X);
    uint4 xr[kLoads];
    auto load_x = [&](int p) {
        if (p >= phases) return;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int i = u * kThreads + tid, r = i / (kBlocks * 4), c = i % (kBlocks * 4);
            const int64_t k = ((int64_t)(p0 + p) * kBlocks * 4 + c) * 8;
            const int n = r < tokens ? (int)max64(0, min64(8, g.a.cols - k)) : 0;  // values there are
            xr[u] = make_uint4(0, 0, 0, 0);
            if (g.vec && n == 8) {
                xr[u] = ld_v4(X + r * g.a.ldx + k);
            } else if (n > 0) {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) w[e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(X)[r * g.a.ldx + k + e] << (16 * (e & 1));
                xr[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    bool unheld = false;  // bf16: fp16 does not hold a block of this thread's; it is staged as zeros, its power of two as 0
    auto store_x = [&](int p) {
        unheld = false;
        if (p >= phases) return;
        const uint32_t to = sbase + (p & 1) * kX, te = xe_at + (p & 1) * kXe;
        // eight bits of a number below 2^-31 of its block's largest are more than fp16 holds there (and a block of tiny numbers'
        // power of two would be too small for `simple`)
        bool low = false;
        int limit[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int i = u * kThreads + tid, r = i / (kBlocks * 4), c = i % (kBlocks * 4);
            uint4 v = xr[u];
            if constexpr (!kF16) {
                float f[8];
                Elt<T>::unpack(v, f);
                uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                m = max(m >> 16, m & 0xffffu);
                if (m >= 0x7f80u) {  // the largest finite magnitude
                    m = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t bits = __float_as_uint(f[e]) >> 16 & 0x7fffu;
                        m = max(m, bits < 0x7f80u ? bits : 0u);
                    }
                }
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t e14 = max(m >> 7, 31u);                     // the largest comes to 2^14 .. 2^15, tiny ones below
                const float down = __uint_as_float((268u - e14) << 23);  // 2^(141 - e14)
                limit[u] = e14 < 81u ? 0x7f80 : ((int)e14 - 31) << 7;
                low |= mx4::least8(v) < limit[u];
                v = make_uint4(Elt<__half>::p2(f[0] * down, f[1] * down), Elt<__half>::p2(f[2] * down, f[3] * down),
                               Elt<__half>::p2(f[4] * down, f[5] * down), Elt<__half>::p2(f[6] * down, f[7] * down));
                if ((c & 3) == 0)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(te + ((c >> 2) * kTokens + r) * 4), "r"((e14 - 14) << 23)
                                 : "memory");
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + r * kRow + c * 16), "r"(v.x), "r"(v.y),
                         "r"(v.z), "r"(v.w)
                         : "memory");
        }
        if constexpr (!kF16) {
            if (!__any_sync(0xffffffffu, low)) return;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int i = u * kThreads + tid, r = i / (kBlocks * 4), c = i % (kBlocks * 4);
                low = mx4::least8(xr[u]) < limit[u];
                low |= __shfl_xor_sync(0xffffffffu, low, 1) != 0;
                low |= __shfl_xor_sync(0xffffffffu, low, 2) != 0;
                if (low) {
                    unheld = true;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to + r * kRow + c * 16), "r"(0u) : "memory");
                    if ((c & 3) == 0)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(te + ((c >> 2) * kTokens + r) * 4), "r"(0u) : "memory");
                }
            }
        }
    };

    load_x(0);
#pragma unroll
    for (int p = 0; p < kRing - 1; ++p) load_codes(p);
    store_x(0);
    load_x(1);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};

    int slot = 0;
    for (int p = 0; p < phases; ++p) {
        tc::cp_async_wait<kRing - 2>();
        const bool any_unheld = !kF16 && __syncthreads_or(unheld);
        if (kF16) __syncthreads();
        load_codes(p + kRing - 1);
        store_x(p + 1);
        load_x(p + 2);
        const uint32_t x0 = sbase + (p & 1) * kX + q * kRow + wj * kShare * 64 + t * 16;
        const uint32_t e0 = xe_at + (p & 1) * kXe + (wj * kShare * kTokens + 2 * t) * 4;
        const uint32_t c0 = ring + slot * kSlot + q * kCodesRow + t * 4, s0 = ring + slot * kSlot + kCodes + q * kShare;
        const int now = slot;
        slot = slot + 1 == kRing ? 0 : slot + 1;
#pragma unroll 2
        for (int b = 0; b < kShare; ++b) {
            const uint32_t w0 = lds_u32(c0 + b * 16), w1 = lds_u32(c0 + 8 * kCodesRow + b * 16);
            const uint32_t b0 = lds_u8(s0 + b), b1 = lds_u8(s0 + 8 * kShare + b);
            uint32_t a[4], c[4];
            float m0, m1;
            const bool easy = __all_sync(0xffffffffu, (simple<T>(b0) || (b0 != 255 && w0 == 0)) && (simple<T>(b1) || (b1 != 255 && w1 == 0)));
            if (easy) {
                a[0] = mx4::pair_f16<0>(w0);
                a[1] = mx4::pair_f16<1>(w0);
                a[2] = mx4::pair_f16<2>(w0);
                a[3] = mx4::pair_f16<3>(w0);
                c[0] = mx4::pair_f16<0>(w1);
                c[1] = mx4::pair_f16<1>(w1);
                c[2] = mx4::pair_f16<2>(w1);
                c[3] = mx4::pair_f16<3>(w1);
                m0 = simple<T>(b0) ? __uint_as_float(b0 << 23) : 1.f;  // (else the row's block is zeros)
                m1 = simple<T>(b1) ? __uint_as_float(b1 << 23) : 1.f;
            } else {
                const uint4 r0 = decode_rare<T>(w0, b0), r1 = decode_rare<T>(w1, b1);
                m0 = rare_factor<T>(b0);
                m1 = rare_factor<T>(b1);
                a[0] = r0.x, a[1] = r0.y, a[2] = r0.z, a[3] = r0.w;
                c[0] = r1.x, c[1] = r1.y, c[2] = r1.z, c[3] = r1.w;
            }
            const uint4 x = lds_v4(x0 + b * 64);
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            float d[4];
            mma_f16(d, a[0], c[0], a[1], c[1], x.x, x.y, zero);
            mma_f16(d, a[2], c[2], a[3], c[3], x.z, x.w, d);
            if constexpr (kF16) {
                acc[0] = fmaf(d[0], m0, acc[0]);
                acc[1] = fmaf(d[1], m0, acc[1]);
                acc[2] = fmaf(d[2], m1, acc[2]);
                acc[3] = fmaf(d[3], m1, acc[3]);
            } else {
                float ea, eb;
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ea), "=f"(eb) : "r"(e0 + b * kTokens * 4));
                if (easy) {
                    acc[0] = fmaf(d[0], m0 * ea, acc[0]);
                    acc[1] = fmaf(d[1], m0 * eb, acc[1]);
                    acc[2] = fmaf(d[2], m1 * ea, acc[2]);
                    acc[3] = fmaf(d[3], m1 * eb, acc[3]);
                } else {
                    // (whose product may leave fp32's range where the sum does not)
                    if (ea != 0.f) {  // (an infinite value's product with the zeros of a block that is not held)
                        acc[0] = (float)(acc[0] + (double)d[0] * m0 * ea);
                        acc[2] = (float)(acc[2] + (double)d[2] * m1 * ea);
                    }
                    if (eb != 0.f) {
                        acc[1] = (float)(acc[1] + (double)d[1] * m0 * eb);
                        acc[3] = (float)(acc[3] + (double)d[3] * m1 * eb);
                    }
                }
            }
        }
        if (any_unheld)
            for (int b = 0; b < kShare; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (lds_u32(e0 + (b * kTokens + e) * 4) == 0) {
                        const int64_t k = ((int64_t)(p0 + p) * kBlocks + wj * kShare + b) * kMx4Block;
                        const uint32_t c = ring + (uint32_t)now * kSlot + q * kCodesRow + b * 16;
                        const float2 y = add_values(X + (2 * t + e) * g.a.ldx + k, (int)min64(kMx4Block, g.a.cols - k), c, c + 8 * kCodesRow,
                                                    lds_u8(s0 + b), lds_u8(s0 + 8 * kShare + b), make_float2(acc[e], acc[2 + e]));
                        acc[e] = y.x;
                        acc[2 + e] = y.y;
                    }
    }
    tc::cp_async_wait<0>();
    __syncthreads();
    // partial sums: [warp][token][16 features]
    float* sums = reinterpret_cast<float*>(smem_raw);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        sums[(warp * kTokens + 2 * t + (e & 1)) * 16 + q + 8 * (e >> 1)] = acc[e];
    __syncthreads();
    const int items = kWf * tokens * 16;  // (features fastest)
    T* Y = static_cast<T*>(g.a.Y);
    for (int i = tid; i < items; i += kThreads) {
        const int f = i % 16, w = i / 16 % kWf, token = i / 16 / kWf;
        float y = 0.f;
        for (int j = 0; j < kWk; ++j) y += sums[((j * kWf + w) * kTokens + token) * 16 + f];
        if (C > 1) sums[(w * kTokens + token) * 16 + f] = y;  // (this thread's own)
        else if (f0 + w * 16 + f < g.a.rows) Y[token * g.a.ldy + f0 + w * 16 + f] = Elt<T>::from_f(y);
    }
    if (C > 1) {
        cluster_sync();
        const int n = (items + C - 1) / C;
        for (int i = crank * n + tid; i < min(items, (crank + 1) * n); i += kThreads) {
            const int f = i % 16, w = i / 16 % kWf, token = i / 16 / kWf;
            float y = 0.f;
            for (int j = 0; j < C; ++j)
                y += __uint_as_float(ld_cluster_u32(cluster_map(sbase + (uint32_t)((w * kTokens + token) * 16 + f) * 4, j)));
            if (f0 + w * 16 + f < g.a.rows) Y[token * g.a.ldy + f0 + w * 16 + f] = Elt<T>::from_f(y);
        }
        cluster_sync();  // nobody reads this CTA's sums any more
    }
}

template <typename T>
cudaError_t run(const Mx4Args& a, cudaStream_t s) {
    static bool done[64];
    auto kern = mx4_rows_kernel<T>;
    const int d = device_props().device;
    if (d < 0 || d >= 64 || !done[d]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        if (d >= 0 && d < 64) done[d] = true;
    }
    RowsArgs g;
    g.a = a;
    g.blocks = mx4_blocks(a.cols);
    g.phases = (int32_t)((g.blocks + kBlocks - 1) / kBlocks);
    g.vec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx % 8 == 0;
    g.scales4 = g.blocks % 4 == 0 && reinterpret_cast<uintptr_t>(a.scales) % 4 == 0;
    const int64_t fx = ((int64_t)a.rows + 16 * kWf - 1) / (16 * kWf);
    // as many CTAs along the contraction as the SMs hold at once
    int c = 1;
    while (c < 8 && fx * (c + 1) <= (int64_t)device_props().sm_count * kPerSm && g.phases >= 2 * (c + 1)) ++c;
    if (fx * c > 0x7fffffffll) return cudaErrorInvalidValue;
    count_launches(1);
    return launch_pdl_cluster(kern, dim3((unsigned)(fx * c)), dim3(kThreads), kSmem, (unsigned)c, s, g);
}

}  // namespace

cudaError_t launch_mx4_rows(int dt, const Mx4Args& a, cudaStream_t s) {
    return dt == kF16 ? run<__half>(a, s) : run<__nv_bfloat16>(a, s);
}

}  // namespace spops
