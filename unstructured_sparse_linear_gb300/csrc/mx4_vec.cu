// X W^T for a microscaled 4-bit weight and one token (fp16 / bf16, any alignment of X and Y).
//
// mx4_vec_kernel: a warp's lanes share a row of W (or 32 / L of them, rows of few blocks): a lane loads 16 bytes, the
// values of one block, so a warp reads 512 bytes in a row, and four such loads are under way, the next row's among them.
// The codes become fp16 numbers by conversion and meet X as fp16 numbers in fused products with fp32 sums (6 cycles of a
// scheduler for two values and a token; bringing W to X's type first took 9), one sum per block, which is then multiplied with
// the block's scale. bf16 X is staged as fp16 numbers times a power of two for each 32 of them, which is exact where none but
// zeros lies below 2^-31 of the largest. A block for which it is not, or whose scale is uncommon, is multiplied value by value or
// scaled in 64 bits, found by one test behind its products. Sums are added over the lanes in one order. Bound by what a warp
// issues (45 instructions a word of codes; the schedulers issue in 64 to 70 % of the cycles, the integer pipe is at 53 to 56 %), and
// the call and the first load. 4096 x 4096: 6.3 us, fp16 5.1 (8.5 with the kernel for eight tokens, fp16 6.6), 11008 x 4096
// 12.2, fp16 10.8 (tcgen05 tiles 13.5 and 11.3).
#include <type_traits>

#include "internal.h"
#include "mx4.cuh"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAhead = 4;     // blocks of a lane under way
constexpr int kPitch = 80;    // bytes between blocks of X: 8 lanes' 16-byte reads meet no bank conflict
constexpr int kStaged = 512;  // blocks staged at a time

struct VecArgs {
    Mx4Args a;
    int64_t blocks;
    int32_t lanes, vec, rounds;  // lanes of a row; X's rows begin on 16-byte boundaries; rows that a warp's lanes take in turn
};

__device__ __forceinline__ void fma2(uint32_t w, uint32_t x, float& lo, float& hi) {
    asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %2;\n\tmov.b32 {c, d}, %3;\n\t"
        "fma.rn.f32.f16 %0, a, c, %0;\n\tfma.rn.f32.f16 %1, b, d, %1;\n\t}"
        : "+f"(lo), "+f"(hi)
        : "r"(w), "r"(x));
}

// Whether the values of a block with this scale are their codes times it in X's type too (or NaN): neither rounded nor
// infinite there.
template <typename T>
__device__ __forceinline__ bool exact_in(uint32_t b) {
    return std::is_same<T, __half>::value ? b - 104u <= 36u || b == 255u : b <= 252u || b == 255u;
}

// acc with a block's products, where its scale times X's power of two e is no normal number in fp32 or its values are not their
// codes times the scale. sum: the codes' products with X as staged. (A call: it would crowd the loop.)
template <typename T>
__device__ __noinline__ float add_uncommon(float acc, float sum, float e, const T* x, int64_t left, uint4 codes, uint32_t b) {
    const bool zeros = (codes.x | codes.y | codes.z | codes.w) == 0 && b != 255;
    if (e != 0.f && zeros) return acc + sum;  // (zeros, or NaN)
    const float scale = mx4::scale_f32(b);
    if (e != 0.f && exact_in<T>(b)) return (float)(acc + (double)sum * scale * e);
    float y = 0.f;  // value by value, as X's type has them, and X as it was given
#pragma unroll 1
    for (int k = 0; k < kMx4Block && k < left; ++k) {
        const uint32_t w = k < 8 ? codes.x : k < 16 ? codes.y : k < 24 ? codes.z : codes.w;
        y = fmaf(Elt<T>::to_f(Elt<T>::from_f(mx4::value_f32(w >> (4 * (k & 7)), scale))), Elt<T>::to_f(x[k]), y);
    }
    return acc + y;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) mx4_vec_kernel(const VecArgs g) {
    constexpr bool kF16 = std::is_same<T, __half>::value;
    __shared__ __align__(16) uint8_t xs[kStaged * kPitch];
    __shared__ float xe[kStaged];  // bf16: what X was divided by
    const int tid = threadIdx.x, lane = tid & 31, L = g.lanes, sub = lane & (L - 1);
    const int64_t rows_cta = (int64_t)kWarps * (32 / L);  // of a round
    const int64_t row0 = (int64_t)blockIdx.x * g.rounds * rows_cta + (int64_t)(tid >> 5) * (32 / L) + lane / L;
    const uint32_t xbase = smem_u32(xs);
    const T* X = static_cast<const T*>(g.a.X);
    T* Y = static_cast<T*>(g.a.Y);
    pdl_trigger();
    pdl_wait();
    float acc = 0.f;
    for (int64_t s0 = 0; s0 < g.blocks; s0 += kStaged) {  // (several: one round)
        const int n_blocks = (int)min64(kStaged, g.blocks - s0), steps = (n_blocks + L - 1) / L;
        uint4 w[kAhead];
        uint32_t b[kAhead];
        int64_t ask_row = row0;
        int ask_blk = sub, ask_round = 0;
        auto ask = [&](int u) {
            w[u] = make_uint4(0, 0, 0, 0);
            b[u] = 127;
            if (ask_round < g.rounds && ask_row < g.a.rows && ask_blk < n_blocks) {
                const int64_t at = ask_row * g.blocks + s0 + ask_blk;
                w[u] = ld_v4(g.a.codes + at * 16);
                b[u] = g.a.scales[at];
            }
            ask_blk += L;
            if (ask_blk >= steps * L) {
                ask_blk = sub;
                ask_row += rows_cta;
                ++ask_round;
            }
        };
#pragma unroll
        for (int u = 0; u < kAhead; ++u) ask(u);
        if (s0 > 0) __syncthreads();  // the segment before has been read
        for (int i0 = 0; i0 < n_blocks * 4; i0 += kThreads) {
            const int c = i0 + tid;  // 16 bytes of X
            const int64_t k = s0 * kMx4Block + c * 8;
            const int valid = c < n_blocks * 4 ? (int)max64(0, min64(8, g.a.cols - k)) : 0;
            uint32_t v[4] = {0, 0, 0, 0};
            if (g.vec && valid == 8) {
                const uint4 q = ld_v4(X + k);
                v[0] = q.x;
                v[1] = q.y;
                v[2] = q.z;
                v[3] = q.w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < valid)
                        v[e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(X)[k + e] << (16 * (e & 1));
            }
            if constexpr (!kF16) {
                float f[8];
                Elt<T>::unpack(make_uint4(v[0], v[1], v[2], v[3]), f);
                uint32_t m = 0;  // the largest finite magnitude
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t bits = __float_as_uint(f[e]) & 0x7fffffffu;
                    m = max(m, bits < 0x7f800000u ? bits : 0u);
                }
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const int e14 = m ? max((int)(m >> 23), 31) : 141;  // the largest comes to 2^14 .. 2^15, small ones below
                const float down = __uint_as_float((uint32_t)(268 - e14) << 23);  // 2^(141 - e14)
                bool low = mx4::least8(make_uint4(v[0], v[1], v[2], v[3])) < (e14 - 31) << 7;  // (more than fp16 holds there)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __half2 h = __floats2half2_rn(f[2 * e] * down, f[2 * e + 1] * down);
                    v[e] = reinterpret_cast<const uint32_t&>(h);
                }
                float back = __uint_as_float((uint32_t)(e14 - 14) << 23);  // 2^(e14 - 141)
                if (__any_sync(0xffffffffu, low)) {
                    low |= __shfl_xor_sync(0xffffffffu, low, 1) != 0;
                    low |= __shfl_xor_sync(0xffffffffu, low, 2) != 0;
                    if (low) back = 0.f;
                }
                if ((c & 3) == 0 && c < n_blocks * 4) xe[c >> 2] = back;
            }
            if (c < n_blocks * 4)
                *reinterpret_cast<uint4*>(xs + (c >> 2) * kPitch + (c & 3) * 16) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        __syncthreads();
        int64_t row = row0;
        int blk = sub, step = 0;
        const int total = g.rounds * steps;
        for (int it = 0; it < total; it += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (it + u >= total) break;
                if (blk < n_blocks) {
                    const uint32_t c[4] = {w[u].x, w[u].y, w[u].z, w[u].w}, sc = b[u];
                    const uint32_t x = xbase + blk * kPitch;
                    const float e = kF16 ? 1.f : xe[blk], both = mx4::scale_f32(sc) * e;
                    float sum = 0.f, sum1 = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t p[4] = {mx4::pair_f16<0>(c[k]), mx4::pair_f16<1>(c[k]), mx4::pair_f16<2>(c[k]),
                                               mx4::pair_f16<3>(c[k])};
                        uint4 y;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                                     : "r"(x + k * 16));
                        fma2(p[0], y.x, sum, sum1);
                        fma2(p[1], y.y, sum, sum1);
                        fma2(p[2], y.z, sum, sum1);
                        fma2(p[3], y.w, sum, sum1);
                    }
                    sum += sum1;
                    if (exact_in<T>(sc) && both >= 0x1p-126f && both <= 3.402823466e38f) {
                        acc = fmaf(sum, both, acc);
                    } else {
                        const int64_t k = (s0 + blk) * kMx4Block;
                        acc = add_uncommon(acc, sum, e, X + k, g.a.cols - k, w[u], sc);
                    }
                }
                ask(u);
                blk += L;
                if (++step == steps) {  // the row's last block of this segment
                    if (s0 + n_blocks == g.blocks) {
                        float y = acc;
                        for (int o = L / 2; o > 0; o /= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
                        if (row < g.a.rows && sub == 0) Y[row] = Elt<T>::from_f(y);
                        acc = 0.f;
                    }
                    row += rows_cta;
                    blk = sub;
                    step = 0;
                }
            }
        }
    }
}

template <typename T>
cudaError_t run(const Mx4Args& a, cudaStream_t s) {
    VecArgs g;
    g.a = a;
    g.blocks = mx4_blocks(a.cols);
    g.vec = reinterpret_cast<uintptr_t>(a.X) % 16 == 0 && a.ldx % 8 == 0;
    g.lanes = 32;
    while (g.lanes > 4 && g.blocks <= g.lanes * 2) g.lanes /= 2;
    // Every CTA at once where the rows allow it, so that X is staged once and the last CTAs have as much to do as the first.
    const int64_t per = (int64_t)kWarps * (32 / g.lanes), ctas = ((int64_t)a.rows + per - 1) / per;
    const int64_t at_once = (int64_t)device_props().sm_count * 4;
    g.rounds = g.blocks > kStaged ? 1 : (int32_t)min64(1 << 20, (ctas + at_once - 1) / at_once);
    count_launches(1);
    return launch_pdl(mx4_vec_kernel<T>, dim3((unsigned)((ctas + g.rounds - 1) / g.rounds)), dim3(kThreads), 0, s, g);
}

}  // namespace

cudaError_t launch_mx4_vec(int dt, const Mx4Args& a, cudaStream_t s) {
    if (dt == kF16) return run<__half>(a, s);
    return run<__nv_bfloat16>(a, s);
}

}  // namespace spops
