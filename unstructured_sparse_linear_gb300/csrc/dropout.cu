// Dropout from a counter-based generator, without a stored mask: Y = base + keep * X * 65536 / (65536 - threshold).
//
// Value c of row r is kept where its 16-bit number is not below the threshold. The numbers are those of Philox4x32 with
// 7 rounds (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011, where 7 rounds are the
// fewest that pass all their tests): key = the seed, counter = (r * ceil(cols / 8) + c / 8, call), 128 bits a step,
// number c % 8 of them. So the mask depends on neither strides, types nor launch shape, and the backward pass forms it
// again from the same state.
//
// A step a thread: eight values. Sixteen bits a value make it one Philox (14 wide products) per eight; with 32 bits
// the generator and not HBM would bound the kernel. 4096 x 11008 bf16 with a base, 270 MB: 44 us (40.5 at the device's copy
// rate), without one 33.5. Rows that do not begin on 16-byte boundaries go value by value: 4096 x 11007 107 and 106.
#include "common.cuh"
#include "internal.h"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kThreads = 256;

struct Numbers {
    uint32_t w[4];
};
__device__ __forceinline__ Numbers philox7(uint64_t index, uint64_t call, uint64_t seed) {
    uint32_t x0 = (uint32_t)index, x1 = (uint32_t)(index >> 32), x2 = (uint32_t)call, x3 = (uint32_t)(call >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
        x0 = (uint32_t)(b >> 32) ^ x1 ^ k0;
        x1 = (uint32_t)b;
        x2 = (uint32_t)(a >> 32) ^ x3 ^ k1;
        x3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Numbers{{x0, x1, x2, x3}};
}

template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
};
// Up to eight values from p on, zeros behind the last. vec: on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* p, int n, bool vec) {
    Raw<T> r;
    if (vec && n >= 8) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = ld_v4(reinterpret_cast<const char*>(p) + 16 * i);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? Elt<T>::to_f(p[i]) : 0.f;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = Elt<T>::pack(f + i * Elt<T>::kVec);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw<T>& r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) Elt<T>::unpack(r.v[i], f + i * Elt<T>::kVec);
}

// groups: eights of a row. vec: every row of every operand begins on a 16-byte boundary. A thread has kSteps eights at a
// time, all loaded before the first is used.
template <typename T, bool kBase>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutArgs g, int64_t rows, int64_t cols, int64_t groups,
                                                           bool vec) {
    constexpr int kSteps = sizeof(T) == 2 ? 2 : 1;
    pdl_trigger();
    pdl_wait();
    const uint64_t seed = g.state ? g.state[0] : g.seed, call = g.state ? g.state[1] : g.call;
    const float factor = g.threshold < 65536u ? 65536.f / (float)(65536u - g.threshold) : 0.f;
    // kept where the number, in a word's upper half, is not below the threshold: compared in 32 bits, the lower half behind it
    const uint32_t below = g.threshold < 65536u ? g.threshold << 16 : 0u;
    const int64_t items = rows * groups, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < items; i0 += kSteps * step) {
        Raw<T> x[kSteps], b[kSteps];
        int64_t r[kSteps], c[kSteps];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int64_t i = i0 + u * step;
            if (u > 0 && i >= items) break;
            r[u] = rows == 1 ? 0 : i / groups;
            c[u] = (i - r[u] * groups) * 8;
            const int n = (int)min64(cols - c[u], 8);
            x[u] = load8(static_cast<const T*>(g.X) + r[u] * g.ldx + c[u], n, vec);
            if (kBase) b[u] = load8(static_cast<const T*>(g.base) + r[u] * g.ldb + c[u], n, vec);
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int64_t i = i0 + u * step;
            if (u > 0 && i >= items) break;
            const int n = (int)min64(cols - c[u], 8);
            const Numbers w = philox7((uint64_t)i, call, seed);
            float f[8], y[8];
            widen8(x[u], f);
            if (kBase) widen8(b[u], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t number = e & 1 ? w.w[e / 2] : w.w[e / 2] << 16;
                const float kept = number >= below ? f[e] * factor : 0.f;  // (a dropped infinity or NaN is gone)
                f[e] = kBase ? y[e] + kept : kept;
            }
            if (g.threshold == 65536u)
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = kBase ? y[e] : 0.f;
            T* to = static_cast<T*>(g.Y) + r[u] * g.ldy + c[u];
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

template <typename T>
cudaError_t run(const DropoutArgs& a, cudaStream_t s) {
    auto ok = [&](const void* p, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || ld * (int64_t)sizeof(T) % 16 == 0);
    };
    const bool vec = ok(a.X, a.ldx) && ok(a.Y, a.ldy) && (!a.base || ok(a.base, a.ldb));
    int64_t rows = a.rows, cols = a.cols;
    if (cols % 8 == 0 && a.ldx == cols && a.ldy == cols && (!a.base || a.ldb == cols)) {  // one long row
        cols *= rows;
        rows = 1;
    }
    const int64_t groups = (cols + 7) / 8, items = rows * groups;
    const unsigned grid = (unsigned)min64((items + kThreads - 1) / kThreads, (int64_t)device_props().sm_count * 8);
    count_launches(1);
    return a.base ? launch_pdl(dropout_kernel<T, true>, dim3(grid), dim3(kThreads), 0, s, a, rows, cols, groups, vec)
                  : launch_pdl(dropout_kernel<T, false>, dim3(grid), dim3(kThreads), 0, s, a, rows, cols, groups, vec);
}

}  // namespace

cudaError_t launch_dropout(int dt, const DropoutArgs& a, cudaStream_t s) {
    if (dt == kF32) return run<float>(a, s);
    if (dt == kF16) return run<__half>(a, s);
    return run<__nv_bfloat16>(a, s);
}

}  // namespace spops
