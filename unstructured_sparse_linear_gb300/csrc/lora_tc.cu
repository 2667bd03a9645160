// Low-rank adapter operators on the tcgen05 tensor cores (fp16 / bf16).
//
// lora_tile_kernel   P = U W1 and O = base + s P W2 in one launch, for tiles of up to 128 rows
//                    that share an adapter (the forward product and the input gradient);
// lora_wgrad_kernel  G = s P^T U over an adapter's tokens (the weights' gradients).
//
// Precision. P stays in 32 bits where it is kept (TMEM, shared memory, global). As an operand of the
// second product it is the sum of 16-bit parts whose products have fp32 sums (a single bf16 part would add an
// error as large as the output's own rounding). bf16: three parts, all 24 bits of P. fp16, whose range P = U W1
// leaves easily (small gradients, large activations): two; a row (for a weight gradient: a rank's column among a CTA's
// tokens) is first scaled by a power of two, and the second part is kept 2^11 times larger; both are taken back in
// fp32. So 22 bits of P take part, 16 of values of 2^-34 of the row's or column's largest, and whatever lies
// above 2^-50 of it.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "lora.h"
#include "tc.cuh"

namespace spops {
namespace {

constexpr int kKC = 64;                       // 16-bit elements per 128-byte swizzled row
constexpr uint32_t kUBytes = kLoraTile * 128;  // a 128 x 64 tile of U, base or O

// ------------------------------------------------------------------ PTX

// The L2 policy of a gradient's rows: dY is read twice, by two kernels, beside operands that are read or
// written once; where all of it leaves L2 first, more of dY is still there for the second read than under
// the usual order (4096 tokens, 4096 -> 11008, rank 16: 51.9 us, 59.2 without; 8192 92.3, 95.0; with 16384,
// whose 361 MB of dY L2 does not hold either way, 182 and 178).
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// A box of a 2-D tensor. kHint: with the L2 policy (the neutral one is not free: 8192 tokens forward,
// 2048 -> 8192, 62.7 us, 60.4 without).
template <bool kHint>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                            uint64_t policy) {
    if constexpr (kHint)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Four rows of a 2-D tensor (a map whose box is one row of 64 elements) into 4 x 128 bytes.
template <bool kHint>
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&y)[4], uint32_t bar,
                                            uint64_t policy) {
    if constexpr (kHint)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar), "l"(policy)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar)
            : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

// Arrive on the barrier at local address `bar` in CTA `rank` of the cluster; this CTA's shared memory is
// then as this thread (and, through a barrier before, its CTA) left it, for whoever waits there. (A
// release of global memory as well took 0.5 us each time: 1037 tokens 21.7 us, 20.9 so.)
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar, int rank) {
    cluster_release_smem();
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_map(bar, rank)) : "memory");
}

__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "n"(kMbarPollNs)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) { return __uint_as_float(ld_cluster_u32(addr)); }

// Waits of one CTA. After one has run out of time (2 s) every later one of the CTA gives up at
// once, so that a kernel whose copy never arrives ends; the roles then skip their work but keep
// their loops, which hold barriers.
struct Waits {
    volatile int* failed;
    int* err;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (*failed) return false;
        if (mbar_wait(bar, parity, err)) return true;
        *failed = 1;
        return false;
    }
    __device__ __forceinline__ bool cluster(uint32_t bar, uint32_t parity) const {
        if (*failed) return false;
        const uint64_t t0 = global_timer_ns();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_cluster(bar, parity)) return true;
            if ((it & 255u) == 0 && global_timer_ns() - t0 > kMbarTimeoutNs) {
                record_error(err, kDevErrMbarTimeout);
                *failed = 1;
                return false;
            }
        }
    }
};
constexpr uint64_t kDrainNs = 100000000ull;  // after a failed wait: for copies still in flight

// 2^x for the exponent field of a normal fp32 number.
__device__ __forceinline__ float exp2i(int x) { return __uint_as_float((uint32_t)(x + 127) << 23); }

// The power of two that brings m (the largest magnitude) to [2^14, 2^15), and its inverse; 1
// for zero, infinite and NaN m. Both factors are normal numbers.
__device__ __forceinline__ void pow2_scale(float m, float& up, float& down) {
    up = down = 1.f;
    if (m > 0.f && m <= 3.402823466e38f) {
        const int e = max(-110, (int)((__float_as_uint(m) >> 23) & 255u) - 127);
        up = exp2i(14 - e);
        down = exp2i(e - 14);
    }
}

// The lo part of an fp16 pair is kept times 2^kLoShift: hi is at most 2^15 and drops less than one of its own
// units, 2^4, so lo stays below 2^15 as well, and what it cannot hold is below 2^-36 (2^-50 of the largest).
constexpr int kLoShift = 11;

// The parts that P is multiplied in.
template <typename T>
constexpr int kParts = std::is_same<T, __half>::value ? 2 : 3;

// Eight values as eight values of each part. Every part but the last is rounded towards zero and a 2^-25th of the
// value or less is added to what is left, so that all parts of a value have its sign and none is zero: an
// infinity in the other operand then meets parts of one sign. bf16: three parts of 8 bits, the value itself (but for
// the 2^-25th where the last part would be zero). fp16: of values that pow2_scale has scaled.
template <typename T>
__device__ __forceinline__ void split8(const float* x, uint4 (&part)[kParts<T>]) {
    uint32_t w[kParts<T>][4];
    float zero[2] = {0.f, 0.f};  // NaN once an infinity or a NaN has been multiplied in
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        zero[0] = fmaf(a, 0.f, zero[0]);
        zero[1] = fmaf(b, 0.f, zero[1]);
        if constexpr (std::is_same<T, __half>::value) {
            const __half2 h = __halves2half2(__float2half_rz(a), __float2half_rz(b));
            const float2 f = __half22float2(h);
            const float la = fmaf(a - f.x, (float)(1 << kLoShift), a * (float)(1.0 / (1 << (25 - kLoShift))));
            const float lb = fmaf(b - f.y, (float)(1 << kLoShift), b * (float)(1.0 / (1 << (25 - kLoShift))));
            const __half2 l = __floats2half2_rn(la, lb);
            w[0][i] = reinterpret_cast<const uint32_t&>(h);
            w[1][i] = reinterpret_cast<const uint32_t&>(l);
        } else {
            const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
            const float ra = fmaf(a, 0x1p-26f, a - __uint_as_float(ha)), rb = fmaf(b, 0x1p-26f, b - __uint_as_float(hb));
            const uint32_t ma = __float_as_uint(ra) & 0xffff0000u, mb = __float_as_uint(rb) & 0xffff0000u;
            const float la = fmaf(a, 0x1p-28f, ra - __uint_as_float(ma)), lb = fmaf(b, 0x1p-28f, rb - __uint_as_float(mb));
            w[0][i] = __byte_perm(ha, hb, 0x7632);
            w[1][i] = __byte_perm(ma, mb, 0x7632);
            w[2][i] = __byte_perm(__float_as_uint(la), __float_as_uint(lb), 0x7632);
        }
    }
    if (!(zero[0] + zero[1] == 0.f)) {  // infinities and NaN are their first part, beside zeros
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (fabsf(x[i]) <= 3.402823466e38f) continue;
            const uint32_t shift = 16 * (i & 1), keep = ~(0xffffu << shift);
            const T y = Elt<T>::from_f(x[i]);
            w[0][i / 2] = (w[0][i / 2] & keep) | (uint32_t) reinterpret_cast<const uint16_t&>(y) << shift;
#pragma unroll
            for (int p = 1; p < kParts<T>; ++p) w[p][i / 2] &= keep;
        }
    }
#pragma unroll
    for (int p = 0; p < kParts<T>; ++p) part[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// Stores to shared memory of a CTA of the cluster that complete on a barrier of that CTA (bar and
// addr both mapped there): the receiver waits for their bytes, the sender for nothing.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint4 v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_async_b32(uint32_t addr, uint32_t v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(v),
                 "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Place (in 16-byte units) of piece c of row r among the partial sums that a rank receives from
// one rank: `own` rows of RP / 4 pieces, piece-major, so that the 32 rows that a warp sends at one
// piece are whole 128-byte lines (a line per row and piece took 2.5 us for RP = 64), the rows
// permuted so that the reads of 256 / RP rows x RP / 8 piece pairs meet no bank conflict.
template <int RP>
__device__ __forceinline__ int p_place(int r, int c, int own) {
    constexpr int rw = 256 / RP;  // rows that a warp reads at once
    return c * own + (rw >= 8 ? r : r ^ (rw * ((c >> 1) & (8 / rw - 1))));
}

// The same among the sums that every rank receives of all rows: a warp reads 32 rows at one piece, and sends
// 256 / RP rows x RP / 8 pieces of one half.
__device__ __forceinline__ int sum_place(int r, int c) { return c * kLoraTile + (r ^ ((c >> 1) & 7)); }

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// N consecutive fp32 TMEM columns of the thread's lane, complete on return (the load and its wait
// are one statement, so that no use can be scheduled between them).
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float* v) {
    static_assert(N == 8 || N == 16 || N == 32, "shapes");
    uint32_t r[N];
    if constexpr (N == 8) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
            : "r"(taddr)
            : "memory");
    } else if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr)
            : "memory");
    } else if constexpr (N == 32) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
              "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
              "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
              "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(taddr)
            : "memory");
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

// N 32-bit TMEM columns of the thread's lane, complete on return.
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[N]) {
    static_assert(N == 4 || N == 8 || N == 16 || N == 32, "shapes");
    if constexpr (N == 4) {
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n\t"
            "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
            : "memory");
    } else if constexpr (N == 8) {
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
            "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
            : "memory");
    } else if constexpr (N == 16) {
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
            "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
            "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
    } else {
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n\t"
            "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
            "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
            "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
            "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
            : "memory");
    }
}

// Copies of B bytes (4 or 8) from global to shared memory, and the arrival on `bar` of a thread
// once its earlier ones are complete.
template <int B>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A 64-row x RP tile of rows [row0, row0 + 64) of the row-major rows x rank matrix W, by one warp,
// for ranks whose rows TMA cannot address (rank not a multiple of 8): zeros beyond the matrix,
// 64-column blocks of 8 KB in the 128-byte-swizzled layout. Even ranks with aligned rows are
// copied asynchronously (the caller's cp_async_arrive signals them), odd ones by plain loads.
template <typename T, int RP>
__device__ __forceinline__ void load_b_tile(uint32_t dst, const T* W, int64_t row0, int64_t rows, int rank) {
    const int lane = threadIdx.x & 31;
    const int m = (int)min64(64, rows - row0);
    const char* src = reinterpret_cast<const char*>(W + row0 * rank);
    constexpr int kChunks = RP / 8;
    auto at = [&](int row, int col) {  // of 16-bit elements
        return dst + (col >> 6) * 8192 + tc::sw128_off(row, (col >> 3) & 7) + (col & 7) * 2;
    };
    if (rank & 1) {
#pragma unroll 2
        for (int i = lane; i < 64 * kChunks; i += 32) {
            const int row = i / kChunks, c = i % kChunks;
            uint32_t w[4] = {0, 0, 0, 0};
            if (row < m) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(src) + (int64_t)row * rank;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c * 8 + e < rank) w[e >> 1] |= (uint32_t)p[c * 8 + e] << (16 * (e & 1));
            }
            st_shared_v4(at(row, c * 8), make_uint4(w[0], w[1], w[2], w[3]));
        }
        return;
    }
    // pieces of two or four elements; zeros first in the pieces that hold any
    const int full = rank / 8;  // whole 16-byte pieces of a row
    for (int i = lane; i < 64 * (kChunks - full); i += 32) {
        const int row = i / (kChunks - full), c = full + i % (kChunks - full);
        if (c * 8 >= rank || row >= m) st_shared_v4(at(row, c * 8), make_uint4(0, 0, 0, 0));
        else  // the tail of the piece that rank ends in
            for (int e = rank & 7; e < 8; e += 2)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(at(row, c * 8 + e)), "r"(0) : "memory");
    }
    if (m < 64)
        for (int i = lane; i < (64 - m) * full; i += 32)
            st_shared_v4(at(m + i / full, i % full * 8), make_uint4(0, 0, 0, 0));
    if (rank % 4 == 0) {
        const int n = rank / 4;
        for (int i = lane; i < m * n; i += 32) cp_async_small<8>(at(i / n, i % n * 4), src + (int64_t)i * 8);
    } else {
        const int n = rank / 2;
        for (int i = lane; i < m * n; i += 32) cp_async_small<4>(at(i / n, i % n * 2), src + (int64_t)i * 4);
    }
}

// ------------------------------------------------------------------ tile kernel

// Warps: 0 loads (TMA), 1 multiplies (one thread), 2 to 9 finish (two threads per row, each with
// half of the columns).
constexpr int kTileThreads = 320;
constexpr int kEpi = 256;
constexpr uint32_t kTileBars = 1024;  // barriers, flags and row factors, behind the stages and P

template <typename T, int RP>
struct TileCfg {
    static constexpr int kBlocks = (RP + 63) / 64;
    static constexpr uint32_t kW = RP > 64 ? 16384 : 8192;       // weight tile of a stage
    static constexpr uint32_t kStage = kUBytes + kW;
    // fp16: the parts of P, RP columns each in swizzled blocks of 128 rows x 64 columns; its fp32 (partial)
    // sums, 128 RP of them.
    static constexpr uint32_t kH = (2 * RP + 63) / 64 * kUBytes;
    static_assert(kH >= RP * 512u, "the partial sums fit");
    static constexpr int kPerSm = RP > 64 ? 1 : 2;
    static constexpr int kMinCluster = kLoraTile * RP / 8 / kEpi;
    // Dynamic shared memory per CTA: all of the SM's 228 KB but 1 KB that the system keeps per CTA.
    static constexpr uint32_t kBudget = (228 * 1024) / kPerSm - 1024;
    static constexpr int kStages = (int)((kBudget - kTileBars - kH) / kStage);
    static constexpr uint32_t kSmem = kStages * kStage + kH + kTileBars;
    // bf16: parts of P that are operands in TMEM, from column kPartsAt on, RP / 2 columns each. In shared memory three
    // would take a stage of the ring (8192 tokens, 2048 -> 8192, rank 64: 78.5 us, 60.8 so; rank 128 takes 188 either
    // way, for its 24 products per chunk: with two parts 148). For rank 64 the first one is left in shared memory: two
    // CTAs share the SM's TMEM.
    static constexpr int kInTmem = kParts<T> == 2 ? 0 : RP == 64 ? 2 : 3;
    static constexpr uint32_t kPartsAt = RP > 64 ? 256 : 64;
    // P: columns 0 .. RP - 1; O: two buffers of 64 at 128 and 192
    static constexpr uint32_t kTmem = kInTmem && RP > 64 ? 512 : 256;
    static_assert(kPartsAt + kInTmem * RP / 2 <= (RP > 64 ? 512 : 128) && kPartsAt >= (RP > 64 ? 256 : RP), "TMEM columns");
};

// Row-strided operands come in boxes of 128, 32 or 8 consecutive rows, or four rows anywhere.
constexpr int kBoxes = 4;
constexpr int kBoxRows[kBoxes] = {128, 32, 8, 1};
struct TileMaps {
    CUtensorMap u[kBoxes], base[kBoxes], a, b, o;  // o: boxes of 32 rows
};

struct TileArgs {
    LoraPlanView v;
    const void* B;
    const float* scale;
    const void* base;
    void* O;
    float* P;
    int64_t ldb, ldo;
    int32_t K, N, rank;
    float scale_all;
    int hand;  // B tiles are copied by threads
    int* err;
};

// How lane i of the loading warp fetches rows 4 i .. 4 i + 3 of a tile: as (the first lane of) a
// box of 128, 32 or 8 consecutive tokens (mode 0, 1, 2), as four tokens anywhere (mode 3; rows past
// the tile repeat its last one), or not at all (mode -1: no such row, or another lane's box).
// A gather of four rows costs the copy engine about as much as a box: a whole tile of them took
// 1.2 us a chunk, three times a box of 128 rows.
struct RowSource {
    int mode, y[4];
};
__device__ __forceinline__ RowSource row_source(const LoraTile& t, const int32_t* order, int lane) {
    RowSource r;
    if (t.rows == kLoraTile && t.tok0 >= 0) {
        r.mode = lane == 0 ? 0 : -1;
        r.y[0] = t.tok0;
        r.y[1] = r.y[2] = r.y[3] = 0;
        return r;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) r.y[i] = order[t.pos0 + min(4 * lane + i, t.rows - 1)];
    const bool run4 = 4 * lane + 4 <= t.rows && r.y[3] - r.y[0] == 3;  // ascending, so consecutive
    const int next = __shfl_down_sync(0xffffffffu, r.y[0], 1);
    const unsigned runs = __ballot_sync(0xffffffffu, run4);
    const unsigned links = __ballot_sync(0xffffffffu, next == r.y[3] + 1);  // lane and lane + 1 (not lane 31)
    const int l8 = lane & ~7, l2 = lane & ~1;
    if (((runs >> l8) & 0xffu) == 0xffu && ((links >> l8) & 0x7fu) == 0x7fu) r.mode = lane == l8 ? 1 : -1;
    else if (((runs >> l2) & 3u) == 3u && ((links >> l2) & 1u)) r.mode = lane == l2 ? 2 : -1;
    else r.mode = 4 * lane < t.rows ? 3 : -1;
    return r;
}

// A cluster of C CTAs takes a tile: rank c multiplies a share of the K chunks into its TMEM; the
// fp32 partial P are sent through distributed shared memory to the rank that owns the row, which
// adds them in rank order and sends the sums (fp16: their two parts) to all; and rank c forms a share of
// the 64-column chunks of O. One ring of stages carries both phases, so the loads of base run
// ahead while P is being summed: a stage holds a 128 x 64 tile
// of U with a tile of W1, then a 128 x 64 tile of base, in which O is formed in place, with a tile
// of W2.
template <typename T, bool kBack, int RP>
__global__ void __launch_bounds__(kTileThreads, TileCfg<T, RP>::kPerSm)
lora_tile_kernel(const TileArgs g, const __grid_constant__ TileMaps maps) {
    using Cfg = TileCfg<T, RP>;
    constexpr int S = Cfg::kStages;
    constexpr bool kF16 = std::is_same<T, __half>::value;
    constexpr uint32_t kFmt = kF16 ? 0u : 1u;
    constexpr uint32_t kIdesc1 = tc::instr_desc_f16(kFmt, 0, kBack ? 1 : 0, 128, RP);
    constexpr uint32_t kIdesc2 = tc::instr_desc_f16(kFmt, 0, kBack ? 1 : 0, 128, 64);
    constexpr uint32_t kABytes = RP * 128, kBBytes = Cfg::kBlocks * 8192;
    // No static shared memory, so the dynamic part starts on the 1 KB boundary that the swizzled
    // tiles need (checked).
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    struct Shared {
        uint64_t full[S], empty[S], d1, h, parts, d2_full[2], d2_empty[2], pub, read, freed, drain;
        uint32_t tmem;
        volatile int failed;
        float down[kLoraTile];  // fp16: what a row's parts were scaled by, inverted
    };
    static_assert(sizeof(Shared) <= kTileBars, "barriers");
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw + S * Cfg::kStage + Cfg::kH);
    const uint32_t sbase = smem_u32(smem_raw);
    const uint32_t hbase = sbase + S * Cfg::kStage;
    if (sbase & 1023u) {  // the same on every CTA
        record_error(g.err, kDevErrSmemAlign);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cluster_size(), crank = (int)cluster_rank();
    const int cid = blockIdx.x / C, ncl = gridDim.x / C;
    if (warp == 2 && lane == 0) {
        for (int i = 0; i < kBoxes; ++i) {
            tma_prefetch_map(&maps.u[i]);
            tma_prefetch_map(&maps.base[i]);
        }
        tma_prefetch_map(&maps.a);
        tma_prefetch_map(&maps.b);
        tma_prefetch_map(&maps.o);
    }
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&sh.full[s]), g.hand ? 1 + 32 : 1);
            mbar_init(smem_u32(&sh.empty[s]), 4);  // four commits, or the four warps of a group
        }
        mbar_init(smem_u32(&sh.d1), 1);
        mbar_init(smem_u32(&sh.h), 1);
        mbar_init(smem_u32(&sh.parts), kEpi / 32);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.d2_full[i]), 1);
            mbar_init(smem_u32(&sh.d2_empty[i]), 4);
        }
        mbar_init(smem_u32(&sh.pub), 1);
        mbar_init(smem_u32(&sh.read), C);
        mbar_init(smem_u32(&sh.freed), C);
        mbar_init(smem_u32(&sh.drain), 1);
        fence_mbar_init();
        sh.failed = 0;
    }
    __syncthreads();
    if (C > 1) cluster_sync_relaxed();  // the other ranks' barriers are initialised
    // All before this line overlaps the kernel before this one, and touches no memory that it writes.
    pdl_wait();
    // Every cluster's first tile (the list has a slot per cluster; what lies behind its end is not used).
    const int ntiles = g.v.counts[kLoraCntTiles];
    const LoraTile tile0 = g.v.tiles[cid];
    uint32_t tmem = 0;
    if (warp > 0) {  // (the loads need none, and begin at once)
        // TMEM is allocated after the wait, so that no CTA holds it while one of the kernel before
        // wants it, and before the trigger for the same reason. The trigger also tells a dependent
        // kernel that all before this one is complete (the weight gradients' rely on that).
        if (warp == 1) {
            tc::tmem_alloc(smem_u32(&sh.tmem), Cfg::kTmem);
            pdl_trigger();
        }
        tc::fence_before_sync();
        named_barrier(2, kTileThreads - 32);
        tc::fence_after_sync();
        tmem = sh.tmem;
    }
    const Waits wait{&sh.failed, g.err};
    const int nkc = (g.K + kKC - 1) / kKC, nnc = g.O ? (g.N + kKC - 1) / kKC : 0;
    const int clog = 31 - __clz(C);  // C is a power of two; the chunk counts are below 2^26
    const int ka = (nkc * crank) >> clog, na = (nnc * crank) >> clog;
    const int nk = ((nkc * (crank + 1)) >> clog) - ka, nn = ((nnc * (crank + 1)) >> clog) - na;

    if (warp == 0) {
        // ---------------- loads
        const uint64_t policy = kBack ? evict_first_policy() : 0;
        uint32_t q = 0;
        bool ok = true;
        const int64_t brows = kBack ? g.K : g.N;
        for (int it = cid; it < ntiles && ok; it += ncl) {
            const LoraTile t = it == cid ? tile0 : g.v.tiles[it];
            const RowSource rows = row_source(t, g.v.order, lane);
            const uint32_t ubytes = (uint32_t)((t.rows + 3) / 4) * 512u;
            for (int j = 0; j < nk + nn; ++j, ++q) {
                const bool p1 = j < nk;
                const uint32_t s = q % S, st = sbase + s * Cfg::kStage, fb = smem_u32(&sh.full[s]);
                if (q >= S) ok = __all_sync(0xffffffffu, wait(smem_u32(&sh.empty[s]), (q / S - 1) & 1u));
                if (!ok) break;
                const bool from_rows = p1 || g.base;
                const bool b_tile = p1 ? kBack : !kBack;  // this phase's weights: a tile of B, else of A
                if (lane == 0) {
                    const uint32_t w = b_tile ? (g.hand ? 0u : kBBytes) : kABytes;
                    mbar_arrive_expect_tx(fb, (from_rows ? ubytes : 0u) + w);
                }
                __syncwarp();
                const int x = (p1 ? ka + j : na + j - nk) * kKC;
                if (from_rows) {
                    const CUtensorMap* m = p1 ? maps.u : maps.base;
                    if (rows.mode >= 0 && rows.mode < 3) tma_load_2d<kBack>(st + lane * 512, m + rows.mode, x, rows.y[0], fb, policy);
                    else if (rows.mode == 3) tma_gather4<kBack>(st + lane * 512, m + 3, x, rows.y, fb, policy);
                }
                if (lane == 0) {
                    if (!b_tile) {
                        tma_load_3d(st + kUBytes, &maps.a, x, 0, t.adapter, fb);
                    } else if (!g.hand) {
#pragma unroll
                        for (int b = 0; b < Cfg::kBlocks; ++b)
                            tma_load_3d(st + kUBytes + b * 8192, &maps.b, b * 64, x, t.adapter, fb);
                    }
                }
                if (g.hand) {
                    if (b_tile) {
                        load_b_tile<T, RP>(st + kUBytes, static_cast<const T*>(g.B) + t.adapter * brows * g.rank, x,
                                           brows, g.rank);
                        fence_proxy_async_smem();
                    }
                    cp_async_arrive(fb);
                }
            }
        }
        if (sh.failed) {  // let the copies in flight land before the shared memory is given up
            for (uint32_t i = q > S ? q - S : 0; i < q; ++i)
                mbar_wait_for(smem_u32(&sh.full[i % S]), (i / S) & 1u, nullptr, kDrainNs);
        }
    } else if (warp == 1) {
        // ---------------- multiplications
        if (lane == 0) {
            uint32_t q = 0, n2 = 0, tt = 0;
            bool ok = true;
            for (int it = cid; it < ntiles && ok; it += ncl, ++tt) {
                for (int j = 0; j < nk && ok; ++j, ++q) {
                    const uint32_t s = q % S, st = sbase + s * Cfg::kStage;
                    ok = wait(smem_u32(&sh.full[s]), (q / S) & 1u);
                    if (!ok) break;
                    if (g.hand) fence_proxy_async_smem();  // the copies of threads
                    tc::fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ad = tc::smem_desc_sw128(st + kk * 32, 16, 1024);
                        const uint64_t bd = kBack ? tc::smem_desc_sw128(st + kUBytes + kk * 2048, 8192, 1024)
                                                  : tc::smem_desc_sw128(st + kUBytes + kk * 32, 16, 1024);
                        tc::mma_f16(tmem, ad, bd, kIdesc1, (j > 0 || kk > 0) ? 1u : 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc::mma_commit(smem_u32(&sh.empty[s]));
                }
                if (!ok) break;
                tc::mma_commit(smem_u32(&sh.d1));
                // P's parts are here, and its columns read
                ok = kF16 ? wait.cluster(smem_u32(&sh.h), tt & 1u) : wait(smem_u32(&sh.parts), tt & 1u);
                if (!ok) break;
                fence_proxy_async_smem();  // the parts came from threads (fp16: of every rank)
                tc::fence_after_sync();
                for (int j = 0; j < nn; ++j, ++q, ++n2) {
                    const uint32_t s = q % S, st = sbase + s * Cfg::kStage, b = n2 & 1u;
                    ok = wait(smem_u32(&sh.full[s]), (q / S) & 1u);
                    if (ok && n2 >= 2) ok = wait(smem_u32(&sh.d2_empty[b]), (n2 / 2 - 1) & 1u);
                    if (!ok) break;
                    if (g.hand) fence_proxy_async_smem();
                    tc::fence_after_sync();
                    // fp16: the lo parts' products first; what they add up to is divided by 2^kLoShift as the first of hi's
                    // is added.
                    constexpr int kSteps = RP / 16;
#pragma unroll
                    for (int n = 0; n < kParts<T> * kSteps; ++n) {
                        const int i = kF16 ? (n + kSteps) % (2 * kSteps) : n, w = i % kSteps;
                        const uint32_t d = tmem + 128 + b * 64;
                        const uint64_t bd = kBack
                                                ? tc::smem_desc_sw128(st + kUBytes + w * 2048, 8192, 1024)
                                                : tc::smem_desc_sw128(st + kUBytes + (w / 4) * 8192 + (w % 4) * 32, 16, 1024);
                        const int in_tmem = i - (kParts<T> - Cfg::kInTmem) * kSteps;
                        if (in_tmem >= 0) {
                            tc::mma_f16_ts(d, tmem + Cfg::kPartsAt + in_tmem * 8, bd, kIdesc2, n > 0 ? 1u : 0u);
                            continue;
                        }
                        const uint64_t ad = tc::smem_desc_sw128(hbase + (i / 4) * 16384 + (i % 4) * 32, 16, 1024);
                        if (kF16 && n == kSteps) tc::mma_f16_scaled<kLoShift>(d, ad, bd, kIdesc2);
                        else tc::mma_f16(d, ad, bd, kIdesc2, n > 0 ? 1u : 0u);
                    }
                    tc::mma_commit(smem_u32(&sh.d2_full[b]));
                }
            }
            if (sh.failed) {
                tc::mma_commit(smem_u32(&sh.drain));
                mbar_wait_for(smem_u32(&sh.drain), 0, nullptr, kDrainNs);
            }
        }
        __syncwarp();
    } else {
        // ---------------- P, then O
        // While P is summed a row has two threads, each with half of its columns.
        const int quarter = warp & 3, grp = (warp - 2) >> 2, row = quarter * 32 + lane, et = tid - 64;
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const int own = kLoraTile >> clog;  // rows that this rank sums: [crank * own, ...)
        // Tokens without an adapter, O = base, P = 0: first, while the loads for the first sums are
        // under way (1037 tokens of 24 adapters: 20.7 us, and 21.2 with them last).
        const bool copy = g.O && (g.O != g.base);
        if (copy || g.P) {
            for (int64_t pos = (int64_t)g.v.off[g.v.n] + blockIdx.x; pos < g.v.tokens; pos += gridDim.x) {
                const int64_t t = g.v.order[pos];
                if (copy) {
                    const uint4* src = g.base ? reinterpret_cast<const uint4*>(static_cast<const T*>(g.base) + t * g.ldb)
                                              : nullptr;
                    uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(g.O) + t * g.ldo);
                    for (int i = et; i < g.N / 8; i += kEpi) to[i] = src ? src[i] : make_uint4(0, 0, 0, 0);
                }
                if (g.P)
                    for (int j = et; j < g.rank; j += kEpi) g.P[t * g.rank + j] = 0.f;
            }
        }
        uint32_t q = 0, n2 = 0, tt = 0;
        for (int it = cid; it < ntiles; it += ncl, ++tt) {
            const LoraTile t = it == cid ? tile0 : g.v.tiles[it];
            const int tok = g.v.order[t.pos0 + min(row, t.rows - 1)];
            const int tok_first = __shfl_sync(0xffffffffu, tok, 0);
            const bool run32 = __all_sync(0xffffffffu, row < t.rows && tok == tok_first + lane);
            const float s = g.scale_all * (g.scale ? g.scale[t.adapter] : 1.f);
            // what this thread sums: columns 8 c8 .. of row r (`sums` is the same for a whole warp)
            constexpr int kG = RP / 8;
            const bool sums = et < own * kG;
            const int rl = et / kG, c8 = et % kG, r = crank * own + rl;
            const int ptok = g.P && sums && r < t.rows ? g.v.order[t.pos0 + r] : -1;  // and the token of that row
            q += nk;
            {
                // Each rank sends its partial rows to the ranks that sum them, a slot per source.
                float p[RP / 2];
                wait(smem_u32(&sh.d1), tt & 1u);
                __syncwarp();  // (waits end lane by lane; what follows is for the whole warp)
                tc::fence_after_sync();
                if (nk > 0) {
                    constexpr int kLd = RP / 2 < 32 ? RP / 2 : 32;
#pragma unroll
                    for (int c = 0; c < RP / 2 / kLd; ++c)
                        tmem_load<kLd>(lane_addr + grp * (RP / 2) + c * kLd, p + c * kLd);
                } else {
#pragma unroll
                    for (int j = 0; j < RP / 2; ++j) p[j] = 0.f;
                }
                tc::fence_before_sync();
                // every rank is done with the last tile's parts of P, whose place the sums take
                if (tt > 0) wait.cluster(smem_u32(&sh.freed), (tt - 1) & 1u);
                __syncwarp();
                const int to = row >> (7 - clog);
                const uint32_t dst = cluster_map(hbase + crank * own * (RP * 4), to);
                const uint32_t bar = cluster_map(smem_u32(&sh.pub), to);
#pragma unroll
                for (int c = 0; c < RP / 8; ++c)
                    st_async_v4(dst + (uint32_t)p_place<RP>(row & (own - 1), grp * (RP / 8) + c, own) * 16,
                                make_uint4(__float_as_uint(p[4 * c]), __float_as_uint(p[4 * c + 1]),
                                           __float_as_uint(p[4 * c + 2]), __float_as_uint(p[4 * c + 3])),
                                bar);
            }
            if (et == 0) {  // what is to arrive here: every rank's sums of `own` rows, then all rows' parts
                mbar_arrive_expect_tx(smem_u32(&sh.pub), (uint32_t)kLoraTile * RP * 4);
                mbar_arrive_expect_tx(smem_u32(&sh.h), (uint32_t)kLoraTile * (RP * 4 + (kF16 ? 4 : 0)));
            }
            wait.cluster(smem_u32(&sh.pub), tt & 1u);
            __syncwarp();
            // Sums in rank order: eight columns of one row per thread (the cluster is large enough).
            float x[8];
            if (sums) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll 4
                for (int c = 0; c < C; ++c) {
                    const uint32_t from = hbase + c * own * (RP * 4);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 v = ld_shared_v4(from + (uint32_t)p_place<RP>(rl, 2 * c8 + h, own) * 16);
                        x[4 * h] += __uint_as_float(v.x);
                        x[4 * h + 1] += __uint_as_float(v.y);
                        x[4 * h + 2] += __uint_as_float(v.z);
                        x[4 * h + 3] += __uint_as_float(v.w);
                    }
                }
            }
            named_barrier(1, kEpi);
            if (et < C) mbar_arrive_remote(smem_u32(&sh.read), et);
            if (ptok >= 0) {
                float* to = g.P + (int64_t)ptok * g.rank + c8 * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c8 * 8 + e < g.rank) to[e] = x[e];
            }
            wait.cluster(smem_u32(&sh.read), tt & 1u);  // every rank has read its slots
            __syncwarp();
            // s P goes to every rank.
            if (sums) {
                float m = 0.f, up = 1.f, down = 1.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (columns beyond the rank are U times zeros: NaN where U holds an infinity)
                    x[e] = c8 * 8 + e < g.rank ? x[e] * s : 0.f;
                    const float y = fabsf(x[e]);
                    if (y <= 3.402823466e38f) m = fmaxf(m, y);  // (infinities leave the others their scale)
                }
                if (kF16) {  // the row's pieces lie in kG neighbouring lanes
#pragma unroll
                    for (int d = kG / 2; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                    pow2_scale(m, up, down);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= up;
                }
                // fp16: two parts; bf16: the values, which every rank takes apart itself (as many bytes as two parts)
                uint4 send[2];
                uint32_t to[2];
                if constexpr (kF16) {
                    split8<T>(x, send);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int at = c8 + p * kG;
                        to[p] = hbase + (at >> 3) * kUBytes + tc::sw128_off(r, at & 7);
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        send[p] = make_uint4(__float_as_uint(x[4 * p]), __float_as_uint(x[4 * p + 1]),
                                             __float_as_uint(x[4 * p + 2]), __float_as_uint(x[4 * p + 3]));
                        to[p] = hbase + (uint32_t)sum_place(r, 2 * c8 + p) * 16;
                    }
                }
                for (int c = 0; c < C; ++c) {
                    const uint32_t bar = cluster_map(smem_u32(&sh.h), c);
                    st_async_v4(cluster_map(to[0], c), send[0], bar);
                    st_async_v4(cluster_map(to[1], c), send[1], bar);
                    if (kF16 && c8 == 0)
                        st_async_b32(cluster_map(smem_u32(&sh.down[r]), c), __float_as_uint(down), bar);
                }
            }
            wait.cluster(smem_u32(&sh.h), tt & 1u);
            __syncwarp();
            const float down = kF16 ? sh.down[row] : 1.f;
            if constexpr (!kF16) {
                // Half of a row's columns per thread.
                constexpr int kInSmem = 3 - Cfg::kInTmem;  // (over the place of the values)
                float p[RP / 2];
#pragma unroll
                for (int i = 0; i < RP / 8; ++i) {
                    const uint4 v = ld_shared_v4(hbase + (uint32_t)sum_place(row, grp * (RP / 8) + i) * 16);
                    p[4 * i] = __uint_as_float(v.x);
                    p[4 * i + 1] = __uint_as_float(v.y);
                    p[4 * i + 2] = __uint_as_float(v.z);
                    p[4 * i + 3] = __uint_as_float(v.w);
                }
                if (kInSmem) named_barrier(1, kEpi);
                uint32_t words[3][RP / 4];
#pragma unroll
                for (int i = 0; i < RP / 16; ++i) {
                    uint4 part[3];
                    split8<T>(p + 8 * i, part);
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        const int at = grp * (RP / 16) + i + q * kG;
                        if (q < kInSmem) st_shared_v4(hbase + (at >> 3) * kUBytes + tc::sw128_off(row, at & 7), part[q]);
                        words[q][4 * i] = part[q].x;
                        words[q][4 * i + 1] = part[q].y;
                        words[q][4 * i + 2] = part[q].z;
                        words[q][4 * i + 3] = part[q].w;
                    }
                }
#pragma unroll
                for (int q = kInSmem; q < 3; ++q)
                    tmem_store<RP / 4>(lane_addr + Cfg::kPartsAt + (q - kInSmem) * (RP / 2) + grp * (RP / 4), words[q]);
                tc::fence_before_sync();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.parts));
            }

            // Chunks of O, in turns between the two groups of four warps (thread = row): the steps of
            // one chunk depend on each other, so two are under way at a time.
            int held = -1;  // the stage whose store may still be reading it
            for (int j = 0; j < nn; ++j, ++q, ++n2) {
                if ((int)(n2 & 1u) != grp) continue;
                const uint32_t sl = q % S, st = sbase + sl * Cfg::kStage;
                const int n0 = (na + j) * kKC;
                if (lane == 0 && held >= 0) {
                    bulk_wait_read<0>();
                    mbar_arrive(smem_u32(&sh.empty[held]));
                }
                bool ok = wait(smem_u32(&sh.full[sl]), (q / S) & 1u);
                ok = wait(smem_u32(&sh.d2_full[grp]), (n2 / 2) & 1u) && ok;
                __syncwarp();
                tc::fence_after_sync();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float o[32];
                    tmem_load<32>(lane_addr + 128 + grp * 64 + h * 32, o);
                    if (h == 1) {
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sh.d2_empty[grp]));
                    }
                    uint4 y[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        y[c] = g.base ? ld_shared_v4(st + tc::sw128_off(row, h * 4 + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float f[8];
                        Elt<T>::unpack(y[c], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = kF16 ? fmaf(o[c * 8 + e], down, f[e]) : f[e] + o[c * 8 + e];
                        st_shared_v4(st + tc::sw128_off(row, h * 4 + c), Elt<T>::pack(f));
                    }
                }
                // A warp's 32 rows leave together: by one TMA store where their tokens are consecutive
                // (drained while the warp goes on), else as rows of 128 bytes by eight lanes each.
                if (run32) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (ok) tma_store_2d(&maps.o, n0, tok, st + quarter * 4096);
                        bulk_commit();
                    }
                    held = (int)sl;
                } else {
                    __syncwarp();
                    const int c = lane & 7;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = quarter * 32 + i * 4 + (lane >> 3);
                        const int to = __shfl_sync(0xffffffffu, tok, i * 4 + (lane >> 3));
                        if (ok && r < t.rows && n0 + c * 8 < g.N)
                            *reinterpret_cast<uint4*>(static_cast<T*>(g.O) + (int64_t)to * g.ldo + n0 + c * 8) =
                                ld_shared_v4(st + tc::sw128_off(r, c));
                    }
                    fence_proxy_async_smem();  // O was written here by threads, what comes next is by TMA
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.empty[sl]));
                }
            }
            if (lane == 0 && held >= 0) {
                bulk_wait_read<0>();
                mbar_arrive(smem_u32(&sh.empty[held]));
            }
            named_barrier(1, kEpi);
            // This rank's products with P's parts are complete (their accumulators were read). Not after the
            // last tile: nobody would wait for that, and a CTA leaves only when nothing is on its way to it.
            if (et < C && it + ncl < ntiles) mbar_arrive_remote(smem_u32(&sh.freed), et);
        }
        if (lane == 0) bulk_wait<0>();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (sh.failed && tid == 0)  // the other ranks' stores may still be on their way to this CTA and back
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < kDrainNs / 100;) {
        }
    if (C > 1) cluster_sync_relaxed();  // nobody sends sums, parts or arrivals to this CTA any more
    if (warp == 1) tc::tmem_dealloc(tmem, Cfg::kTmem);
}

// ------------------------------------------------------------------ weight gradients

// Warps: 0 loads U (TMA), 1 multiplies (one thread), the others (four, from rank 17 on eight) write P's parts into
// the stages.
constexpr int kWgCols = 128;  // columns of U per cluster (the M of the products)
constexpr uint32_t kWgBars = 512;

template <typename T, int RP>
struct WgCfg {
    static constexpr int kTok = kParts<T> == 3 && RP > 64 ? 32 : 64;  // tokens of a stage
    static constexpr uint32_t kBlock = kTok * 128;                   // of 64 columns of them
    static constexpr uint32_t kU = kWgCols / 64 * kBlock;
    // RP columns of each part of P, one part behind the other, in blocks.
    static constexpr uint32_t kP = (kParts<T> * RP + 63) / 64 * kBlock;
    // One product takes all parts, each to sums of its own that are added in the end: the count of products is what
    // a third part costs (8192 tokens of 4 adapters, 2048 -> 8192, rank 16, a gradient: 82.9 us with two products per 16
    // tokens, 89.9 with three). At rank 128 the parts are too wide for that; bf16 adds them to the same sums there.
    static constexpr int kProducts = kParts<T> * RP <= 256 ? 1 : kParts<T>;
    static constexpr int kN = kParts<T> * RP / kProducts;
    static constexpr uint32_t kStage = kU + kP;
    static constexpr int kPerSm = RP <= 32 ? 3 : 2;
    static constexpr int kPWarps = RP <= 16 ? 4 : 8, kEpi = 32 * kPWarps, kThreads = 64 + kEpi;
    static constexpr uint32_t kBars = kWgBars + (kPWarps + 1) * RP * 4;  // and the columns' largest values and factors
    static constexpr uint32_t kBudget = (228 * 1024) / kPerSm / 1024 * 1024 - 1024;
    static constexpr int kStages = (int)((kBudget - kBars) / kStage);
    static constexpr uint32_t kSmem = kStages * kStage + kBars;
    static constexpr uint32_t kTmem = kN <= 32 ? 32 : kN <= 64 ? 64 : kN <= 128 ? 128 : 256;
    static_assert(kStages >= 2 && kStages * kStage >= RP * kWgCols * 4u, "the partial sums fit in the ring");
};

struct WgArgs {
    LoraPlanView v;
    LoraWgradArgs w[2];
    int blocks[2];  // 128-column blocks of each product
    const float* scale;
    float scale_all;
    int32_t rank;
    int early;  // the kernel before this one triggers once all before it is complete, and writes the dependent P
    int* err;
};

// A cluster takes 128 columns of one adapter's gradient; its CTAs split the adapter's tokens in
// chunks and their fp32 partial sums are added in rank order through distributed shared
// memory. U's rows are the K axis: a chunk is 64 (or 32) rows x 128 columns, an MN-major operand just as
// TMA writes it (boxes of 64 columns; four rows at a time where the tokens are not consecutive).
// Rows past the adapter's last token are asked for beyond the tensor, which fills zeros. P is
// read in fp32 and written to the stage as its parts by the warps that later drain the
// accumulators.
template <typename T, int RP>
__global__ void __launch_bounds__(WgCfg<T, RP>::kThreads, WgCfg<T, RP>::kPerSm)
lora_wgrad_kernel(const WgArgs g, const __grid_constant__ CUtensorMap map_u0, const __grid_constant__ CUtensorMap map_g0,
                  const __grid_constant__ CUtensorMap map_u1, const __grid_constant__ CUtensorMap map_g1) {
    using Cfg = WgCfg<T, RP>;
    constexpr int S = Cfg::kStages, kTok = Cfg::kTok, kPWarps = Cfg::kPWarps, kEpi = Cfg::kEpi;
    constexpr uint32_t kBlock = Cfg::kBlock;
    constexpr bool kF16 = std::is_same<T, __half>::value;
    constexpr uint32_t kIdesc = tc::instr_desc_f16(kF16 ? 0u : 1u, 1, 1, 128, Cfg::kN);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    struct Shared {
        uint64_t full[S], empty[S], done, drain;
        uint32_t tmem;
        volatile int failed;
        float col_max[kPWarps][RP];  // per warp; fp16: the largest of every rank's column of P
        float down[RP];        // what the columns were scaled by, inverted
    };
    static_assert(sizeof(Shared) <= Cfg::kBars, "barriers");
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw + S * Cfg::kStage);
    const uint32_t sbase = smem_u32(smem_raw);
    if (sbase & 1023u) {  // the same on every CTA
        record_error(g.err, kDevErrSmemAlign);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cluster_size(), crank = (int)cluster_rank();
    if (!g.early) pdl_wait();
    const int per = g.blocks[0] + g.blocks[1];
    const int item = blockIdx.x / C;
    const int adapter = g.v.aorder[item / per], blk = item % per;  // the longest first
    const int which = blk >= g.blocks[0];
    const LoraWgradArgs& w = g.w[which];
    const int n0 = (which ? blk - g.blocks[0] : blk) * kWgCols;
    // 16-byte stores of the gradient
    const bool vec_out = (reinterpret_cast<uintptr_t>(w.G) & 15) == 0 && (!w.rank_minor || g.rank % 8 == 0);
    const int p0 = g.v.off[adapter], cnt = g.v.off[adapter + 1] - p0;
    const int chunks = (cnt + kTok - 1) / kTok;
    const int ca = (int)((int64_t)chunks * crank / C), cb = (int)((int64_t)chunks * (crank + 1) / C);
    const int nc = cb - ca;
    const int pa = p0 + ca * kTok, pe = min(p0 + cnt, p0 + cb * kTok);  // this CTA's positions

    if (warp == 1) {
        tc::tmem_alloc(smem_u32(&sh.tmem), Cfg::kTmem);
        pdl_trigger();
    }
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1 + kPWarps);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        mbar_init(smem_u32(&sh.done), 1);
        mbar_init(smem_u32(&sh.drain), 1);
        fence_mbar_init();
        sh.failed = 0;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const Waits wait{&sh.failed, g.err};
    const bool dependent = g.early && w.dependent;

    if (warp == 0) {
        // ---------------- loads of U
        const uint64_t policy = evict_first_policy();
        const CUtensorMap* mu = which ? &map_u1 : &map_u0;
        const CUtensorMap* mg = which ? &map_g1 : &map_g0;
        int j = 0;
        for (; j < nc; ++j) {
            const int s = j % S;
            const uint32_t st = sbase + s * Cfg::kStage, fb = smem_u32(&sh.full[s]);
            const int b = pa + j * kTok, m = min(kTok, pe - b);
            // lane = 4 tokens (group lane % kTok / 4) and one of the two 64-column blocks
            constexpr int kGroups = kTok / 4;
            int y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = lane % kGroups * 4 + i;
                y[i] = at < m ? g.v.order[b + at] : g.v.tokens;  // past the last row: zeros
            }
            const int first = __shfl_sync(0xffffffffu, y[0], 0), last = __shfl_sync(0xffffffffu, y[3], kGroups - 1);
            const bool box = m == kTok && last - first == kTok - 1;
            if (j >= S && !__all_sync(0xffffffffu, wait(smem_u32(&sh.empty[s]), (j / S - 1) & 1u))) break;
            if (lane == 0) mbar_arrive_expect_tx(fb, Cfg::kU);
            __syncwarp();
            if (box) {
                if (lane < kWgCols / 64) tma_load_2d<true>(st + lane * kBlock, mu, n0 + lane * 64, first, fb, policy);
            } else if (lane < kWgCols / 64 * kGroups) {
                const int c = lane / kGroups;
                tma_gather4<true>(st + c * kBlock + lane % kGroups * 512, mg, n0 + c * 64, y, fb, policy);
            }
        }
        if (sh.failed) {
            for (int i = max(0, j - S); i < j; ++i)
                mbar_wait_for(smem_u32(&sh.full[i % S]), (i / S) & 1u, nullptr, kDrainNs);
        }
    } else if (warp == 1) {
        // ---------------- multiplications
        if (lane == 0) {
            for (int j = 0; j < nc; ++j) {
                const int s = j % S;
                const uint32_t st = sbase + s * Cfg::kStage;
                if (!wait(smem_u32(&sh.full[s]), (j / S) & 1u)) break;
                tc::fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < kTok / 16; ++kk)
#pragma unroll
                    for (int p = 0; p < Cfg::kProducts; ++p) {
                        const uint64_t ad = tc::smem_desc_sw128(st + kk * 2048, kBlock, 1024);
                        const uint64_t bd =
                            tc::smem_desc_sw128(st + Cfg::kU + p * (RP / 64) * kBlock + kk * 2048, kBlock, 1024);
                        tc::mma_f16(tmem, ad, bd, kIdesc, (j > 0 || kk > 0 || p > 0) ? 1u : 0u);
                    }
                tc::mma_commit(smem_u32(&sh.empty[s]));
            }
            tc::mma_commit(smem_u32(&sh.done));
            if (sh.failed) {
                tc::mma_commit(smem_u32(&sh.drain));
                mbar_wait_for(smem_u32(&sh.drain), 0, nullptr, kDrainNs);
            }
        }
        __syncwarp();
    } else {
        // ---------------- P's parts
        if (dependent) pdl_wait();  // the kernel before this one writes this P
        const int et = tid - 64;
        const int r = g.rank;
        const bool vec = r % 4 == 0 && (reinterpret_cast<uintptr_t>(w.P) & 15) == 0;
        // eight values of a token's P from column j0
        auto load8 = [&](int64_t t, int j0, float* x) {
            const float* src = w.P + t * r + j0;
            if (vec) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 f = j0 + 4 * i < r ? *reinterpret_cast<const float4*>(src + 4 * i) : make_float4(0, 0, 0, 0);
                    x[4 * i] = f.x;
                    x[4 * i + 1] = f.y;
                    x[4 * i + 2] = f.z;
                    x[4 * i + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = j0 + i < r ? src[i] : 0.f;
            }
        };
        constexpr int kCh = RP / 8;            // 8-column pieces per token
        constexpr int kPer = kTok * kCh / kEpi;  // pieces per thread of a chunk
        auto piece_token = [&](int j, int i) {  // the token of this thread's piece i of chunk j, -1: none
            const int at = pa + j * kTok + (et + i * kEpi) / kCh;
            return at < pe ? g.v.order[at] : -1;
        };
        auto load_piece = [&](int tok, int i, float* x) {
            if (tok >= 0) {
                load8(tok, (et + i * kEpi) % kCh * 8, x);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
            }
        };
        // fp16: every rank's column has a factor of its own (the sums are taken column by column), from the
        // largest magnitude among this CTA's tokens, eight (of eight warps four) pieces at a time (two memory
        // latencies: with four of four warps this took a third of the kernel). A thread's pieces are all of the same eight columns.
        const int c8 = et % kCh * 8;
        float up[8];
        if (kF16) {
            float m[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = 0.f;
            constexpr int kScan = kPWarps == 4 ? 8 : 4;
            for (int j = 0; j < nc * kPer; j += kScan) {
                int tok[kScan];
#pragma unroll
                for (int i = 0; i < kScan; ++i) tok[i] = piece_token((j + i) / kPer, (j + i) % kPer);
                float x[kScan][8];
#pragma unroll
                for (int i = 0; i < kScan; ++i) load_piece(tok[i], (j + i) % kPer, x[i]);
#pragma unroll
                for (int i = 0; i < kScan; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {  // (infinities leave the others their scale)
                        const float y = fabsf(x[i][e]);
                        if (y <= 3.402823466e38f) m[e] = fmaxf(m[e], y);
                    }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int d = 16; d >= kCh; d >>= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], d));
                if (lane < kCh) sh.col_max[warp - 2][c8 + e] = m[e];
            }
            named_barrier(1, kEpi);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float down;
                float most = sh.col_max[0][c8 + e];
#pragma unroll
                for (int v = 1; v < kPWarps; ++v) most = fmaxf(most, sh.col_max[v][c8 + e]);
                pow2_scale(most, up[e], down);
                if (et < kCh) sh.down[c8 + e] = down;
            }
        }
        // The next chunk's values, and the tokens of the one after, are on their way while a chunk
        // is written.
        float x[kPer][8];
        int tok[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) load_piece(piece_token(0, i), i, x[i]);
#pragma unroll
        for (int i = 0; i < kPer; ++i) tok[i] = piece_token(1, i);
        for (int j = 0; j < nc; ++j) {
            const int s = j % S;
            const uint32_t st = sbase + s * Cfg::kStage + Cfg::kU;
            float xn[kPer][8];
#pragma unroll
            for (int i = 0; i < kPer; ++i) load_piece(tok[i], i, xn[i]);
#pragma unroll
            for (int i = 0; i < kPer; ++i) tok[i] = piece_token(j + 2, i);
            if (j >= S) wait(smem_u32(&sh.empty[s]), (j / S - 1) & 1u);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int at = (et + i * kEpi) / kCh, c = (et + i * kEpi) % kCh;
                if (kF16)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[i][e] *= up[e];
                uint4 part[kParts<T>];
                split8<T>(x[i], part);
#pragma unroll
                for (int p = 0; p < kParts<T>; ++p) {
                    const int col = p * kCh + c;
                    st_shared_v4(st + (col >> 3) * kBlock + tc::sw128_off(at, col & 7), part[p]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.full[s]));
#pragma unroll
            for (int i = 0; i < kPer; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = xn[i][e];
        }
        wait(smem_u32(&sh.done), 0);
        __syncwarp();
        tc::fence_after_sync();
        // partial sums [j][128 columns] over the ring, which nothing uses any more
        const int quarter = warp & 3, row = quarter * 32 + lane;
        if (kF16) named_barrier(1, kEpi);  // the columns' factors are there
#pragma unroll
        for (int h = 0; h < RP / (4 * kPWarps); ++h) {
            const int c = h * (kPWarps / 4) + ((warp - 2) >> 2);
            const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + c * 16;
            float y[16];
            if (nc > 0) {
                // the last part's sums first; fp16: the second part was 2^kLoShift times larger
                constexpr int kSums = kParts<T> / Cfg::kProducts;
                tmem_load<16>(at + (kSums - 1) * RP, y);
#pragma unroll
                for (int p = kSums - 2; p >= 0; --p) {
                    float h[16];
                    tmem_load<16>(at + p * RP, h);
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = kF16 ? fmaf(y[i], 1.f / (1 << kLoShift), h[i]) : y[i] + h[i];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (kF16) y[i] *= sh.down[c * 16 + i];
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) st_shared_f32(sbase + ((c * 16 + i) * kWgCols + row) * 4, y[i]);
        }
        tc::fence_before_sync();
    }
    __syncthreads();
    if (C > 1) {
        cluster_release_smem();
        cluster_sync_relaxed();
    }
    {
        // this rank's share of the columns, every sum in rank order, eight values at a time: of a
        // row j (N is a multiple of 8), or of a column where the ranks are the contiguous axis
        const int nx = kWgCols / C, x0 = nx * crank, r = g.rank;
        const float s = g.scale_all * (g.scale ? g.scale[adapter] : 1.f);
        T* G = static_cast<T*>(w.G) + (int64_t)adapter * r * w.N;
        const int r8 = (r + 7) / 8, n8 = nx / 8;
        const int items = sh.failed ? 0 : (w.rank_minor ? nx * r8 : r * n8);
        for (int i = tid; i < items; i += Cfg::kThreads) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.f;
            if (w.rank_minor) {
                const int j0 = i / nx * 8, x = x0 + i % nx;
                if (n0 + x >= w.N) continue;
                for (int c = 0; c < C; ++c) {
                    const uint32_t from = cluster_map(sbase + (j0 * kWgCols + x) * 4, c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] += ld_cluster_f32(from + e * kWgCols * 4);  // (j < RP)
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= s;
                T* to = G + (int64_t)(n0 + x) * r + j0;
                if (vec_out) {
                    *reinterpret_cast<uint4*>(to) = Elt<T>::pack(y);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (j0 + e < r) to[e] = Elt<T>::from_f(y[e]);
                }
            } else {
                const int j = i / n8, x = x0 + i % n8 * 8;
                if (n0 + x >= w.N) continue;
                for (int c = 0; c < C; ++c) {
                    const uint32_t from = cluster_map(sbase + (j * kWgCols + x) * 4, c);
                    const float4 a = ld_cluster_f4(from), b = ld_cluster_f4(from + 16);
                    y[0] += a.x;
                    y[1] += a.y;
                    y[2] += a.z;
                    y[3] += a.w;
                    y[4] += b.x;
                    y[5] += b.y;
                    y[6] += b.z;
                    y[7] += b.w;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= s;
                T* to = G + (int64_t)j * w.N + n0 + x;
                if (vec_out) {
                    *reinterpret_cast<uint4*>(to) = Elt<T>::pack(y);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) to[e] = Elt<T>::from_f(y[e]);
                }
            }
        }
    }
    if (g.early && !dependent) pdl_wait();  // so that the kernel before this one has ended when this one has
    __syncthreads();
    if (C > 1) cluster_sync_relaxed();  // nobody reads this CTA's sums any more
    if (warp == 1) tc::tmem_dealloc(tmem, Cfg::kTmem);
}

// ------------------------------------------------------------------ host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return f;
}

// Tensor map of a dim-dimensional tensor of 16-bit elements (strides in elements, of dimensions
// 1 ..) with the 128-byte swizzle and boxes 64 elements wide.
bool encode(CUtensorMap* map, bool bf16, const void* base, int dim, const int64_t* sizes, const int64_t* strides,
            int box1) {
    cuuint64_t d[3], st[2];
    cuuint32_t box[3] = {64, (cuuint32_t)box1, 1}, elem[3] = {1, 1, 1};
    for (int i = 0; i < dim; ++i) d[i] = (cuuint64_t)sizes[i];
    for (int i = 0; i + 1 < dim; ++i) st[i] = (cuuint64_t)strides[i] * 2;
    return encode_fn()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dim,
                       const_cast<void*>(base), d, st, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(CUtensorMap* map, bool bf16, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const int64_t sizes[2] = {cols, rows}, strides[1] = {ld};
    return encode(map, bf16, p, 2, sizes, strides, box_rows);
}

// What a row-strided operand needs for 16-byte TMA rows.
bool rows_ok(const void* p, int64_t cols, int64_t ld) {
    return cols % 8 == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld < (1ll << 38);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), int64_t clusters, int c, int threads, uint32_t smem, cudaStream_t s,
                            const Args&... args) {
    const cudaError_t e = launch_pdl_cluster(kern, dim3((unsigned)(clusters * c)), dim3((unsigned)threads), smem,
                                             (unsigned)c, s, args...);
    count_launches(1);
    return e;
}

// The dynamic shared memory limit of a kernel, raised once per device.
template <typename K>
cudaError_t allow_smem(K kern, uint32_t smem, bool (&done)[64]) {
    const int d = device_props().device;
    if (d >= 0 && d < 64 && done[d]) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && d >= 0 && d < 64) done[d] = true;
    return e;
}

template <typename T, bool kBack, int RP>
cudaError_t run_tiles(const LoraArgs& a, const LoraPlanView& v, cudaStream_t s) {
    using Cfg = TileCfg<T, RP>;
    static bool done[64];
    auto kern = lora_tile_kernel<T, kBack, RP>;
    cudaError_t e = allow_smem(kern, Cfg::kSmem, done);
    if (e != cudaSuccess) return e;
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    TileMaps m;
    const int64_t in = kBack ? a.N : a.K, out = kBack ? a.K : a.N;
    const int64_t sa[3] = {in, a.rank, v.n}, ta[2] = {in, in * a.rank};
    const int64_t sb[3] = {a.rank, out, v.n}, tb[2] = {a.rank, out * a.rank};
    TileArgs g;
    g.hand = a.rank % 8 != 0;
    bool ok = encode(&m.a, bf, a.A, 3, sa, ta, RP);
    m.b = m.o = m.a;  // maps that are not used are valid ones
    if (!g.hand) ok = ok && encode(&m.b, bf, a.B, 3, sb, tb, 64);
    for (int i = 0; i < kBoxes; ++i) {
        ok = ok && encode_rows(&m.u[i], bf, a.U, v.tokens, a.K, a.ldu, kBoxRows[i]);
        m.base[i] = m.u[i];
        if (a.O && a.base) ok = ok && encode_rows(&m.base[i], bf, a.base, v.tokens, a.N, a.ldb, kBoxRows[i]);
    }
    if (a.O) ok = ok && encode_rows(&m.o, bf, a.O, v.tokens, a.N, a.ldo, 32);
    if (!ok) return cudaErrorInvalidValue;
    g.v = v;
    g.B = a.B;
    g.scale = a.scale;
    g.base = a.O ? a.base : nullptr;
    g.O = a.O;
    g.P = a.P;
    g.ldb = a.ldb;
    g.ldo = a.ldo;
    g.K = a.K;
    g.N = a.N;
    g.rank = a.rank;
    g.scale_all = a.scale_all;
    g.err = device_error_word();
    // As many CTAs per tile as the SMs hold at once for the tiles to expect (cap is the most there can
    // be), and enough that a thread sums eight columns at most.
    const int64_t slots = (int64_t)device_props().sm_count * Cfg::kPerSm;
    const int64_t cap = lora_tiles_cap(v.tokens, v.n, kLoraTile);
    const int64_t expected =
        min64(cap, ((int64_t)v.tokens + kLoraTile - 1) / kLoraTile + (v.n > 1 ? min64(v.tokens, v.n) / 2 : 0));
    int c = 8;
    while (c > Cfg::kMinCluster && expected * c > slots) c /= 2;
    const int64_t clusters = max64(1, min64(cap, slots / c));
    return launch_clusters(kern, clusters, c, kTileThreads, Cfg::kSmem, s, g, m);
}

template <typename T, int RP>
cudaError_t run_wgrad(const LoraWgradArgs* w, int nw, int32_t rank, const float* scale, float scale_all,
                      const LoraPlanView& v, bool early, cudaStream_t s) {
    using Cfg = WgCfg<T, RP>;
    static bool done[64];
    auto kern = lora_wgrad_kernel<T, RP>;
    cudaError_t e = allow_smem(kern, Cfg::kSmem, done);
    if (e != cudaSuccess) return e;
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    CUtensorMap mu[2], mg[2];
    WgArgs g;
    g.blocks[1] = 0;
    for (int i = 0; i < nw; ++i) {
        g.w[i] = w[i];
        g.blocks[i] = (w[i].N + kWgCols - 1) / kWgCols;
        if (!encode_rows(&mu[i], bf, w[i].U, v.tokens, w[i].N, w[i].ldu, Cfg::kTok) ||
            !encode_rows(&mg[i], bf, w[i].U, v.tokens, w[i].N, w[i].ldu, 1))
            return cudaErrorInvalidValue;
    }
    if (nw == 1) {
        mu[1] = mu[0];
        mg[1] = mg[0];
    }
    g.v = v;
    g.scale = scale;
    g.scale_all = scale_all;
    g.rank = rank;
    g.early = early;
    g.err = device_error_word();
    const int64_t items = (int64_t)v.n * (g.blocks[0] + g.blocks[1]);
    int c = 1;
    const int64_t slots = (int64_t)device_props().sm_count * Cfg::kPerSm;
    while (c < 8 && items * c * 2 <= slots && (int64_t)v.tokens >= 64ll * c * 2) c *= 2;
    if (items * c > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_clusters(kern, items, c, Cfg::kThreads, Cfg::kSmem, s, g, mu[0], mg[0], mu[1], mg[1]);
}

template <typename T>
cudaError_t run_wgrad_rank(const LoraWgradArgs* w, int nw, int32_t rank, const float* scale, float scale_all,
                           const LoraPlanView& v, bool early, cudaStream_t s) {
    if (rank <= 16) return run_wgrad<T, 16>(w, nw, rank, scale, scale_all, v, early, s);
    if (rank <= 32) return run_wgrad<T, 32>(w, nw, rank, scale, scale_all, v, early, s);
    if (rank <= 64) return run_wgrad<T, 64>(w, nw, rank, scale, scale_all, v, early, s);
    return run_wgrad<T, 128>(w, nw, rank, scale, scale_all, v, early, s);
}

template <typename T, bool kBack>
cudaError_t run_tiles_rank(const LoraArgs& a, const LoraPlanView& v, cudaStream_t s) {
    if (a.rank <= 16) return run_tiles<T, kBack, 16>(a, v, s);
    if (a.rank <= 32) return run_tiles<T, kBack, 32>(a, v, s);
    if (a.rank <= 64) return run_tiles<T, kBack, 64>(a, v, s);
    return run_tiles<T, kBack, 128>(a, v, s);
}

}  // namespace

bool lora_tiles_ok(int dt, const LoraArgs& a, const LoraPlanView& v) {
    if (dt == kF32 || !encode_fn()) return false;
    if (!rows_ok(a.U, a.K, a.ldu) || a.N % 8 != 0) return false;
    if (a.O && (!rows_ok(a.O, a.N, a.ldo) || (a.base && !rows_ok(a.base, a.N, a.ldb)))) return false;
    return (reinterpret_cast<uintptr_t>(a.A) | reinterpret_cast<uintptr_t>(a.B)) % 16 == 0;
}

cudaError_t launch_lora_tiles(int dt, bool back, const LoraArgs& a, const LoraPlanView& v, cudaStream_t s) {
    if (dt == kF16)
        return back ? run_tiles_rank<__half, true>(a, v, s) : run_tiles_rank<__half, false>(a, v, s);
    return back ? run_tiles_rank<__nv_bfloat16, true>(a, v, s) : run_tiles_rank<__nv_bfloat16, false>(a, v, s);
}

bool lora_wgrad_tiles_ok(int dt, const LoraWgradArgs* w, int nw) {
    if (dt == kF32 || !encode_fn()) return false;
    for (int i = 0; i < nw; ++i)
        if (!rows_ok(w[i].U, w[i].N, w[i].ldu)) return false;
    return true;
}

cudaError_t launch_lora_wgrad_tiles(int dt, const LoraWgradArgs* w, int nw, int32_t rank, const float* scale,
                                    float scale_all, const LoraPlanView& v, bool after_lora, cudaStream_t s) {
    return dt == kF16 ? run_wgrad_rank<__half>(w, nw, rank, scale, scale_all, v, after_lora, s)
                      : run_wgrad_rank<__nv_bfloat16>(w, nw, rank, scale, scale_all, v, after_lora, s);
}

}  // namespace spops
