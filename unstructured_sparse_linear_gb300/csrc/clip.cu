// Global 2-norm of many tensors and clipping by it:
//     norm = sqrt(sum of g^2 over every gradient),  c = min(1, max_norm / (norm + 1e-6)),
//     out = c g (rounded once to the gradient's type).
// One launch whatever the number of tensors: the table of the set lies in device memory, with
// every tensor cut into chunks of 32 KB; the chunks are dealt to the CTAs (one per SM) in
// contiguous, equal ranges, so the sums have one order (no float atomics) and a CTA looks its first
// tensor up once. One thread keeps a ring of six chunks (192 KB) in flight with bulk copies of
// whole 16-byte granules (the neighbours' bytes in the first and the last one are masked), 16 warps
// work on them; scaled chunks leave from where they lie by bulk stores, the elements of granules
// that belong to a neighbour too by plain ones. With loads to registers instead (two CTAs of 512
// threads, 64 bytes a thread, two chunks under way) 166 MB of bf16 took 88 us.
// Between the passes the CTAs wait for each other (a cooperative launch) and add their partial sums
// themselves, in one order. The second pass walks backwards: its first six chunks are still in
// shared memory, the ones before them are the part of the set that L2 was asked to keep.
//
// Squares are added in fp32 within a warp's share of up to 4 chunks, then in fp64. A thread's
// group whose fp32 sum leaves [1e-30, 1e30] (squares that overflow or vanish in fp32, up to the
// largest and down to the smallest numbers of the type) is added again in fp64 from the same
// registers, so the norm itself neither overflows nor underflows before it is rounded.
// Bound: HBM (2 N b plus what of the second read misses L2).
#include "clip.h"
#include "common.cuh"
#include "internal.h"

namespace spops {
namespace {

constexpr int kWarps = 16;                // working warps
constexpr int kWork = kWarps * 32;
constexpr int kThreads = kWork + 32;      // and one that loads
constexpr int kStages = 6;
constexpr uint64_t kDrainNs = 1000000ull;  // after a failed wait: for copies still in flight
constexpr uint32_t kStage = 32768;
constexpr uint32_t kKeep = 96u << 20;  // bytes of the set that the first pass asks L2 to keep (166 MB: 79.5 us, with 64 MB 80.2)
constexpr int kVecs = kStage / 16 / kWork;  // granules per thread and chunk

__global__ void grad_set_fill_kernel(ClipEntry* set, const __grid_constant__ ClipFill f, int n,
                                     unsigned long long* arrived) {
    const int i = threadIdx.x;
    if (i < n) set[i] = f.e[i];
    if (i == 0) *arrived = 0;
}

// The tensor that chunk c belongs to: the last one with first <= c (tensors without elements share
// their first chunk with the next one). Called by the whole CTA: `first` does not fall, so the
// tensors with first <= c are counted, one round of loads per 544 tensors instead of the ten
// dependent ones of a bisection.
__device__ __forceinline__ int find_tensor(const ClipEntry* set, int tensors, int64_t c) {
    int n = 0;
    for (int b = 0; b < tensors; b += kThreads) {
        const int i = b + (int)threadIdx.x;
        n += __syncthreads_count(i < tensors && set[i].first <= c);
    }
    return n - 1;
}

// L2 policies for bulk copies, and the copies with one.
__device__ __forceinline__ uint64_t l2_policy(bool keep) {
    uint64_t p;
    if (keep) asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    else asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void bulk_g2s_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void bulk_s2g_hint(void* dst, uint32_t src, uint32_t bytes, uint64_t policy) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;" ::"l"(dst), "r"(src),
                 "r"(bytes), "l"(policy)
                 : "memory");
}

// A chunk in a stage: len elements from byte `off` of `granules` 16-byte granules on, of type
// dtype; out: where they go.
struct Piece {
    char* out;
    int len, off, granules, dtype;
};

struct __align__(16) Shared {
    uint64_t full[kStages], empty[kStages];
    Piece piece[kStages];
    double warp[kWarps];
    float c;
    volatile int failed;
    volatile int stop;  // the chunks not yet asked for are not wanted
    int go;             // every CTA has added its squares
};
constexpr uint32_t kSmem = kStages * kStage + ((sizeof(Shared) + 127) / 128 * 128);

// The CTA's chunks are c0 + i, i < n; chunk i lies in stage i % kStages in both passes, and its load is
// an even or odd use of the stage as i / kStages is: the first pass counts up, and a second one that
// starts at the last chunk counts down from there.
__device__ __forceinline__ uint32_t use_parity(uint32_t i) { return (i / kStages) & 1u; }

// Asks for chunk i of tensor `e`, once its stage is free; false if that took too long or the rest is not
// wanted. wait: the stage was used before.
__device__ __forceinline__ bool load_chunk(const ClipEntry& e, int64_t c, uint32_t i, bool wait, uint64_t policy,
                                           uint32_t sbase, Shared& sh, int* err) {
    const int esize = e.dtype == kF32 ? 4 : 2;
    const int64_t per = kClipChunk / esize, at = (c - e.first) * per;
    Piece p;
    p.dtype = e.dtype;
    p.len = (int)min64(per, e.count - at);
    p.out = static_cast<char*>(e.out) + at * esize;
    const char* in = static_cast<const char*>(e.in) + at * esize;
    p.off = (int)(reinterpret_cast<uintptr_t>(in) & 15);
    p.granules = (p.off + p.len * esize + 15) / 16;
    const uint32_t s = i % kStages, full = smem_u32(&sh.full[s]);
    if (wait) {
        if (sh.failed) return false;
        if (!mbar_wait(smem_u32(&sh.empty[s]), use_parity(i) ^ 1u, err)) {
            sh.failed = 1;
            return false;
        }
        if (sh.stop) return false;
    }
    sh.piece[s] = p;
    mbar_arrive_expect_tx(full, (uint32_t)p.granules * 16);
    bulk_g2s_hint(sbase + s * kStage, in - p.off, (uint32_t)p.granules * 16, full, policy);
    return true;
}

// The loading thread. First pass: chunks 0 .. n - 1, to stay in L2 the `keep` before the last kStages; t: the tensor of
// the first one. Second pass: from n - 1 - kStages down (the last kStages chunks are in their stages).
__device__ __forceinline__ void load_chunks(const ClipEntry* set, int tensors, int t, int64_t c0, uint32_t n, int64_t keep,
                                            bool both, uint32_t sbase, Shared& sh, int* err) {
    const uint64_t pass = l2_policy(false), stay = l2_policy(true);
    uint32_t i = 0;
    bool ok = true;
    for (; i < n && ok; ++i) {
        const int64_t c = c0 + i;
        while (t + 1 < tensors && set[t + 1].first <= c) ++t;
        ok = load_chunk(set[t], c, i, i >= kStages, i + kStages + keep < n || i + kStages >= n ? pass : stay, sbase, sh, err);
    }
    if (both && ok)
        for (i = n > kStages ? n - kStages : 0; i-- > 0 && ok;) {
            const int64_t c = c0 + i;
            while (set[t].first > c) --t;
            ok = load_chunk(set[t], c, i, true, pass, sbase, sh, err);
        }
    if (sh.failed) {  // let the copies in flight land before the shared memory is given up
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < kDrainNs) {
        }
    }
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

struct Sum {
    float f = 0.f;   // groups in the range where fp32 squares are safe
    double d = 0.0;  // the others
};

// One group of a thread: x[0 .. N).
template <int N>
__device__ __forceinline__ void add_group(const float (&x)[N], Sum& s) {
    float p = 0.f, m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p = fmaf(x[i], x[i], p);
        m = fmaxf(m, fabsf(x[i]));
    }
    if ((p >= 1e-30f && p <= 1e30f) || (p == 0.f && m == 0.f)) {
        s.f += p;
    } else {  // also NaN and infinities, which stay what they are
        double q = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) q += (double)x[i] * (double)x[i];
        s.d += q;
    }
}

// The sum over the warp, in every lane: fp32 where all of it is there. fp64 runs at a 64th of the
// fp32 rate here, so it is kept to a few values per warp (reductions in fp64 by every thread took
// 20 us of a 30 us call).
__device__ __forceinline__ double warp_sum(const Sum& s) {
    float f = s.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) f += __shfl_xor_sync(0xffffffffu, f, d);
    double x = (double)f;
    if (__any_sync(0xffffffffu, s.d != 0.0)) {  // (NaN != 0)
        double y = s.d;
#pragma unroll
        for (int d = 16; d; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
        x += y;
    }
    return x;
}

template <typename T>
__device__ __forceinline__ void squares(const Piece& p, uint32_t st, Sum& s) {
    constexpr int V = Elt<T>::kVec;
    const int tid = threadIdx.x, first = p.off / (int)sizeof(T), last = first + p.len;  // elements of the stage
    float x[kVecs * V];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kWork + tid;
        Elt<T>::unpack(i < p.granules ? ld_shared_v4(st + i * 16) : make_uint4(0, 0, 0, 0), x + u * V);
        if (i == 0 || i == p.granules - 1)
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (i * V + k < first || i * V + k >= last) x[u * V + k] = 0.f;
    }
    add_group(x, s);
}

__device__ __forceinline__ void init_ring(Shared& sh) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), kWarps);
        }
        fence_mbar_init();
        sh.failed = 0;
        sh.stop = 0;
    }
    __syncthreads();
}

// Waits for chunk i; false (on some lanes perhaps) once a wait has run out of time.
__device__ __forceinline__ bool wait_stage_one(Shared& sh, uint32_t i, int* err) {
    if (sh.failed) return false;
    if (mbar_wait(smem_u32(&sh.full[i % kStages]), use_parity(i), err)) return true;
    sh.failed = 1;
    return false;
}
__device__ __forceinline__ bool wait_stage(Shared& sh, uint32_t i, int* err) {
    const bool ok = wait_stage_one(sh, i, err);
    __syncwarp();
    return ok;
}

// The first pass of a working warp: its squares of the CTA's n chunks. The stages of the last `hold`
// chunks are not given back.
__device__ __forceinline__ double sum_chunks(uint32_t n, uint32_t hold, uint32_t sbase, Shared& sh, int* err) {
    const int lane = threadIdx.x & 31;
    double total = 0.0;
    Sum s;
    for (uint32_t i = 0; i < n; ++i) {
        const uint32_t st = sbase + (i % kStages) * kStage;
        wait_stage(sh, i, err);
        const Piece p = sh.piece[i % kStages];
        if (p.dtype == kF32) squares<float>(p, st, s);
        else if (p.dtype == kF16) squares<__half>(p, st, s);
        else squares<__nv_bfloat16>(p, st, s);
        __syncwarp();
        if (lane == 0 && i + hold < n) mbar_arrive(smem_u32(&sh.empty[i % kStages]));
        if ((i & 3u) == 3u || i + 1 == n) {  // short fp32 runs
            total += warp_sum(s);
            s = Sum();
        }
    }
    return total;
}

// The CTA's sum from its warps', by warp 0 (in every lane).
__device__ __forceinline__ double cta_sum(const Shared& sh) {
    const int lane = threadIdx.x & 31;
    double x = lane < kWarps ? sh.warp[lane] : 0.0;
#pragma unroll
    for (int d = kWarps / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

__global__ void __launch_bounds__(kThreads, 1) grad_norm_kernel(const ClipEntry* __restrict__ set, int tensors,
                                                               int64_t chunks, double* __restrict__ partial, int* err) {
    extern __shared__ __align__(128) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + kStages * kStage);
    const uint32_t sbase = smem_u32(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    const int64_t c0 = chunks * blockIdx.x / gridDim.x;
    const uint32_t n = (uint32_t)(chunks * (blockIdx.x + 1) / gridDim.x - c0);
    init_ring(sh);
    const int t = n > 0 ? find_tensor(set, tensors, c0) : 0;
    if (warp == kWarps) {
        if (lane == 0 && n > 0) load_chunks(set, tensors, t, c0, n, 0, false, sbase, sh, err);
    } else {
        const double total = sum_chunks(n, 0, sbase, sh, err);
        if (lane == 0) sh.warp[warp] = total;
    }
    __syncthreads();
    if (warp == 0) {
        const double x = cta_sum(sh);
        if (lane == 0) partial[blockIdx.x] = x;
    }
}

// The sum of the partial sums in one order, by the calling warp (the same in every lane).
__device__ __forceinline__ double total_of(const double* partial, int ctas) {
    double x = 0.0;
    for (int b = 0; b < ctas; b += 256) {
        double v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = b + u * 32 + (threadIdx.x & 31);
            v[u] = i < ctas ? __ldcg(partial + i) : 0.0;  // (written since this kernel started)
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) x += v[u];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// sqrt(x) = root 2^half, root in [1, 2) (0, infinity and NaN: themselves, half = 0): fp32 from here on, as
// fp64's square root and division are some fifty dependent operations at a 64th of the rate.
__device__ __forceinline__ float root_of(double x, int& half) {
    half = 0;
    if (!(x > 0.0 && x <= 1.7976931348623157e308)) return (float)x;
    const int e = (int)((__double2hiint(x) >> 20) & 0x7ff) - 1023;  // (sums of squares of fp32 values are normal)
    half = e >> 1;
    return sqrtf((float)(x * __hiloint2double((1023 - 2 * half) << 20, 0)));  // of [1, 4)
}
// f 2^k, without leaving the range on the way.
__device__ __forceinline__ float scaled(float f, int k) {
    const int a = k / 2;
    return f * __int_as_float((a + 127) << 23) * __int_as_float((k - a + 127) << 23);
}
__device__ __forceinline__ float norm_of(double total) {
    int half;
    const float root = root_of(total, half);
    return scaled(root, half);
}
// min(1, max_norm / (norm + 1e-6)).
__device__ __forceinline__ float factor_of(double total, double max_norm) {
    int half;
    const float root = root_of(total, half), norm = scaled(root, half), m = (float)max_norm;
    if (isinf(m)) return 1.f;
    // beyond the reach of 1e-6 (and where norm may be infinite) the power of two is taken last
    const float c = half > 100 ? scaled(m / root, -half) : m / (norm + 1e-6f);
    return c >= 1.f ? 1.f : c;  // NaN stays NaN
}

// Waits until every CTA of the (cooperative) grid has come here; what their calling threads wrote before is
// then visible to this one. arrived counts up for good, by gridDim.x per launch. Gives up after 2 s.
__device__ __forceinline__ int wait_for_all(unsigned long long* arrived, int* err) {
    __threadfence();
    const unsigned long long before = atomicAdd(arrived, 1ull);
    const unsigned long long all = (before / gridDim.x + 1) * gridDim.x;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        unsigned long long now;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(now) : "l"(arrived) : "memory");
        if (now >= all) return 1;
        if (global_timer_ns() - t0 > kMbarTimeoutNs) {
            record_error(err, kDevErrGridBarrier);
            return 0;
        }
    }
}

__global__ void __launch_bounds__(32) grad_norm_finish_kernel(const double* __restrict__ partial, int ctas,
                                                              float* __restrict__ norm_out) {
    pdl_wait();
    const double total = total_of(partial, ctas);
    if (threadIdx.x == 0) *norm_out = norm_of(total);
}

// The chunk times c: whole granules of the tensor in place (they leave by a bulk store), elements
// of shared granules, and everything where out's granules are not in's, straight to out.
template <typename T>
__device__ __forceinline__ void scale_chunk(const Piece& p, uint32_t st, float c, bool bulk) {
    constexpr int V = Elt<T>::kVec;
    const int tid = threadIdx.x, first = p.off / (int)sizeof(T), last = first + p.len;
    T* out = reinterpret_cast<T*>(p.out) - first;  // of element 0 of the stage
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kWork + tid;
        if (i >= p.granules) continue;
        float x[V];
        Elt<T>::unpack(ld_shared_v4(st + i * 16), x);
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] *= c;
        if (bulk && i * V >= first && i * V + V <= last) {
            st_shared_v4(st + i * 16, Elt<T>::pack(x));
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (i * V + k >= first && i * V + k < last) out[i * V + k] = Elt<T>::from_f(x[k]);
        }
    }
}

// Both passes in one cooperative launch (its CTAs wait for one another between the passes): the last six
// chunks of every CTA stay in shared memory and are not read again, 29 MB of the set in all.
__global__ void __launch_bounds__(kThreads, 1)
grad_clip_kernel(const ClipEntry* __restrict__ set, int tensors, int64_t chunks, double* __restrict__ partial,
                 unsigned long long* __restrict__ arrived, double max_norm, int in_place, float* __restrict__ norm_out,
                 int* err) {
    extern __shared__ __align__(128) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + kStages * kStage);
    const uint32_t sbase = smem_u32(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = chunks * blockIdx.x / gridDim.x;
    const uint32_t n = (uint32_t)(chunks * (blockIdx.x + 1) / gridDim.x - c0);
    init_ring(sh);
    const int t = n > 0 ? find_tensor(set, tensors, c0) : 0;
    if (warp == kWarps) {
        if (lane == 0 && n > 0)
            load_chunks(set, tensors, t, c0, n, kKeep / kStage / gridDim.x, true, sbase, sh, err);
    } else {
        const double total = sum_chunks(n, kStages, sbase, sh, err);
        if (lane == 0) sh.warp[warp] = total;
        named_barrier(1, kWork);
        if (warp == 0) {
            const double x = cta_sum(sh);
            if (lane == 0) {
                partial[blockIdx.x] = x;
                sh.go = wait_for_all(arrived, err);
            }
            __syncwarp();
            const double sum = total_of(partial, gridDim.x);
            if (lane == 0) {
                sh.c = factor_of(sum, max_norm);
                if (blockIdx.x == 0 && sh.go) *norm_out = norm_of(sum);
            }
        }
        named_barrier(1, kWork);
        const float c = sh.c;
        if (!sh.go || (c == 1.f && in_place)) {  // in place with c = 1 every gradient holds its value
            if (threadIdx.x == 0) {
                sh.stop = 1;
                if (n > kStages)  // what the loading thread waits for
                    for (int w = 0; w < kWarps; ++w) mbar_arrive(smem_u32(&sh.empty[(n - 1) % kStages]));
            }
        } else {
            const uint64_t pass = l2_policy(false);
            int held = -1;  // the stage whose store may still be reading it
            for (uint32_t i = n; i-- > 0;) {
                const uint32_t s = i % kStages, st = sbase + s * kStage;
                const bool ok = i + kStages >= n ? !sh.failed : wait_stage(sh, i, err);
                const Piece p = sh.piece[s];
                const bool bulk = ((reinterpret_cast<uintptr_t>(p.out) & 15) == (uintptr_t)p.off);
                if (ok) {
                    if (p.dtype == kF32) scale_chunk<float>(p, st, c, bulk);
                    else if (p.dtype == kF16) scale_chunk<__half>(p, st, c, bulk);
                    else scale_chunk<__nv_bfloat16>(p, st, c, bulk);
                }
                fence_proxy_async_smem();
                named_barrier(1, kWork);
                if (threadIdx.x == 0) {
                    const int esize = p.dtype == kF32 ? 4 : 2;
                    const int a = p.off ? 1 : 0, b = (p.off + p.len * esize) / 16;  // whole granules [a, b)
                    if (ok && bulk && b > a)
                        bulk_s2g_hint(p.out - p.off + a * 16, st + a * 16, (uint32_t)(b - a) * 16, pass);
                    bulk_commit();
                    // the store before this one has been read out: its stage is free
                    bulk_wait_read<1>();
                    if (held >= 0)
                        for (int w = 0; w < kWarps; ++w) mbar_arrive(smem_u32(&sh.empty[held]));
                    held = (int)s;
                }
            }
            if (threadIdx.x == 0) bulk_wait<0>();
        }
    }
    __syncthreads();
}

}  // namespace

cudaError_t launch_grad_set_fill(void* set, int64_t at, const ClipFill& f, int n, cudaStream_t s) {
    grad_set_fill_kernel<<<1, kClipFill, 0, s>>>(grad_set_entries(set) + at, f, n, grad_set_arrived(set));
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_grad_norm(void* set, int32_t tensors, int64_t chunks, bool in_place, bool scale, double max_norm,
                             float* norm_out, double* partial, cudaStream_t s) {
    static bool done[64];
    const int d = device_props().device;
    if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
    if (!done[d]) {
        cudaError_t e = cudaFuncSetAttribute(grad_norm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(grad_clip_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        done[d] = true;
    }
    int* err = device_error_word();
    const ClipEntry* entries = grad_set_entries(set);
    const int ctas = (int)max64(1, min64(chunks, min64(device_props().sm_count, kClipMaxCtas)));
    if (scale) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        count_launches(1);
        return cudaLaunchKernelEx(&cfg, grad_clip_kernel, entries, (int)tensors, chunks, partial, grad_set_arrived(set),
                                  max_norm, (int)in_place, norm_out, err);
    }
    grad_norm_kernel<<<ctas, kThreads, kSmem, s>>>(entries, tensors, chunks, partial, err);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_pdl(grad_norm_finish_kernel, dim3(1), dim3(32), 0, s, (const double*)partial, ctas, norm_out);
    count_launches(2);
    return e;
}

}  // namespace spops
