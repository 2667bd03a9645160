// Gradient clipping by the global 2-norm of many tensors:
//     norm = sqrt(sum of g^2 over every gradient),  c = min(1, max_norm / (norm + 1e-6)),
//     out = c g (rounded once to the gradient's type).
// Two launches whatever the number of tensors: the table of the set lies in device memory,
// with every tensor cut into chunks of 32 KB; the chunks are dealt to the CTAs in
// contiguous, equal ranges, so the sums have one order (no atomics) and a CTA looks its first
// tensor up once. The second kernel adds the CTAs' partial sums itself, in one order, and walks
// its range backwards: the part of the set that the first pass read last is still in L2.
//
// Squares are added in fp32 within a warp's share of up to 4 chunks, then in fp64. A
// group whose fp32 sum leaves [1e-30, 1e30] (squares that overflow or vanish in fp32, up to the
// largest and down to the smallest numbers of the type) is added again in fp64 from the same
// registers, so the norm itself neither overflows nor underflows before it is rounded.
// Bound: HBM (2 N b plus what of the second read misses L2).
#include "clip.h"
#include "common.cuh"
#include "internal.h"

namespace spops {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 2;

__global__ void grad_set_fill_kernel(ClipEntry* set, const __grid_constant__ ClipFill f, int n) {
    const int i = threadIdx.x;
    if (i < n) set[i] = f.e[i];
}

// fp64 runs at a 64th of the fp32 rate here, so it is kept to a few values per CTA: threads and
// warps add in fp32, what leaves a warp is fp64 (a block reduction in fp64 by every thread took
// 20 us of a 30 us call).

// The tensor that chunk c belongs to: the last one with first <= c (tensors without elements share
// their first chunk with the next one). Called by the whole CTA: `first` does not fall, so the
// tensors with first <= c are counted, one round of loads per 512 tensors instead of the ten
// dependent ones of a bisection.
__device__ __forceinline__ int find_tensor(const ClipEntry* set, int tensors, int64_t c) {
    int n = 0;
    for (int b = 0; b < tensors; b += kThreads) {
        const int i = b + (int)threadIdx.x;
        n += __syncthreads_count(i < tensors && set[i].first <= c);
    }
    return n - 1;
}

// One chunk: len elements of a tensor, the same on every thread.
struct Piece {
    const char* in;
    char* out;
    int len, dtype, esize;
    __device__ __forceinline__ int head() const {  // elements before a 16-byte boundary of in
        return min(len, (int)((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / esize);
    }
};

__device__ __forceinline__ Piece piece_of(const ClipEntry& e, int64_t c) {
    Piece p;
    p.dtype = e.dtype;
    p.esize = e.dtype == kF32 ? 4 : 2;
    const int64_t per = kClipChunk / p.esize, at = (c - e.first) * per;
    p.in = static_cast<const char*>(e.in) + at * p.esize;
    p.out = static_cast<char*>(e.out) + at * p.esize;
    p.len = (int)min64(per, e.count - at);
    return p;
}

__device__ __forceinline__ float load_one(const char* p, int dtype) {
    if (dtype == kF32) return *reinterpret_cast<const float*>(p);
    if (dtype == kF16) return __half2float(*reinterpret_cast<const __half*>(p));
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
}

// A thread's share of a chunk: kVecs 16-byte vectors, and one of the up to 2 * 8 - 1 elements
// before the first and behind the last of them.
constexpr int kVecs = kClipChunk / 16 / kThreads;
struct Share {
    uint4 v[kVecs];
    float edge;
};
__device__ __forceinline__ void fetch(const Piece& p, Share& s) {
    const int tid = threadIdx.x, head = p.head(), V = 16 / p.esize;
    const int nv = (p.len - head) / V, rest = p.len - nv * V;
    const uint4* q = reinterpret_cast<const uint4*>(p.in + head * p.esize);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kThreads + tid;
        s.v[u] = i < nv ? ld_v4(q + i) : make_uint4(0, 0, 0, 0);
    }
    s.edge = tid < rest ? load_one(p.in + (tid < head ? tid : nv * V + tid) * p.esize, p.dtype) : 0.f;
}

struct Sum {
    float f = 0.f;   // groups in the range where fp32 squares are safe
    double d = 0.0;  // the others
};

// One group: x[0 .. n) of a thread.
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

// The sum over the warp, in every lane: fp32 where all of it is there.
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
__device__ __forceinline__ void squares(const Share& h, Sum& s) {
    constexpr int V = Elt<T>::kVec;
    float x[kVecs * V];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) Elt<T>::unpack(h.v[u], x + u * V);
    add_group(x, s);
    if (h.edge != 0.f) {  // (NaN != 0)
        const float e[1] = {h.edge};
        add_group(e, s);
    }
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_norm_kernel(const ClipEntry* __restrict__ set, int tensors,
                                                             int64_t chunks, double* __restrict__ partial) {
    __shared__ double s_warp[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double total = 0.0;  // the warp's
    if (c0 < c1) {
        Sum s;
        int t = find_tensor(set, tensors, c0);
        int groups = 0;
        Share now, next;
        Piece p = piece_of(set[t], c0);
        fetch(p, now);
        for (int64_t c = c0; c < c1; ++c) {
            const int dtype = p.dtype;
            if (c + 1 < c1) {  // the next chunk's loads are under way while this one is summed
                while (t + 1 < tensors && set[t + 1].first <= c + 1) ++t;
                p = piece_of(set[t], c + 1);
                fetch(p, next);
            }
            if (dtype == kF32) squares<float>(now, s);
            else if (dtype == kF16) squares<__half>(now, s);
            else squares<__nv_bfloat16>(now, s);
            now = next;
            if (++groups == 4 || c + 1 == c1) {  // short fp32 runs: at most 4 groups and 4 single elements
                total += warp_sum(s);
                s = Sum();
                groups = 0;
            }
        }
    }
    if (lane == 0) s_warp[warp] = total;
    __syncthreads();
    if (warp == 0) {
        double x = lane < kWarps ? s_warp[lane] : 0.0;
#pragma unroll
        for (int d = kWarps / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane == 0) partial[blockIdx.x] = x;
    }
}

// sqrt of the sum of the partial sums in one order, by the calling warp (the same in every lane).
__device__ __forceinline__ double total_norm(const double* partial, int ctas) {
    double x = 0.0;
    for (int i = threadIdx.x & 31; i < ctas; i += 32) x += __ldcg(partial + i);  // written while this kernel was starting
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return sqrt(x);
}

__global__ void __launch_bounds__(32) grad_norm_finish_kernel(const double* __restrict__ partial, int ctas,
                                                              float* __restrict__ norm_out) {
    pdl_wait();
    const double norm = total_norm(partial, ctas);
    if (threadIdx.x == 0) *norm_out = (float)norm;
}

template <typename T>
__device__ __forceinline__ void store_scaled(const Piece& p, const Share& h, float c) {
    constexpr int V = Elt<T>::kVec;
    const int tid = threadIdx.x, head = p.head();
    const int nv = (p.len - head) / V, rest = p.len - nv * V;
    T* o = reinterpret_cast<T*>(p.out);
    if (tid < rest) o[tid < head ? tid : nv * V + tid] = Elt<T>::from_f(h.edge * c);
    o += head;
    const bool vec = (reinterpret_cast<uintptr_t>(o) & 15) == 0;  // out's boundaries are in's
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const int i = u * kThreads + tid;
        if (i < nv) {
            float x[V];
            Elt<T>::unpack(h.v[u], x);
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] *= c;
            if (vec) {
                __stcs(reinterpret_cast<uint4*>(o) + i, Elt<T>::pack(x));
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) o[(int64_t)i * V + k] = Elt<T>::from_f(x[k]);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_scale_kernel(const ClipEntry* __restrict__ set, int tensors,
                                                              int64_t chunks, const double* __restrict__ partial,
                                                              int ctas, double max_norm, int in_place,
                                                              float* __restrict__ norm_out) {
    __shared__ float s_c;
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    int t = c0 < c1 ? find_tensor(set, tensors, c1 - 1) : 0;
    pdl_wait();
    if (threadIdx.x < 32) {
        const double norm = total_norm(partial, ctas);
        if (threadIdx.x == 0) {
            const double q = max_norm / (norm + 1e-6);
            s_c = q >= 1.0 || isinf(max_norm) ? 1.f : (float)q;  // NaN stays NaN
            if (blockIdx.x == 0) *norm_out = (float)norm;
        }
    }
    __syncthreads();
    const float c = s_c;
    if (c == 1.f && in_place) return;  // every gradient already holds its value
    if (c0 >= c1) return;
    Share now, next;
    Piece p = piece_of(set[t], c1 - 1), q = p;
    fetch(p, now);
    for (int64_t k = c1 - 1; k >= c0; --k) {
        if (k > c0) {
            while (set[t].first > k - 1) --t;
            q = piece_of(set[t], k - 1);
            fetch(q, next);
        }
        if (p.dtype == kF32) store_scaled<float>(p, now, c);
        else if (p.dtype == kF16) store_scaled<__half>(p, now, c);
        else store_scaled<__nv_bfloat16>(p, now, c);
        now = next;
        p = q;
    }
}

}  // namespace

cudaError_t launch_grad_set_fill(ClipEntry* set, int64_t at, const ClipFill& f, int n, cudaStream_t s) {
    grad_set_fill_kernel<<<1, kClipFill, 0, s>>>(set + at, f, n);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_grad_norm(const ClipEntry* set, int32_t tensors, int64_t chunks, bool in_place, bool scale,
                             double max_norm, float* norm_out, double* partial, cudaStream_t s) {
    const int64_t want = (int64_t)device_props().sm_count * kCtasPerSm;
    const int ctas = (int)max64(1, min64(chunks, min64(want, kClipMaxCtas)));
    grad_norm_kernel<<<ctas, kThreads, 0, s>>>(set, tensors, chunks, partial);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (scale)
        e = launch_pdl(grad_scale_kernel, dim3(ctas), dim3(kThreads), 0, s, set, (int)tensors, chunks,
                       (const double*)partial, ctas, max_norm, (int)in_place, norm_out);
    else
        e = launch_pdl(grad_norm_finish_kernel, dim3(1), dim3(32), 0, s, (const double*)partial, ctas, norm_out);
    count_launches(2);
    return e;
}

}  // namespace spops
