// Gradient clipping by the global 2-norm of many tensors:
//     norm = sqrt(sum of g^2 over every gradient),  c = min(1, max_norm / (norm + 1e-6)),
//     out = c g (rounded once to the gradient's type).
// Two launches whatever the number of tensors: the table of the set lies in device memory,
// with every tensor cut into chunks of 8192 elements; the chunks are dealt to the CTAs in
// contiguous, equal ranges, so the sums have one order (no atomics) and a CTA looks its first
// tensor up once. The second kernel adds the CTAs' partial sums itself, in one order, and walks
// its range backwards: the part of the set that the first pass read last is still in L2.
//
// Squares are added in fp32 within a thread's 16 to 32 elements of a chunk, then in fp64. A
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

__global__ void grad_set_fill_kernel(ClipEntry* set, const __grid_constant__ ClipFill f, int n) {
    const int i = threadIdx.x;
    if (i < n) set[i] = f.e[i];
}

// The sum over the block in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double x, double* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += s_warp[w];
    return t;
}

// The tensor that chunk c belongs to (tensors without elements share their first chunk with
// the next one; the last tensor with first <= c is the owner).
__device__ __forceinline__ int find_tensor(const ClipEntry* set, int tensors, int64_t c) {
    int lo = 0, hi = tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (set[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Leading elements of p before a 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p) {
    return (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
}

struct Sum {
    float f = 0.f;   // groups in the range where fp32 squares are safe
    double d = 0.0;  // the rest, and f so far
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

template <typename T>
__device__ __forceinline__ void chunk_squares(const T* p, int len, Sum& s) {
    constexpr int V = Elt<T>::kVec;
    constexpr int U = kClipChunk / V / kThreads;  // vectors per thread of a whole chunk
    const int tid = threadIdx.x;
    const int head = min(len, head_of(p));
    const int nv = (len - head) / V;
    const uint4* q = reinterpret_cast<const uint4*>(p + head);
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + tid;
        v[u] = i < nv ? ld_nc_v4(q + i) : make_uint4(0, 0, 0, 0);
    }
    const int rest = len - nv * V;  // head and tail: at most 14 elements
    float e[1] = {0.f};
    if (tid < rest) e[0] = Elt<T>::to_f(p[tid < head ? tid : nv * V + tid]);
    float x[U * V];
#pragma unroll
    for (int u = 0; u < U; ++u) Elt<T>::unpack(v[u], x + u * V);
    add_group(x, s);
    if (tid < rest) add_group(e, s);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const ClipEntry* __restrict__ set, int tensors,
                                                             int64_t chunks, double* __restrict__ partial) {
    __shared__ double s_warp[kWarps];
    pdl_trigger();
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    Sum s;
    if (c0 < c1) {
        int t = find_tensor(set, tensors, c0);
        int groups = 0;
        for (int64_t c = c0; c < c1; ++c) {
            while (t + 1 < tensors && set[t + 1].first <= c) ++t;
            const ClipEntry e = set[t];
            const int64_t at = (c - e.first) * kClipChunk;
            const int len = (int)min64(kClipChunk, e.count - at);
            if (e.dtype == kF32) chunk_squares(static_cast<const float*>(e.in) + at, len, s);
            else if (e.dtype == kF16) chunk_squares(static_cast<const __half*>(e.in) + at, len, s);
            else chunk_squares(static_cast<const __nv_bfloat16*>(e.in) + at, len, s);
            if (++groups == 8) {  // short fp32 runs: at most 8 groups and 8 single elements
                s.d += (double)s.f;
                s.f = 0.f;
                groups = 0;
            }
        }
    }
    const double total = block_sum(s.d + (double)s.f, s_warp);
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

// sqrt of the sum of the partial sums, the same in every thread of every CTA.
__device__ __forceinline__ double total_norm(const double* partial, int ctas, double* s_warp) {
    double x = 0.0;
    for (int i = threadIdx.x; i < ctas; i += kThreads) x += __ldcg(partial + i);  // written while this kernel was starting
    return sqrt(block_sum(x, s_warp));
}

__global__ void __launch_bounds__(kThreads) grad_norm_finish_kernel(const double* __restrict__ partial, int ctas,
                                                                    float* __restrict__ norm_out) {
    __shared__ double s_warp[kWarps];
    pdl_wait();
    const double norm = total_norm(partial, ctas, s_warp);
    if (threadIdx.x == 0) *norm_out = (float)norm;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* o, int len, float c) {
    constexpr int V = Elt<T>::kVec;
    constexpr int U = kClipChunk / V / kThreads;
    const int tid = threadIdx.x;
    const int head = min(len, head_of(p));
    if (head_of(o) != head_of(p)) {  // the two sides' 16-byte boundaries differ
        for (int i = tid; i < len; i += kThreads) o[i] = Elt<T>::from_f(Elt<T>::to_f(p[i]) * c);
        return;
    }
    const int nv = (len - head) / V;
    const uint4* q = reinterpret_cast<const uint4*>(p + head);
    uint4* w = reinterpret_cast<uint4*>(o + head);
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + tid;
        if (i < nv) v[u] = ld_v4(q + i);
    }
    const int rest = len - nv * V;
    if (tid < rest) {
        const int i = tid < head ? tid : nv * V + tid;
        o[i] = Elt<T>::from_f(Elt<T>::to_f(p[i]) * c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + tid;
        if (i < nv) {
            float x[V];
            Elt<T>::unpack(v[u], x);
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] *= c;
            w[i] = Elt<T>::pack(x);
        }
    }
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const ClipEntry* __restrict__ set, int tensors,
                                                              int64_t chunks, const double* __restrict__ partial,
                                                              int ctas, double max_norm, int in_place,
                                                              float* __restrict__ norm_out) {
    __shared__ double s_warp[kWarps];
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    int t = c0 < c1 ? find_tensor(set, tensors, c1 - 1) : 0;
    pdl_wait();
    const double norm = total_norm(partial, ctas, s_warp);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    const double q = max_norm / (norm + 1e-6);
    const float c = q >= 1.0 || isinf(max_norm) ? 1.f : (float)q;  // NaN stays NaN
    if (c == 1.f && in_place) return;  // every gradient already holds its value
    for (int64_t k = c1 - 1; k >= c0; --k) {
        while (set[t].first > k) --t;
        const ClipEntry e = set[t];
        const int64_t at = (k - e.first) * kClipChunk;
        const int len = (int)min64(kClipChunk, e.count - at);
        if (e.dtype == kF32) chunk_scale(static_cast<const float*>(e.in) + at, static_cast<float*>(e.out) + at, len, c);
        else if (e.dtype == kF16)
            chunk_scale(static_cast<const __half*>(e.in) + at, static_cast<__half*>(e.out) + at, len, c);
        else
            chunk_scale(static_cast<const __nv_bfloat16*>(e.in) + at, static_cast<__nv_bfloat16*>(e.out) + at, len, c);
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
    const int64_t want = (int64_t)device_props().sm_count * 4;
    const int ctas = (int)max64(1, min64(chunks, min64(want, kClipMaxCtas)));
    grad_norm_kernel<<<ctas, kThreads, 0, s>>>(set, tensors, chunks, partial);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (scale)
        e = launch_pdl(grad_scale_kernel, dim3(ctas), dim3(kThreads), 0, s, set, (int)tensors, chunks,
                       (const double*)partial, ctas, max_norm, (int)in_place, norm_out);
    else
        e = launch_pdl(grad_norm_finish_kernel, dim3(1), dim3(kThreads), 0, s, (const double*)partial, ctas, norm_out);
    count_launches(2);
    return e;
}

}  // namespace spops
