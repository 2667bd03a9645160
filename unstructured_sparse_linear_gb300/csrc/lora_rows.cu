// General kernels of the low-rank adapter operators: any type, size and alignment, fp32
// arithmetic on the CUDA cores. They also serve small batches (single generated tokens).
//
// Products of one adapter's rows, P = U W1 (K -> rank) and O = base + s P W2 (rank -> N), with
// W1 = A^T, W2 = B^T forward and W1 = B, W2 = A for the input gradient. A thread-block cluster
// takes a tile of up to 8 rows of one adapter: every CTA multiplies a share of K, the partial
// P of all ranks are added through distributed shared memory in rank order (every rank forms
// the same sums, so results are deterministic and P never goes to global memory), and every
// CTA writes a share of the N columns. P stays in fp32 throughout; O is rounded once.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "lora.h"

namespace spops {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int R = kLoraRows;
constexpr int kJW = 4;  // ranks per warp task of the forward product

struct RowsArgs {
    LoraArgs a;
    LoraPlanView v;
    int vec;      // 16-byte loads of U and A/B rows along K (forward)
    int vec_r;    // 16-byte loads of B rows along rank (forward)
    int vec_copy;  // 16-byte accesses of base and O
};

// Elements [i, i + V) of p as floats; vec: one 16-byte load.
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
    Elt<T>::unpack(ld_v4(p), f);
}

// Forward dot products: part[ks][row][j] = sum over this CTA's and this warp's share of k of
// U[row, k] A[j, k]. Lanes along k; a warp takes kJW values of j and NR rows.
template <typename T, int NR, bool kVec>
__device__ __forceinline__ void dots_forward(const T* const* urow, const T* A, int64_t K, int64_t k0, int64_t k1,
                                             int j0, int rank, int ks, int ksplit, float (&acc)[kJW][NR]) {
    constexpr int V = kVec ? Elt<T>::kVec : 1;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < kJW; ++q)
#pragma unroll
        for (int i = 0; i < NR; ++i) acc[q][i] = 0.f;
    const T* arow[kJW];
#pragma unroll
    for (int q = 0; q < kJW; ++q) arow[q] = A + (int64_t)min(j0 + q, rank - 1) * K;
#pragma unroll 2
    for (int64_t k = k0 + (int64_t)(ks * 32 + lane) * V; k < k1; k += (int64_t)ksplit * 32 * V) {
        float w[kJW][V];
#pragma unroll
        for (int q = 0; q < kJW; ++q) {
            if constexpr (kVec) load_vec(arow[q] + k, w[q]);
            else w[q][0] = Elt<T>::to_f(arow[q][k]);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            float u[V];
            if constexpr (kVec) load_vec(urow[i] + k, u);
            else u[0] = Elt<T>::to_f(urow[i][k]);
#pragma unroll
            for (int q = 0; q < kJW; ++q)
#pragma unroll
                for (int e = 0; e < V; ++e) acc[q][i] = fmaf(w[q][e], u[e], acc[q][i]);
        }
    }
#pragma unroll
    for (int q = 0; q < kJW; ++q)
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int d = 16; d; d >>= 1) acc[q][i] += __shfl_xor_sync(0xffffffffu, acc[q][i], d);
}

template <typename T, int NR, bool kVec>
__device__ __forceinline__ void phase1_forward(const T* const* urow, const T* A, int64_t K, int64_t k0, int64_t k1,
                                               int rank, int ksplit, int rp, float* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int njg = (rank + kJW - 1) / kJW;
    const int ks = warp / (kWarps / ksplit);  // ksplit is 1, 2, 4 or 8
    const T* ur[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) ur[i] = urow[i];
    for (int jg = warp % (kWarps / ksplit); jg < njg; jg += kWarps / ksplit) {
        float acc[kJW][NR];
        dots_forward<T, NR, kVec>(ur, A, K, k0, k1, jg * kJW, rank, ks, ksplit, acc);
        if (lane == 0)
#pragma unroll
            for (int q = 0; q < kJW; ++q)
                if (jg * kJW + q < rank)
#pragma unroll
                    for (int i = 0; i < NR; ++i) part[((size_t)ks * R + i) * rp + jg * kJW + q] = acc[q][i];
    }
}

// Gradient direction: part[warp][row][j] = sum over k = this CTA's share, dealt to the warps,
// of U[row, k] B[k, j]. Lanes along j (rank is the contiguous axis of B); with rank <= 16 a
// warp takes 32 / jl rows of B at once.
template <typename T, int NR>
__device__ __forceinline__ void phase1_backward(const T* const* urow, const T* B, int64_t k0, int64_t k1,
                                                int rank, int rp, float* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int jl = 32;
    while (jl > 1 && (jl >> 1) >= rank) jl >>= 1;
    const int kl = 32 / jl, kq = lane / jl, j0 = lane & (jl - 1);
    for (int jb = 0; jb < rank; jb += 32) {
        const int j = jb + j0;
        float acc[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) acc[i] = 0.f;
        if (j < rank) {
#pragma unroll 2
            for (int64_t k = k0 + warp * kl + kq; k < k1; k += kWarps * kl) {
                const float w = Elt<T>::to_f(B[k * rank + j]);
#pragma unroll
                for (int i = 0; i < NR; ++i) acc[i] = fmaf(w, Elt<T>::to_f(urow[i][k]), acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            float x = acc[i];
            for (int d = 16; d >= jl; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
            if (lane < jl && j < rank) part[((size_t)warp * R + i) * rp + j] = x;
        }
    }
}

// barrier.cluster in two halves: what a CTA does between them overlaps the others' arrival.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The tile's P of one rank (rows 0 .. NR - 1), from shared memory.
template <int NR>
__device__ __forceinline__ void load_h(const float* p, float (&h)[NR]) {
    if constexpr (NR >= 4) {
#pragma unroll
        for (int i = 0; i < NR / 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(p)[i];
            h[4 * i] = v.x;
            h[4 * i + 1] = v.y;
            h[4 * i + 2] = v.z;
            h[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NR; ++i) h[i] = p[i];
    }
}

// Columns [n0, n1) of O = base (zeros) for the rows tok[0 .. rows), several loads under way.
template <typename T>
__device__ __forceinline__ void copy_rows(const RowsArgs& g, const int32_t* tok, int rows, int64_t n0, int64_t n1) {
    const T* base = static_cast<const T*>(g.a.base);
    T* O = static_cast<T*>(g.a.O);
    if (!O || (const T*)O == base || n1 <= n0) return;
    const int64_t ldo = g.a.ldo, ldb = g.a.ldb;
    if (g.vec_copy) {
        constexpr int V = Elt<T>::kVec;
        const int per = (int)((n1 - n0) / V), total = rows * per;
#pragma unroll 4
        for (int x = threadIdx.x; x < total; x += kThreads) {
            const int64_t t = tok[x / per], n = n0 + (int64_t)(x % per) * V;
            *reinterpret_cast<uint4*>(O + t * ldo + n) = base ? ld_v4(base + t * ldb + n) : make_uint4(0, 0, 0, 0);
        }
    } else {
        const int64_t per = n1 - n0, total = rows * per;
#pragma unroll 4
        for (int64_t x = threadIdx.x; x < total; x += kThreads) {
            const int64_t t = tok[x / per], n = n0 + x % per;
            O[t * ldo + n] = base ? base[t * ldb + n] : Elt<T>::from_f(0.f);
        }
    }
}

// Columns of O per thread at a time, kThreads apart. (64 tokens of 48 adapters, 4096 to 11008: 8.6 us; with
// one 10.3, four 9.0; two whose weights are loaded before P is formed 9.4.)
constexpr int kCols = 2;

// One tile of NR rows at most: this CTA's shares of K and of the columns.
template <typename T, bool kBack, int NR>
__device__ __forceinline__ void one_tile(const RowsArgs& g, const LoraSmall* tile, const LoraSmall& t, float* part,
                                         float (*hs)[R], int C, int crank, int ksplit, int rp, int64_t k0, int64_t k1,
                                         int64_t n0, int64_t n1) {
    constexpr int V = Elt<T>::kVec;
    const LoraArgs& a = g.a;
    const int tid = threadIdx.x, r = a.rank;
    const int64_t K = a.K, N = a.N;
    const T* A = static_cast<const T*>(a.A) + (int64_t)t.adapter * r * (kBack ? N : K);
    const T* B = static_cast<const T*>(a.B) + (int64_t)t.adapter * r * (kBack ? K : N);
    const T* base = static_cast<const T*>(a.base);
    T* O = static_cast<T*>(a.O);
    const T* urow[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) urow[i] = static_cast<const T*>(a.U) + (int64_t)t.tok[i] * a.ldu;

    const int64_t col = n0 + tid;
    const int64_t bstep = (int64_t)kThreads * r;
    const float s = a.scale_all * (a.scale ? a.scale[t.adapter] : 1.f);

    if constexpr (kBack) phase1_backward<T, NR>(urow, B, k0, k1, r, rp, part);
    else if (g.vec) phase1_forward<T, NR, true>(urow, A, K, k0, k1, r, ksplit, rp, part);
    else phase1_forward<T, NR, false>(urow, A, K, k0, k1, r, ksplit, rp, part);
    if (C > 1) {
        cluster_release_smem();
        cluster_sync_relaxed();
    } else {
        __syncthreads();
    }
    for (int x = tid; x < t.rows * r; x += kThreads) {
        const int i = x / r, j = x - i * r;
        // in the order of (share of K, rank), eight loads under way at a time
        float sum = 0.f;
        for (int ks = 0; ks < ksplit; ++ks) {
            const float* p = part + ((size_t)ks * R + i) * rp + j;
            if (C > 1) {
                const uint32_t at = smem_u32(p);
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = q < C ? __uint_as_float(ld_cluster_u32(cluster_map(at, q))) : 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q) sum += v[q];
            } else {
                sum += *p;
            }
        }
        hs[j][i] = sum * s;
        if (a.P && crank == 0 && blockIdx.y == 0) a.P[(int64_t)tile->tok[i] * r + j] = sum;
    }
    // Every rank has read the partial sums once all have passed the wait below (they are rewritten
    // by the next tile, and no CTA leaves while another still reads its shared memory).
    if (C > 1) {
        cluster_release_smem();
        cluster_arrive_relaxed();
    }
    __syncthreads();
    if (O)
        for (int64_t n = col; n - tid < n1; n += kCols * kThreads) {
            float acc[kCols][NR];
            T bv[kCols][NR];  // base: on its way while the sums are formed, added last
            bool in[kCols];
#pragma unroll
            for (int q = 0; q < kCols; ++q) {
                in[q] = n + q * kThreads < n1;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    acc[q][i] = 0.f;
                    bv[q][i] = Elt<T>::from_f(0.f);
                    if (base && in[q]) bv[q][i] = base[(int64_t)t.tok[i] * a.ldb + n + q * kThreads];
                }
            }
            auto step = [&](int j, const float (&w)[kCols]) {
                float h[NR];
                load_h<NR>(hs[j], h);
#pragma unroll
                for (int q = 0; q < kCols; ++q)
#pragma unroll
                    for (int i = 0; i < NR; ++i) acc[q][i] = fmaf(w[q], h[i], acc[q][i]);
            };
            if constexpr (kBack) {
#pragma unroll 4
                for (int j = 0; j < r; ++j) {
                    float w[kCols];
#pragma unroll
                    for (int q = 0; q < kCols; ++q) w[q] = in[q] ? Elt<T>::to_f(A[(int64_t)j * N + n + q * kThreads]) : 0.f;
                    step(j, w);
                }
            } else if (g.vec_r) {
                auto steps = [&](int j, const uint4 (&v)[kCols]) {
                    float f[kCols][V];
#pragma unroll
                    for (int q = 0; q < kCols; ++q) Elt<T>::unpack(v[q], f[q]);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float w[kCols];
#pragma unroll
                        for (int q = 0; q < kCols; ++q) w[q] = f[q][e];
                        step(j + e, w);
                    }
                };
                const T* b = B + n * r;
#pragma unroll 2
                for (int j = 0; j < r; j += V) {
                    uint4 v[kCols];
#pragma unroll
                    for (int q = 0; q < kCols; ++q) v[q] = in[q] ? ld_v4(b + q * bstep + j) : make_uint4(0, 0, 0, 0);
                    steps(j, v);
                }
            } else {
                const T* b = B + n * r;
#pragma unroll 4
                for (int j = 0; j < r; ++j) {
                    float w[kCols];
#pragma unroll
                    for (int q = 0; q < kCols; ++q) w[q] = in[q] ? Elt<T>::to_f(b[q * bstep + j]) : 0.f;
                    step(j, w);
                }
            }
#pragma unroll
            for (int q = 0; q < kCols; ++q)
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    if (in[q] && i < t.rows)
                        O[(int64_t)t.tok[i] * a.ldo + n + q * kThreads] = Elt<T>::from_f(Elt<T>::to_f(bv[q][i]) + acc[q][i]);
        }
    if (C > 1) cluster_wait();
}

template <typename T, bool kBack>
__global__ void __launch_bounds__(kThreads, 2) lora_rows_kernel(const RowsArgs g) {
    extern __shared__ __align__(16) float part[];  // [ksplit][R][rp]
    __shared__ __align__(16) float hs[kLoraMaxRank][R];
    const LoraArgs& a = g.a;
    const int tid = threadIdx.x;
    const int C = (int)cluster_size(), crank = (int)cluster_rank();
    // With few tiles several clusters (gridDim.y) take one: each forms P, and a share of the columns.
    const int cid = blockIdx.x / C, ncl = gridDim.x / C;
    pdl_wait();
    // Backward: the weight gradients' kernel begins beside this one, and relies on all before it being
    // complete, so the trigger is behind the wait. Forward: the next call's CTAs come as this one's
    // leave (waiting beside them they cost 1.5 us of then 11.5: 64 tokens of 48 adapters, 4096 to 11008).
    if (kBack) pdl_trigger();
    // (the list has a slot for every cluster; what lies behind its end is not used)
    LoraSmall t = g.v.small[cid];
    const int ntiles = g.v.counts[kLoraCntSmall];
    const int r = a.rank;
    const int njg = (r + kJW - 1) / kJW;
    const int ksplit = kBack ? kWarps : (njg >= kWarps ? 1 : kWarps / njg);
    const int rp = (r + 3) & ~3;
    // shares of K and of the columns in units of 8 elements (C is a power of two)
    const int clog = 31 - __clz(C);
    const int64_t ku = (a.K + 7) / 8, nu = (a.N + 7) / 8;
    const int64_t k0 = (ku * crank >> clog) * 8, k1 = min64(a.K, (ku * (crank + 1) >> clog) * 8);
    const int share = blockIdx.y * C + crank, slog = clog + 31 - __clz(gridDim.y);  // (powers of two both)
    const int64_t n0 = (nu * share >> slog) * 8, n1 = min64(a.N, (nu * (share + 1) >> slog) * 8);

    // The trip count and every barrier are the same on all CTAs of a cluster.
    for (int it = cid; it < ntiles; it += ncl) {
        if (it != cid) {
            t = g.v.small[it];
            __syncthreads();  // the previous tile's P has been read
        }
        if (t.adapter < 0) {  // no adapter: O = base, P = 0
            copy_rows<T>(g, g.v.small[it].tok, t.rows, n0, n1);
            if (a.P && share == 0)
                for (int x = tid; x < t.rows * r; x += kThreads)
                    a.P[(int64_t)g.v.small[it].tok[x / r] * r + x % r] = 0.f;
        } else if (t.rows == 1) {
            one_tile<T, kBack, 1>(g, g.v.small + it, t, part, hs, C, crank, ksplit, rp, k0, k1, n0, n1);
        } else if (t.rows == 2) {
            one_tile<T, kBack, 2>(g, g.v.small + it, t, part, hs, C, crank, ksplit, rp, k0, k1, n0, n1);
        } else if (t.rows <= 4) {
            one_tile<T, kBack, 4>(g, g.v.small + it, t, part, hs, C, crank, ksplit, rp, k0, k1, n0, n1);
        } else {
            one_tile<T, kBack, 8>(g, g.v.small + it, t, part, hs, C, crank, ksplit, rp, k0, k1, n0, n1);
        }
    }
}

// ------------------------------------------------------------------ weight gradients

constexpr int kWgJ = 16;   // ranks per CTA
constexpr int kWgT = 32;   // tokens staged at a time

struct WgradRowsArgs {
    LoraWgradArgs w[2];
    int blocks[2];  // column blocks of each product
    int nw, jb;     // products, rank blocks
    int32_t rank;
    const float* scale;
    float scale_all;
    LoraPlanView v;
};

// One cluster: 256 columns x 16 ranks of one adapter's gradient; its CTAs split the adapter's
// tokens and the partial sums are added in rank order through distributed shared memory. A
// thread owns a column: U is read coalesced, P is broadcast from shared memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) lora_wgrad_rows_kernel(const WgradRowsArgs g) {
    __shared__ __align__(16) float s_p[kWgT][kWgJ];
    __shared__ int s_tok[kWgT];
    __shared__ float s_acc[kWgJ][kThreads];
    const int tid = threadIdx.x;
    const int C = (int)cluster_size(), crank = (int)cluster_rank();
    const int per = (g.blocks[0] + (g.nw > 1 ? g.blocks[1] : 0)) * g.jb;
    const int64_t item = blockIdx.x / C;
    const int adapter = (int)(item / per);
    int x = (int)(item - (int64_t)adapter * per);
    const int j0 = x % g.jb * kWgJ;
    x /= g.jb;
    const int which = x >= g.blocks[0];
    const LoraWgradArgs& w = g.w[which];
    const int64_t n = (int64_t)(x - (which ? g.blocks[0] : 0)) * kThreads + tid;
    const int r = g.rank;
    pdl_trigger();
    pdl_wait();
    const int p0 = g.v.off[adapter], cnt = g.v.off[adapter + 1] - p0;
    const int b0 = p0 + (int)((int64_t)cnt * crank / C), b1 = p0 + (int)((int64_t)cnt * (crank + 1) / C);
    const T* U = static_cast<const T*>(w.U);
    float acc[kWgJ];
#pragma unroll
    for (int j = 0; j < kWgJ; ++j) acc[j] = 0.f;
    for (int b = b0; b < b1; b += kWgT) {
        const int m = min(kWgT, b1 - b);
        __syncthreads();
        if (tid < m) s_tok[tid] = g.v.order[b + tid];
        __syncthreads();
        for (int i = tid; i < kWgT * kWgJ; i += kThreads) {
            const int q = i / kWgJ, j = i % kWgJ;
            s_p[q][j] = q < m && j0 + j < r ? w.P[(int64_t)s_tok[q] * r + j0 + j] : 0.f;
        }
        __syncthreads();
        if (n < w.N) {
#pragma unroll 4
            for (int q = 0; q < m; ++q) {
                const float u = Elt<T>::to_f(U[(int64_t)s_tok[q] * w.ldu + n]);
#pragma unroll
                for (int j = 0; j < kWgJ; ++j) acc[j] = fmaf(u, s_p[q][j], acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kWgJ; ++j) s_acc[j][tid] = acc[j];
    if (C > 1) {
        cluster_release_smem();
        cluster_sync_relaxed();
    } else {
        __syncthreads();
    }
    const float s = g.scale_all * (g.scale ? g.scale[adapter] : 1.f);
    T* G = static_cast<T*>(w.G) + (int64_t)adapter * r * w.N;
    if (n < w.N)
        for (int j = crank; j < kWgJ && j0 + j < r; j += C) {
            float sum = 0.f;
            for (int q = 0; q < C; ++q)
                sum += C > 1 ? __uint_as_float(ld_cluster_u32(cluster_map(smem_u32(&s_acc[j][tid]), q))) : s_acc[j][tid];
            const T y = Elt<T>::from_f(sum * s);
            if (w.rank_minor) G[n * r + j0 + j] = y;
            else G[(int64_t)(j0 + j) * w.N + n] = y;
        }
    if (C > 1) cluster_sync_relaxed();  // nobody reads this CTA's sums any more
}

// Cluster size for `items` clusters: CTAs for at most two per SM at once (384 tokens of one adapter
// in clusters of 8 are two waves, 14.2 us; 10.9 us in clusters of 4), at most 8 (the portable limit).
int pick_cluster(int64_t items, int64_t most) {
    const int64_t want = 2 * (int64_t)device_props().sm_count;
    int c = 1;
    while (c < 8 && items * c * 2 <= want && c * 2 <= most) c *= 2;
    return c;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), int64_t clusters, int c, int split, size_t smem, cudaStream_t s,
                           Args&&... args) {
    const cudaError_t e = launch_pdl_cluster(kern, dim3((unsigned)(clusters * c), (unsigned)split), dim3(kThreads), smem,
                                             (unsigned)c, s, std::forward<Args>(args)...);
    count_launches(1);
    return e;
}

template <typename T>
cudaError_t run_rows(bool back, const LoraArgs& a, const LoraPlanView& v, cudaStream_t s) {
    RowsArgs g;
    g.a = a;
    g.v = v;
    constexpr int V = Elt<T>::kVec;
    g.vec = a.K % V == 0 && a.ldu % V == 0 && ((uintptr_t)a.U | (uintptr_t)a.A) % 16 == 0;
    g.vec_r = a.rank % V == 0 && (uintptr_t)a.B % 16 == 0;
    g.vec_copy = a.N % 8 == 0 && a.ldo % V == 0 && a.ldb % V == 0 && ((uintptr_t)a.O | (uintptr_t)a.base) % 16 == 0;
    const int64_t cap = lora_tiles_cap(v.tokens, v.n, kLoraRows);
    // the tiles to expect: cap is reached only where every adapter has a token and a last tile of its
    // own; tokens that pick adapters at random use about 0.6 of them when they are as many
    const int64_t expected = v.tokens / R + (6 * min64(v.tokens, v.n) + 9) / 10;
    const int c = pick_cluster(expected, max64(1, max64(a.K, a.N) / 64));
    const int64_t clusters = min64(cap, (int64_t)device_props().sm_count * 8);
    // Few tiles: a tile's columns are shared by several clusters while there is an SM for every CTA and
    // 8192 products of a column and a rank are left to each. (16 tokens of one adapter, rank 64, 2048 to
    // 8192: 15.0 us with one cluster of 8 per tile, 10.3 us so; 64 tokens of 48 adapters, rank 16, 4096 to
    // 4096, which this leaves alone: 8.4 us, with two clusters a tile 12.5.)
    int split = 1;
    if (a.O)
        while (split < 16 && expected * c * split * 2 <= (int64_t)device_props().sm_count &&
               (int64_t)c * split * 2 * 8192 <= (int64_t)a.N * a.rank)
            split *= 2;
    const int rp = (a.rank + 3) & ~3, njg = (a.rank + kJW - 1) / kJW;
    const int ksplit = back ? kWarps : (njg >= kWarps ? 1 : kWarps / njg);
    const size_t smem = (size_t)ksplit * R * rp * sizeof(float);  // at most 32 KB
    return back ? launch_cluster(lora_rows_kernel<T, true>, clusters, c, split, smem, s, g)
                : launch_cluster(lora_rows_kernel<T, false>, clusters, c, split, smem, s, g);
}

template <typename T>
cudaError_t run_wgrad_rows(const LoraWgradArgs* w, int nw, int32_t rank, const float* scale, float scale_all,
                           const LoraPlanView& v, cudaStream_t s) {
    WgradRowsArgs g;
    g.nw = nw;
    g.jb = (rank + kWgJ - 1) / kWgJ;
    g.blocks[0] = g.blocks[1] = 0;
    for (int i = 0; i < nw; ++i) {
        g.w[i] = w[i];
        g.blocks[i] = (w[i].N + kThreads - 1) / kThreads;
    }
    g.rank = rank;
    g.scale = scale;
    g.scale_all = scale_all;
    g.v = v;
    const int64_t items = (int64_t)v.n * (g.blocks[0] + g.blocks[1]) * g.jb;
    const int c = pick_cluster(items, max64(1, v.tokens / kWgT));
    if (items * c > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_cluster(lora_wgrad_rows_kernel<T>, items, c, 1, 0, s, g);
}

}  // namespace

cudaError_t launch_lora_rows(int dt, bool back, const LoraArgs& a, const LoraPlanView& v, cudaStream_t s) {
    if (dt == kF32) return run_rows<float>(back, a, v, s);
    if (dt == kF16) return run_rows<__half>(back, a, v, s);
    return run_rows<__nv_bfloat16>(back, a, v, s);
}

cudaError_t launch_lora_wgrad_rows(int dt, const LoraWgradArgs* w, int nw, int32_t rank, const float* scale,
                                   float scale_all, const LoraPlanView& v, cudaStream_t s) {
    if (dt == kF32) return run_wgrad_rows<float>(w, nw, rank, scale, scale_all, v, s);
    if (dt == kF16) return run_wgrad_rows<__half>(w, nw, rank, scale, scale_all, v, s);
    return run_wgrad_rows<__nv_bfloat16>(w, nw, rank, scale, scale_all, v, s);
}

// Which kernels: the general one multiplies T r (K + N) times on the CUDA cores and reads an
// adapter's weights for every 8 rows, the tensor-core one has about 13 us of latency (two phases
// with an exchange between them) and reads the weights for every 128 rows, so for every adapter of
// a mixed batch. Measured (bf16, us, general : tensor cores; adapters picked at random):
//   forward, 4096 -> 4096, rank 16: 512 tokens of one adapter 10.8 : 12.6, 1024 16.5 : 12.8; of 8
//   1024 tokens 16.6 : 28.2, 1536 27.7 : 28.4, 2048 27.9 : 30.7; of 48 1024 19.5 : 30.6, 2048 28.3 : 37.3; 2048 ->
//   8192, rank 64: 96 tokens of one adapter 14.2 : 22.5, 128 22.8 : 22.3; of 8 256 24.4 : 25.4, 384 37.3 :
//   28.3; of 48 384 39.5 : 49.7, 512 67.4 : 50.0;
//   input gradient (whose general form reads B element by element): rank 16, 256 tokens of one adapter
//   13.0 : 13.2, 384 19.9 : 13.3; of 8 256 14 : 17.2, 384 20.0 : 19.8; of 48 256 19.5 : 28.3, 384 32.2 :
//   29.4; rank 64, 16 tokens 45 : 19.5.
// An adapter's tokens in runs, which a plan's sizes do not tell, leave the general kernel's times as they are; the
// tensor cores then take 15.2 for 8 adapters' 1024 tokens, 16.2 for 1536, 17.5 for 2048, and 27.0 for 2048 of 48. The
// forward rule lies between the two: past it scattered tokens take up to 9 us more than they could, runs 11 less.
static bool general_is_faster(bool back, const LoraArgs& a, const LoraPlanView& v) {
    const int64_t work = (int64_t)v.tokens * a.rank;
    if (back) return a.rank <= 32 && work <= 4096 + 192 * min64(v.n, 8);
    return work <= 9216 + 960 * min64(v.n, 22);
}

cudaError_t launch_lora(int dt, bool back, const LoraArgs& a, const LoraPlanView& v, cudaStream_t s) {
    if (lora_tiles_ok(dt, a, v) && !general_is_faster(back, a, v)) return launch_lora_tiles(dt, back, a, v, s);
    return launch_lora_rows(dt, back, a, v, s);
}

cudaError_t launch_lora_wgrad(int dt, const LoraWgradArgs* w, int nw, int32_t rank, const float* scale,
                              float scale_all, const LoraPlanView& v, bool after_lora, cudaStream_t s) {
    if (v.tokens > 16 && lora_wgrad_tiles_ok(dt, w, nw))  // (16 tokens: 5 to 9 us either way)
        return launch_lora_wgrad_tiles(dt, w, nw, rank, scale, scale_all, v, after_lora, s);
    return launch_lora_wgrad_rows(dt, w, nw, rank, scale, scale_all, v, s);
}

}  // namespace spops
