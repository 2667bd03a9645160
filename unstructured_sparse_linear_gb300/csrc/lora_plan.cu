// The plan of a batch of tokens for the low-rank adapter operators: the tokens sorted by
// adapter, each adapter's range, and tiles of rows that share one adapter.
//
// One CTA: the sort is a stable LSD radix sort of the adapter ids (8-bit digits; one pass up
// to 255 adapters), in which warp w owns the positions [w L, (w + 1) L): per-warp digit counts
// with match masks, a prefix over digits and warps, and a scatter in the same order. Stable,
// so an adapter's tokens stay ascending (a request's rows stay consecutive) and the sums over
// them have one order. A batch is planned once and used by every projection of every layer, so
// the kernel is built for few dependent steps at decode sizes rather than for many tokens.
#include "common.cuh"
#include "internal.h"
#include "lora.h"

namespace spops {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kAhead = 4;  // ids loaded ahead per lane

// The sort key of token t: its adapter, n for none (any id outside [0, n)).
__device__ __forceinline__ int lora_key(const int32_t* ids, int t, int n) {
    if (!ids) return 0;
    const int a = ids[t];
    return (unsigned)a < (unsigned)n ? a : n;
}

// Exclusive prefix of x over the block, in thread order; *total: the sum.
__device__ __forceinline__ int block_exclusive(int x, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    __syncthreads();  // s_warp may still be read from an earlier call
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    *total = s_warp[31];
    return inc - x + (warp ? s_warp[warp - 1] : 0);
}

__device__ __forceinline__ void write_tile(LoraTile* out, const LoraPlanView& v, int adapter, int p0, int n) {
    const int t0 = v.order[p0];
    LoraTile t;
    t.adapter = adapter;
    t.pos0 = p0;
    t.rows = n;
    t.tok0 = v.order[p0 + n - 1] - t0 == n - 1 ? t0 : -1;  // ascending, so consecutive
    *out = t;
}
__device__ __forceinline__ void write_tile(LoraSmall* out, const LoraPlanView& v, int adapter, int p0, int n) {
    LoraSmall t;
    t.adapter = adapter;
    t.rows = n;
#pragma unroll
    for (int i = 0; i < kLoraRows; ++i) t.tok[i] = v.order[p0 + min(i, n - 1)];
    t.pad[0] = t.pad[1] = 0;
    *out = t;
}

// Tiles of at most `rows` rows for adapters 0 .. na - 1 of off; returns their number.
template <typename Tile>
__device__ int build_tiles(const LoraPlanView& v, int na, int rows, Tile* tiles, int* s_warp) {
    int carry = 0;
    for (int a0 = 0; a0 < na; a0 += kPlanThreads) {
        const int a = a0 + threadIdx.x;
        const int c = a < na ? (v.off[a + 1] - v.off[a] + rows - 1) / rows : 0;
        int total;
        const int before = block_exclusive(c, s_warp, &total);
        if (a < na) v.tstart[a] = carry + before;
        carry += total;
    }
    if (threadIdx.x == 0) v.tstart[na] = carry;
    __syncthreads();
    for (int i = threadIdx.x; i < carry; i += kPlanThreads) {
        int lo = 0, hi = na - 1;  // the last adapter whose first tile is <= i (empty ones share a start)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (v.tstart[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        const int p0 = v.off[lo] + (i - v.tstart[lo]) * rows;
        write_tile(tiles + i, v, lo < v.n ? lo : -1, p0, min(rows, v.off[lo + 1] - p0));
    }
    __syncthreads();
    return carry;
}

__global__ void __launch_bounds__(kPlanThreads, 1) lora_plan_kernel(const int32_t* __restrict__ ids, LoraPlanView v,
                                                                    int passes) {
    __shared__ int cnt[kPlanWarps][256];
    __shared__ int s_warp[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int T = v.tokens, n = v.n;
    const int L = ((T + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int64_t w0 = min64((int64_t)warp * L, T), w1 = min64(w0 + L, T);
    pdl_trigger();
    pdl_wait();

    for (int p = 0; p < passes; ++p) {
        const bool to_order = ((passes - 1 - p) & 1) == 0;
        const int32_t* src = to_order ? v.tmp : v.order;
        int32_t* dst = to_order ? v.order : v.tmp;
        const int shift = 8 * p;
        for (int i = tid; i < kPlanWarps * 256; i += kPlanThreads) (&cnt[0][0])[i] = 0;
        __syncthreads();
        // round 0 counts this warp's digits, round 1 scatters its positions in order
        for (int round = 0; round < 2; ++round) {
            for (int64_t b = w0; b < w1; b += 32 * kAhead) {
                int tok[kAhead], dig[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t i = b + u * 32 + lane;
                    tok[u] = i < w1 ? (p == 0 ? (int)i : src[i]) : -1;
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    dig[u] = tok[u] >= 0 ? (lora_key(ids, tok[u], n) >> shift) & 255 : 256;
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const unsigned same = __match_any_sync(0xffffffffu, dig[u]);
                    const int rank = __popc(same & ((1u << lane) - 1u));
                    int at = 0;
                    if (dig[u] < 256) at = cnt[warp][dig[u]];
                    __syncwarp();
                    if (dig[u] < 256 && rank == 0) cnt[warp][dig[u]] = at + __popc(same);
                    __syncwarp();
                    if (round == 1 && dig[u] < 256) dst[at + rank] = tok[u];
                }
            }
            __syncthreads();
            if (round == 0) {
                int sum = 0;
                if (tid < 256)
                    for (int w = 0; w < kPlanWarps; ++w) sum += cnt[w][tid];
                int total;
                int at = block_exclusive(tid < 256 ? sum : 0, s_warp, &total);
                if (tid < 256)
                    for (int w = 0; w < kPlanWarps; ++w) {
                        const int c = cnt[w][tid];
                        cnt[w][tid] = at;
                        at += c;
                    }
                __syncthreads();
            }
        }
    }

    // off[a]: the first position whose key is >= a
    for (int64_t i = tid; i <= T; i += kPlanThreads) {
        const int prev = i == 0 ? -1 : lora_key(ids, v.order[i - 1], n);
        const int key = i == T ? n + 1 : lora_key(ids, v.order[i], n);
        for (int a = prev + 1; a <= key; ++a) v.off[a] = (int)i;
    }
    __syncthreads();
    const int tiles = build_tiles(v, n, kLoraTile, v.tiles, s_warp);
    const int small = build_tiles(v, n + 1, kLoraRows, v.small, s_warp);
    // the adapters by falling number of tokens (a rank by comparing all pairs; as they are where
    // that would take long)
    for (int a = tid; a < n; a += kPlanThreads) {
        int at = a;
        if (n <= 1024) {
            const int c = v.off[a + 1] - v.off[a];
            at = 0;
            for (int b = 0; b < n; ++b) {
                const int d = v.off[b + 1] - v.off[b];
                at += d > c || (d == c && b < a);
            }
        }
        v.aorder[at] = a;
    }
    if (tid == 0) {
        v.counts[kLoraCntTiles] = tiles;
        v.counts[kLoraCntSmall] = small;
        v.counts[kLoraCntWith] = v.off[n];
    }
}

}  // namespace

cudaError_t launch_lora_plan(const int32_t* ids, const LoraPlanView& v, cudaStream_t s) {
    int passes = 1;
    while (passes < 4 && ((int64_t)v.n >> (8 * passes)) > 0) ++passes;  // keys 0 .. n
    const cudaError_t e = launch_pdl(lora_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, ids, v, passes);
    count_launches(1);
    return e;
}

}  // namespace spops
