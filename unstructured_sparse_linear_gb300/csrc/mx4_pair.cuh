// What the tensor-core products with a 4-bit weight share (mx4_fwd.cu, mx4_back.cu): CTA pairs, their messages, the way out of
// the accumulators, and the host's side.
#pragma once

#include <type_traits>

#include "internal.h"
#include "mx4.cuh"
#include "mx4.h"
#include "pipeline.cuh"

namespace spops {
namespace {

constexpr int kKC = 64;          // contraction elements of a 128-byte row of X
constexpr int kFeatures = 128;   // of a CTA
constexpr int kMaxTokens = 256;  // of a tile
constexpr int kOutTokens = 32;   // of a store: 32 x 32 values

// ------------------------------------------------------------------ PTX of CTA pairs

__device__ __forceinline__ void pair_alloc(uint32_t smem_dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A B^T over both CTAs of the pair, issued by a thread of the even one.
__device__ __forceinline__ void pair_mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the barrier at this address in the CTAs of `mask` once all products issued so far are complete.
__device__ __forceinline__ void pair_commit(uint32_t bar, uint32_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)mask)
        : "memory");
}
// A box of a 2-D tensor into this CTA's shared memory; its bytes are counted on a barrier of the pair (cluster address).
__device__ __forceinline__ void pair_tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Arrive on a barrier of the pair (its cluster address). What it announces is read by this CTA's tensor core, for which
// each writer's proxy fence has made it visible, or lies in TMEM or has left it, which the fences of tcgen05 order: no release of
// the cluster's scope, which took a warp 500 cycles for each stage.
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// What the pair wrote to its shared memory before the messages that were waited for.
__device__ __forceinline__ void acquire_pair_smem() {
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

struct TileArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    void* Y;
    int64_t ldy;
    int64_t blocks;  // of a row of W
    int32_t rows, F, tokens, ftiles, tiles, chunks, nt, stages;
    int32_t part;    // columns of one of the parts of X
    int32_t groups;  // of decoders
    int32_t bufs;    // accumulators
    uint32_t idesc;
    int* err;
};

// A tile's place: 256 features x nt tokens; the tiles of the same tokens follow each other.
struct Place {
    int f0, t0;
};
__device__ __forceinline__ Place place_of(const TileArgs& g, int tile, int half) {
    const int tt = tile / g.ftiles;
    return {(tile - tt * g.ftiles) * (2 * kFeatures) + half * kFeatures, tt * g.nt};
}

// A cluster is one pair, or S pairs that split a tile's contraction; in the second case (one tile per cluster) the fp32
// partial sums meet in shared memory and are added in the order of the splits.
struct Share {
    int half, lead, split, splits;
    int cid, ncl;         // the cluster and their number
    int c0, c1, per;      // this pair's stages of a tile
    int mine;             // tiles of this cluster
    __device__ explicit Share(const TileArgs& g) {
        const int C = (int)cluster_size(), crank = (int)cluster_rank();
        half = crank & 1;
        lead = crank & ~1;
        split = crank >> 1;
        splits = C >> 1;
        cid = (int)(blockIdx.x / (unsigned)C);
        ncl = (int)(gridDim.x / (unsigned)C);
        c0 = (int)((int64_t)g.chunks * split / splits);
        c1 = (int)((int64_t)g.chunks * (split + 1) / splits);
        per = c1 - c0;
        mine = cid < g.tiles && per > 0 ? (g.tiles - cid - 1) / ncl + 1 : 0;
    }
};

// Waits of a pair. What the barriers announce is read by the tensor core and by TMA or lies in TMEM, so no wait makes
// the thread's own loads see another CTA's memory: an acquire of the cluster's scope empties the SM's L1 each time
// (with other steps' help, 8192 tokens, 2048 -> 8192 203 us with it and 197 without).
struct PairWaits {
    volatile int* failed;
    int* err;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
            "mov.u32 n, 256;\n"
            "AGAIN_%=:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "@p bra DONE_%=;\n\t"
            "sub.u32 n, n, 1;\n\t"
            "setp.ne.u32 q, n, 0;\n\t"
            "@q bra AGAIN_%=;\n"
            "DONE_%=:\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "n"(kMbarPollNs)
            : "memory");
        return done || Waits{failed, err}(bar, parity);  // (with the time limit)
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// 32 fp32 TMEM columns of 32 lanes as 8 x 8 matrices, four a register pair: of registers 4 j and 4 j + 1 (+ 2: eight lanes on)
// a thread has columns 8 j + 2 (lane % 4) and the next, of lane `lane` / 4 (hi: 16 lanes on).
__device__ __forceinline__ void tmem_load_matrices(uint32_t taddr, uint32_t (&lo)[16], uint32_t (&hi)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(lo[0]), "=r"(lo[1]), "=r"(lo[2]), "=r"(lo[3]), "=r"(lo[4]), "=r"(lo[5]), "=r"(lo[6]), "=r"(lo[7]), "=r"(lo[8]),
          "=r"(lo[9]), "=r"(lo[10]), "=r"(lo[11]), "=r"(lo[12]), "=r"(lo[13]), "=r"(lo[14]), "=r"(lo[15]), "=r"(hi[0]),
          "=r"(hi[1]), "=r"(hi[2]), "=r"(hi[3]), "=r"(hi[4]), "=r"(hi[5]), "=r"(hi[6]), "=r"(hi[7]), "=r"(hi[8]), "=r"(hi[9]),
          "=r"(hi[10]), "=r"(hi[11]), "=r"(hi[12]), "=r"(hi[13]), "=r"(hi[14]), "=r"(hi[15])
        : "r"(taddr), "r"(taddr + (16u << 16))
        : "memory");
}
__device__ __forceinline__ void st_matrices_trans(uint32_t row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
template <typename Out>
__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b) {
    return Elt<Out>::p2(__uint_as_float(a), __uint_as_float(b));
}

// 32 tokens' sums of a lane. fp32 has two accumulators, the first part's and, nt columns on, the other two's: the tensor core
// cuts a sum off where it adds to it, and so the small parts' products cost the large ones' sum nothing.
template <typename Out>
__device__ __forceinline__ void load_sums(uint32_t from, int nt, float (&y)[32]) {
    tmem_load<32>(from, y);
    if constexpr (sizeof(Out) == 4) {
        float z[32];
        tmem_load<32>(from + (uint32_t)nt, z);
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] += z[e];
    }
}

// Warps 0 to 3, a TMEM lane quarter each: the tiles' sums to Y, by way of shared memory (kOutBufs buffers a warp at out_at), or to
// the place of the partial sums ([token][128 features], fp32).
template <typename Out, int kOutBufs>
__device__ __forceinline__ void finish_tiles(const TileArgs& g, const Share& me, const CUtensorMap& map_y, const PairWaits& wait,
                                             uint64_t* acc_full, uint64_t* acc_empty, uint32_t sbase, uint32_t out_at,
                                             uint32_t tmem, int buf_cols, int warp, int lane) {
    constexpr uint32_t kOutBytes = kOutTokens * 32 * sizeof(Out);
    uint32_t stores = 0, ph = 0;
    int buf = 0;
    for (int i = 0; i < me.mine; ++i) {
        const Place at = place_of(g, me.cid + i * me.ncl, me.half);
        const bool ok = wait(smem_u32(&acc_full[buf]), ph);
        const bool all = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
        const int f = at.f0 + warp * 32;
        const int live = min(g.nt, g.tokens - at.t0);
        if (all)
            for (int c = 0; c < live; c += kOutTokens) {
                const uint32_t from = tmem + ((uint32_t)warp << 21) + (uint32_t)(buf * buf_cols + c);
                const uint32_t st = sbase + out_at + (uint32_t)(warp * kOutBufs + stores) * kOutBytes;
                if (me.splits > 1) {
                    float y[32];
                    load_sums<Out>(from, g.nt, y);
                    const uint32_t p = sbase + (uint32_t)(c * kFeatures + warp * 32 + lane) * 4;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(p + e * kFeatures * 4), "f"(y[e]) : "memory");
                } else if (f < g.F) {
                    if (lane == 0) bulk_wait_read<kOutBufs - 1>();  // the last store from this buffer has left it
                    __syncwarp();
                    if constexpr (sizeof(Out) == 4) {
                        float y[32];
                        load_sums<Out>(from, g.nt, y);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(st + e * 128 + lane * 4), "f"(y[e]) : "memory");
                    } else {
                        // 8 x 8 matrices, features by tokens, transposed on their way (a value at a time took twice as long):
                        // a store has those of 8 tokens and all 32 features, 16 bytes a row with the map's swizzle.
                        uint32_t lo[16], hi[16];
                        tmem_load_matrices(from, lo, hi);
                        const uint32_t to = st + (uint32_t)(lane & 7) * 64u + (uint32_t)((lane >> 3) ^ ((lane & 7) >> 1)) * 16u;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            st_matrices_trans(to + j * 512, pack2<Out>(lo[4 * j], lo[4 * j + 1]), pack2<Out>(lo[4 * j + 2], lo[4 * j + 3]),
                                              pack2<Out>(hi[4 * j], hi[4 * j + 1]), pack2<Out>(hi[4 * j + 2], hi[4 * j + 3]));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&map_y, f, at.t0 + c, st);
                        bulk_commit();
                    }
                    stores = stores + 1 == kOutBufs ? 0 : stores + 1;
                }
            }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) pair_arrive(cluster_map(smem_u32(&acc_empty[buf]), me.lead));
        __syncwarp();
        if (++buf == g.bufs) {
            buf = 0;
            ph ^= 1;
        }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
}

// The splits' partial sums to Y, a share of the tile's tokens by each pair (all threads, after the cluster has met).
template <typename Out>
__device__ __forceinline__ void add_splits(const TileArgs& g, const Share& me, uint32_t sbase, int threads) {
    const Place at = place_of(g, me.cid, me.half);
    const int n = (g.nt + me.splits - 1) / me.splits, t0 = me.split * n;
    const int live = min(g.nt, g.tokens - at.t0);
    for (int i = threadIdx.x; i < n * (kFeatures / 4); i += threads) {
        const int t = t0 + i / (kFeatures / 4), x = i % (kFeatures / 4) * 4, f = at.f0 + x;
        if (t >= live || t >= t0 + n || f >= g.F) continue;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < me.splits; ++j) {
            const float4 p = ld_cluster_f4(cluster_map(sbase + (uint32_t)(t * kFeatures + x) * 4, 2 * j + me.half));
            y[0] += p.x;
            y[1] += p.y;
            y[2] += p.z;
            y[3] += p.w;
        }
        Out* out = static_cast<Out*>(g.Y) + (int64_t)(at.t0 + t) * g.ldy + f;
        if (f + 4 <= g.F) {  // (rows begin on 16-byte boundaries)
            if constexpr (sizeof(Out) == 4) *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
            else *reinterpret_cast<uint2*>(out) = make_uint2(Elt<Out>::p2(y[0], y[1]), Elt<Out>::p2(y[2], y[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (f + e < g.F) out[e] = Elt<Out>::from_f(y[e]);
        }
    }
}

// ------------------------------------------------------------------ host side

template <typename T>
constexpr CUtensorMapDataType kMapType = sizeof(T) == 1                          ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                         : sizeof(T) == 4                        ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
// Map of a row-strided matrix in boxes of box_cols x box_rows.
template <typename T>
bool encode_matrix(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_cols, int box_rows,
                   CUtensorMapSwizzle swizzle) {
    const cuuint64_t d[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, st[1] = {(cuuint64_t)ld * sizeof(T)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, elem[2] = {1, 1};
    return encode_fn()(map, kMapType<T>, 2, const_cast<void*>(p), d, st, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `pairs` pairs that the device holds at once (asked once per kernel and device).
constexpr int kMaxSplits = 4;
template <typename K>
int clusters_at_once(K kern, int threads, uint32_t smem, int pairs, int (&known)[64][kMaxSplits + 1]) {
    const DeviceProps& p = device_props();
    const int d = p.device;
    if (d >= 0 && d < 64 && known[d][pairs]) return known[d][pairs];
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * pairs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = pairs == 1 ? (p.sm_count > 1 ? p.sm_count / 2 : 1) : 1;
    }
    if (d >= 0 && d < 64) known[d][pairs] = n;
    return n;
}

// A kernel's form for a product: tokens of a tile, splits, 64s of the contraction in a stage, clusters at once.
struct Shape {
    int nt, splits, sub, at_once;
};

// What the kernels take alike, for this shape (sub 64s of the contraction C in a stage). false: too large.
template <typename T, typename Out>
bool tile_args(TileArgs& g, const Mx4Args& a, int32_t F, int32_t C, Shape shape, int parts, CUtensorMap* mx, CUtensorMap* my) {
    g.codes = a.codes;
    g.scales = a.scales;
    g.Y = a.Y;
    g.ldy = a.ldy;
    g.blocks = mx4_blocks(a.cols);
    g.rows = a.rows;
    g.F = F;
    g.tokens = a.tokens;
    g.ftiles = (int32_t)(((int64_t)F + 2 * kFeatures - 1) / (2 * kFeatures));
    g.nt = shape.nt;
    g.chunks = (int32_t)(((int64_t)C + shape.sub * kKC - 1) / (shape.sub * kKC));
    const int64_t tiles = (int64_t)g.ftiles * (((int64_t)a.tokens + shape.nt - 1) / shape.nt);
    // (a split without a chunk would have no sums; the indices of tiles and CTAs have 32 bits)
    if (shape.splits > g.chunks || tiles > 0x7fffffff / (4 * kMaxSplits)) return false;
    g.tiles = (int32_t)tiles;
    g.part = (int32_t)(mx4_split_cols(C) / 3);
    g.err = device_error_word();
    // (rows of whole 16 bytes: copies of others have zeros, or room, behind their columns)
    const int64_t x_cols = parts > 1 ? mx4_split_cols(C) : ((int64_t)C + 7) / 8 * 8, y16 = 16 / (int64_t)sizeof(Out);
    return encode_matrix<T>(mx, a.X, a.tokens, x_cols, a.ldx, kKC, shape.nt / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode_matrix<Out>(my, a.Y, a.tokens, ((int64_t)F + y16 - 1) / y16 * y16, a.ldy, 32, kOutTokens,
                              sizeof(Out) == 4 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B);
}

// Clusters that the device holds at once, for each number of splits.
template <typename K>
cudaError_t count_clusters(K kern, int threads, uint32_t smem, int (&at_once)[kMaxSplits + 1], int (&known)[64][kMaxSplits + 1],
                           bool (&done)[64]) {
    if (!encode_fn()) return cudaErrorNotSupported;
    const cudaError_t e = allow_smem(kern, smem, done);  // (before its clusters are counted)
    if (e != cudaSuccess) return e;
    for (int i = 1; i <= kMaxSplits; ++i) at_once[i] = clusters_at_once(kern, threads, smem, i, known);
    return cudaSuccess;
}

}  // namespace
}  // namespace spops
