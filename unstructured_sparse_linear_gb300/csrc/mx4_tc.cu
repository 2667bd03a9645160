// Products with a microscaled 4-bit weight on the tcgen05 tensor cores (rows of whole 16 bytes).
//
// mx4_tile_kernel  Y[t, f] = sum over c of X[t, c] V(f, c), V = W (forward: f a row of W, c a column) or its transpose
//                  (back: the input gradient).
//
// The weight is the A operand (128 features x 64 of the contraction, decoded from 4 bits to X's type by groups of four warps),
// X the B operand (nt tokens x 64, by TMA), so D is features x tokens. Two CTAs form a pair (cta_group::2): 256 features,
// each CTA decodes its own 128 and holds half of the tokens' rows, so a value is decoded once per nt tokens and X is read
// from L2 once per 256 features. Forward, a row's codes run along the contraction: the operand is K-major; back, they run
// along the features: the same decoding writes an MN-major operand, and no code is ever transposed.
// fp32: the weight's values are bf16 numbers, and X is the sum of three bf16 parts (all 24 bits), which multiply the same
// decoded weight into the same fp32 sums.
#include <type_traits>

#include "internal.h"
#include "mx4.cuh"
#include "mx4.h"
#include "pipeline.cuh"

namespace spops {
namespace {

constexpr int kKC = 64;             // contraction elements of a stage: 128-byte rows
constexpr int kFeatures = 128;      // of a CTA
constexpr int kMaxTokens = 256;     // of a tile
constexpr uint32_t kWBytes = kFeatures * 128;  // of 64 of the contraction
constexpr uint32_t kRing = 6 * (kWBytes + kMaxTokens / 2 * 128);
constexpr int kMaxStages = 10;
constexpr int kOutTokens = 32;  // of a store: 32 x 32 values
constexpr uint32_t kOutAt = kRing;
constexpr int kAhead = 1;  // stages whose codes a decoder has under way

// A stage holds kSub times 64 of the contraction: one, or two where the products of 64 take less time than the messages of a
// stage (up to 128 tokens), and X in kParts parts. Warps 0 to 3 finish (a TMEM lane quarter each), then kGroups groups of
// four decode, one warp loads X, one multiplies.
template <typename Out, int kSub>
struct TileCfg {
    static constexpr int kParts = sizeof(Out) == 4 ? 3 : 1;
    static constexpr int kGroups = kSub == 1 && kParts == 1 ? 6 : 4;
    static constexpr int kLoadWarp = 4 + 4 * kGroups, kMmaWarp = kLoadWarp + 1, kThreads = 32 * (kMmaWarp + 1);
    static constexpr int kTokens = kSub == 1 && kParts == 1 ? kMaxTokens : kMaxTokens / 2;  // at most
    static constexpr uint32_t kOutBytes = kOutTokens * 32 * sizeof(Out), kBarsAt = kOutAt + 4 * 2 * kOutBytes, kSmem = kBarsAt + 1024;
    static_assert(kGroups <= (int)(kRing / (kSub * (kWBytes + kParts * kTokens * 64))), "a group's next stage is at most one round of the ring away");
    static_assert(kTokens * kFeatures * 4u <= kRing, "the partial sums fit");
};

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
// each writer's proxy fence has made it visible, or has left TMEM: no release of the cluster's scope, which took a warp 500
// cycles for each stage.
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
    int64_t tiles;   // ftiles x token tiles
    int32_t rows, F, tokens, ftiles, chunks, nt, stages;
    uint32_t idesc;
    int* err;
};

// A tile's place: 256 features x nt tokens; the tiles of the same tokens follow each other.
struct Place {
    int f0, t0;
};
__device__ __forceinline__ Place place_of(const TileArgs& g, int64_t tile, int half) {
    const int64_t tt = tile / g.ftiles;
    return {(int)(tile - tt * g.ftiles) * (2 * kFeatures) + half * kFeatures, (int)(tt * g.nt)};
}

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

// A cluster is one pair, or S pairs that split a tile's contraction; in the second case (one tile per cluster) the fp32
// partial sums meet in shared memory and are added in the order of the splits.
template <typename T, typename Out, bool kBack, int kSub>
__global__ void __launch_bounds__(TileCfg<Out, kSub>::kThreads, 1)
mx4_tile_kernel(const TileArgs g, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_y) {
    using Cfg = TileCfg<Out, kSub>;
    constexpr int kLoadWarp = Cfg::kLoadWarp, kMmaWarp = Cfg::kMmaWarp, kThreads = Cfg::kThreads, kParts = Cfg::kParts;
    constexpr int kGroups = Cfg::kGroups, kBlocks = 2 * kSub;  // blocks of a decoder and stage
    // No static shared memory, so the dynamic part starts on the 1 KB boundary that the swizzled tiles need (checked).
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    struct Shared {
        uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
        uint32_t tmem;
        volatile int failed;
    };
    static_assert(sizeof(Shared) <= Cfg::kSmem - Cfg::kBarsAt, "barriers");
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw + Cfg::kBarsAt);
    const uint32_t sbase = smem_u32(smem_raw);
    if (sbase & 1023u) {  // the same on every CTA
        record_error(g.err, kDevErrSmemAlign);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t stages = g.stages, x_bytes = (uint32_t)g.nt * 64, stage_bytes = kSub * (kWBytes + kParts * x_bytes);
    const int C = (int)cluster_size(), crank = (int)cluster_rank();
    const int half = crank & 1, lead = crank & ~1, split = crank >> 1, splits = C >> 1;
    const int64_t cid = blockIdx.x / C, ncl = gridDim.x / C;
    const int c0 = (int)((int64_t)g.chunks * split / splits), c1 = (int)((int64_t)g.chunks * (split + 1) / splits);
    const int per = c1 - c0;                                               // chunks of a tile
    const int64_t mine = cid < g.tiles && per > 0 ? (g.tiles - cid + ncl - 1) / ncl : 0;  // tiles of this cluster
    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 2 * 4 + 1);  // decoding warps of the pair, the loader
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_empty[i]), 2 * 4);  // finishing warps of the pair
        }
        sh.failed = 0;
        fence_mbar_init();
    }
    if (tid == 32 * kLoadWarp) {
        tma_prefetch_map(&map_x);
        tma_prefetch_map(&map_y);
    }
    __syncthreads();
    pdl_wait();
    if (warp == kMmaWarp) pair_alloc(smem_u32(&sh.tmem), 512);
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();
    tc::fence_after_sync();
    pdl_trigger();
    const uint32_t tmem = sh.tmem;
    const PairWaits wait{&sh.failed, g.err};

    if (warp == kLoadWarp) {
        if (lane == 0) {
            uint32_t s = 0, ph = 1;
            for (int64_t i = 0; i < mine; ++i) {
                const Place at = place_of(g, cid + i * ncl, half);
                for (int c = c0; c < c1; ++c) {
                    if (wait(smem_u32(&sh.empty[s]), ph)) {
                        const uint32_t bar = smem_u32(&sh.full[s]);
                        if (half == 0) mbar_arrive_expect_tx(bar, 2 * kSub * kParts * x_bytes);  // of both CTAs
#pragma unroll
                        for (int h = 0; h < kSub * kParts; ++h)  // (the parts of X lie one behind the other)
                            pair_tma_load_2d(sbase + s * stage_bytes + kSub * kWBytes + h * x_bytes, &map_x,
                                             (kParts == 1 ? c * kSub + h : c + h * g.chunks) * kKC, at.t0 + half * (g.nt / 2),
                                             cluster_map(bar, lead));
                    }
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // The whole warp walks the chunks and one thread issues: what the products take then lies in uniform registers (a
        // loop of one thread took 650 cycles a chunk, more than its products). A wait that has run out of time is not
        // looked at: the products of whatever is there end, and the error is recorded.
        if (half == 0) {
            const uint32_t mask = 3u << lead;
            const uint64_t a0 = kBack ? tc::smem_desc_sw128(sbase, 8192, 1024) : tc::smem_desc_sw128(sbase, 0, 1024);
            const uint64_t b0 = tc::smem_desc_sw128(sbase + kSub * kWBytes, 0, 1024);
            constexpr uint32_t kStepA = kBack ? 2048 / 16 : 32 / 16, kStepB = 32 / 16;  // 16 of the contraction
            const bool issues = elect_one();
            uint32_t s = 0, ph = 0, buf = 0, acc_ph = 1;
            for (int64_t i = 0; i < mine; ++i) {
                const uint32_t d = tmem + buf * kMaxTokens;
                wait(smem_u32(&sh.acc_empty[buf]), acc_ph);
                tc::fence_after_sync();
                for (int c = 0; c < per; ++c) {
                    wait(smem_u32(&sh.full[s]), ph);
                    acquire_pair_smem();
                    tc::fence_after_sync();
                    if (issues) {
                        const uint32_t off = s * (stage_bytes / 16);
#pragma unroll
                        for (int h = 0; h < kSub * kParts; ++h)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                pair_mma_f16(d, a0 + off + (kParts == 1 ? h : 0) * (kWBytes / 16) + k * kStepA,
                                             b0 + off + h * (x_bytes / 16) + k * kStepB, g.idesc, c > 0 || h > 0 || k > 0);
                        pair_commit(smem_u32(&sh.empty[s]), mask);
                    }
                    __syncwarp();
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (issues) pair_commit(smem_u32(&sh.acc_full[buf]), mask);
                __syncwarp();
                buf ^= 1;
                acc_ph ^= buf ^ 1;
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // A group of four warps takes every kGroups-th stage, so that the steps of one stage (codes that arrive, decoding, the
        // stores' fence, the message) overlap with those of others. A thread has two blocks of each 64 of the contraction.
        // Forward: rows r and r + 64, block `sub` of two; back: row r, block `sub` of both 64-feature halves, which are
        // operand blocks of their own.
        const int id = tid & 127, sub = id & 1, r = id >> 1, group = (warp - 4) >> 2;
        const uint32_t to = sbase + (uint32_t)(r >> 3) * 1024u + (uint32_t)(r & 7) * 128u;
        const uint32_t flip = (uint32_t)(4 * sub ^ (r & 7)) << 4;  // the first 16 bytes' place in their row; the others: ^ k
        const uint32_t full = cluster_map(smem_u32(&sh.full[0]), lead);
        // The next stage to ask for: number ac of tile ai. A thread's blocks lie at pc and pc + second; pos counts what may
        // end within a chunk (forward: blocks of the row; back: rows).
        const int64_t second = kBack ? 2 : 64 * g.blocks;
        const int64_t next64 = kBack ? (int64_t)kKC * g.blocks : 2;  // from 64 of the contraction to the next
        constexpr int kPos = kBack ? kKC : 2;
        const int64_t end = kBack ? g.rows : g.blocks;
        int64_t ai = 0, pos = 0;
        int ac = group;
        const uint8_t *pc = g.codes, *ps = g.scales;
        bool in0 = false, in1 = false;
        auto aim = [&]() {
            while (ac >= per && ai < mine) {
                ac -= per;
                ++ai;
            }
            if (ai >= mine) {
                in0 = in1 = false;
                return;
            }
            const Place at = place_of(g, cid + ai * ncl, half);
            const int64_t c = (int64_t)(c0 + ac) * kSub;
            const int64_t row = kBack ? c * kKC + r : at.f0 + r, blk = kBack ? at.f0 / kMx4Block + sub : 2 * c + sub;
            pos = kBack ? row : blk;
            in0 = kBack ? blk < g.blocks : row < g.rows;
            in1 = kBack ? blk + 2 < g.blocks : row + 64 < g.rows;
            pc = g.codes + (row * g.blocks + blk) * 16;
            ps = g.scales + row * g.blocks + blk;
        };
        aim();
        struct Blocks {
            uint4 w[kBlocks];
            uint32_t b[kBlocks];
        };
        auto ask = [&](Blocks& k) {
#pragma unroll
            for (int h = 0; h < kSub; ++h) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    k.w[2 * h + x] = make_uint4(0, 0, 0, 0);
                    k.b[2 * h + x] = 0;
                    if (pos + h * kPos < end && (x ? in1 : in0)) {
                        const int64_t at = h * next64 + x * second;
                        k.w[2 * h + x] = ld_nc_v4(pc + at * 16);
                        k.b[2 * h + x] = __ldg(ps + at);
                    }
                }
            }
            ac += kGroups;
            pos += kGroups * kSub * kPos;
            pc += kGroups * kSub * next64 * 16;
            ps += kGroups * kSub * next64;
            if (ac >= per) aim();
        };
        Blocks next[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) ask(next[u]);
        uint32_t s = group, ph = 1;
        for (int64_t left = mine * per - group; left > 0; left -= kGroups * kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (left <= u * kGroups) break;
                const bool ok = wait(smem_u32(&sh.empty[s]), ph);
                if (ok) {
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) {
                        const uint32_t w[4] = {next[u].w[x].x, next[u].w[x].y, next[u].w[x].z, next[u].w[x].w}, b = next[u].b[x];
                        const uint32_t at = to + s * stage_bytes + x * 8192u;  // (kWBytes for each 64 of the contraction)
                        if (mx4::plain(b) || (b != 255 && (w[0] | w[1] | w[2] | w[3]) == 0)) {  // (or nothing but zeros)
                            const uint32_t f = mx4::plain(b) ? mx4::factor2(b) : 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t v[4];
                                mx4::decode8<T>(w[k], f, v);
                                st_shared_v4(at + (flip ^ (uint32_t)(k << 4)), make_uint4(v[0], v[1], v[2], v[3]));
                            }
                        } else {
#pragma unroll 1
                            for (int k = 0; k < 4; ++k) {
                                uint32_t v[4];
                                mx4::decode8_any<T>(k == 0 ? w[0] : k == 1 ? w[1] : k == 2 ? w[2] : w[3], b, v);
                                st_shared_v4(at + (flip ^ (uint32_t)(k << 4)), make_uint4(v[0], v[1], v[2], v[3]));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0 && ok) pair_arrive(full + s * 8);
                __syncwarp();
                ask(next[u]);  // (behind the message, which the multiplying warp waits for)
                s += kGroups;
                if (s >= stages) {
                    s -= stages;
                    ph ^= 1;
                }
            }
        }
    } else {
        uint32_t stores = 0;
        for (int64_t i = 0; i < mine; ++i) {
            const Place at = place_of(g, cid + i * ncl, half);
            const uint32_t buf = (uint32_t)i & 1u;
            const bool ok = wait(smem_u32(&sh.acc_full[buf]), (uint32_t)((i >> 1) & 1));
            const bool all = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
            const int f = at.f0 + warp * 32;
            const int live = min(g.nt, g.tokens - at.t0);
            if (all)
                for (int c = 0; c < live; c += kOutTokens) {
                    float y[32];
                    tmem_load<32>(tmem + ((uint32_t)warp << 21) + buf * kMaxTokens + c, y);
                    if (splits > 1) {  // [token][128 features], fp32
                        const uint32_t p = sbase + (uint32_t)(c * kFeatures + warp * 32 + lane) * 4;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(p + e * kFeatures * 4), "f"(y[e]) : "memory");
                    } else if (f < g.F) {
                        const uint32_t st = sbase + kOutAt + (uint32_t)(warp * 2 + (stores & 1)) * Cfg::kOutBytes;
                        if (lane == 0) bulk_wait_read<1>();  // the store before the last has left this buffer
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if constexpr (sizeof(Out) == 4) {
                                asm volatile("st.shared.f32 [%0], %1;" ::"r"(st + e * 128 + lane * 4), "f"(y[e]) : "memory");
                            } else {
                                const Out t = Elt<Out>::from_f(y[e]);
                                asm volatile("st.shared.b16 [%0], %1;" ::"r"(st + e * 64 + lane * 2),
                                             "h"(reinterpret_cast<const uint16_t&>(t))
                                             : "memory");
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&map_y, f, at.t0 + c, st);
                            bulk_commit();
                        }
                        ++stores;
                    }
                }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) pair_arrive(cluster_map(smem_u32(&sh.acc_empty[buf]), lead));
            __syncwarp();
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    }
    if (splits > 1) {
        cluster_sync();
        const Place at = place_of(g, cid, half);
        const int n = (g.nt + splits - 1) / splits, t0 = split * n;  // this CTA's tokens of the tile
        const int live = min(g.nt, g.tokens - at.t0);
        if (!sh.failed && mine > 0)
            for (int i = tid; i < n * (kFeatures / 4); i += kThreads) {
                const int t = t0 + i / (kFeatures / 4), x = i % (kFeatures / 4) * 4, f = at.f0 + x;
                if (t >= live || t >= t0 + n || f >= g.F) continue;
                float y[4] = {0.f, 0.f, 0.f, 0.f};
                for (int j = 0; j < splits; ++j) {
                    const float4 p = ld_cluster_f4(cluster_map(sbase + (uint32_t)(t * kFeatures + x) * 4, 2 * j + half));
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
    if (sh.failed)  // copies and products that are still in flight
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < kDrainNs;) {
        }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // the pair's products are done, nobody reads this CTA's memory any more
    if (warp == kMmaWarp) pair_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host side

template <typename T>
constexpr CUtensorMapDataType kMapType = sizeof(T) == 4                          ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : std::is_same<T, __nv_bfloat16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
// Map of a row-strided matrix in boxes of box_cols x box_rows, with the 128-byte swizzle or without.
template <typename T>
bool encode_matrix(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_cols, int box_rows,
                   bool swizzle) {
    const cuuint64_t d[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, st[1] = {(cuuint64_t)ld * sizeof(T)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, elem[2] = {1, 1};
    return encode_fn()(map, kMapType<T>, 2, const_cast<void*>(p), d, st, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

// Tokens per tile and splits of the contraction with the least estimated time in us, fitted to sweeps over both (384 to
// 11008 features, 6 to 172 chunks, 9 to 8192 tokens; the choice is within a tenth of the best of a sweep): 64 of the
// contraction take 0.265 with two of them a stage and 0.3 with one, or their products; a pass without splits 4.4 beside
// that, and its tiles follow each other; with splits, every wave of clusters begins anew and adds its sums.
struct Shape {
    int nt, splits, sub, at_once;
};
Shape choose(int64_t tokens, int64_t ftiles, int chunks, int parts, const int (&at_once)[kMaxSplits + 1]) {
    const int most = parts == 1 ? kMaxTokens : kMaxTokens / 2;
    Shape best{most, 1, 1, at_once[1]};
    double least = 1e300;
    for (int nt = 32; nt <= most; nt += 32) {
        const int sub = parts == 1 && nt <= kMaxTokens / 2 ? 2 : 1, stages = (chunks + sub - 1) / sub;
        for (int s = 1; s <= kMaxSplits && s <= stages; ++s) {
            const int64_t tiles = ftiles * ((tokens + nt - 1) / nt), waves = (tiles + at_once[s] - 1) / at_once[s];
            const double products = 0.0014 * nt * parts, least64 = sub == 2 ? 0.265 : 0.3;
            const double stage = sub * (products > least64 ? products : least64), steps = (stages + s - 1) / s;
            const double t = s == 1 ? 4.4 + waves * (steps * stage + 0.2) + 0.008 * nt
                                    : waves * (5.0 + 0.3 * s + 0.012 * nt + steps * stage);
            if (t < least) {
                least = t;
                best = {nt, s, sub, at_once[s]};
            }
        }
    }
    return best;
}

template <typename T, typename Out, bool kBack, int kSub>
cudaError_t run_shape(const Mx4Args& a, TileArgs& g, Shape shape, cudaStream_t s) {
    using Cfg = TileCfg<Out, kSub>;
    static bool done[64];
    auto kern = mx4_tile_kernel<T, Out, kBack, kSub>;
    const cudaError_t e = allow_smem(kern, Cfg::kSmem, done);
    if (e != cudaSuccess) return e;
    const int32_t C = kBack ? a.rows : a.cols;
    g.nt = shape.nt;
    g.chunks = (int32_t)(((int64_t)C + kSub * kKC - 1) / (kSub * kKC));
    if (shape.splits > g.chunks) return cudaErrorInvalidValue;  // (a split without a chunk would have no sums)
    g.stages = min((int)(kRing / (kSub * (kWBytes + Cfg::kParts * shape.nt * 64))), kMaxStages);
    g.tiles = (int64_t)g.ftiles * (((int64_t)a.tokens + shape.nt - 1) / shape.nt);
    g.idesc = tc::instr_desc_f16(std::is_same<T, __nv_bfloat16>::value ? 1u : 0u, kBack ? 1u : 0u, 0u, 2 * kFeatures, (uint32_t)shape.nt);
    g.err = device_error_word();
    // (rows of whole 16 bytes: copies of others have zeros, or room, behind their columns)
    const int64_t x_cols = Cfg::kParts > 1 ? mx4_split_cols(C) : ((int64_t)C + 7) / 8 * 8, y16 = 16 / (int64_t)sizeof(Out);
    CUtensorMap mx, my;
    if (!encode_matrix<T>(&mx, a.X, a.tokens, x_cols, a.ldx, kKC, shape.nt / 2, true) ||
        !encode_matrix<Out>(&my, a.Y, a.tokens, ((int64_t)g.F + y16 - 1) / y16 * y16, a.ldy, 32, kOutTokens, false))
        return cudaErrorInvalidValue;
    const int c = 2 * shape.splits;
    const int64_t clusters = shape.splits > 1 ? g.tiles : min64(g.tiles, shape.at_once);
    if (clusters * c > 0x7fffffffll) return cudaErrorInvalidValue;
    count_launches(1);
    return launch_pdl_cluster(kern, dim3((unsigned)(clusters * c)), dim3(Cfg::kThreads), Cfg::kSmem, (unsigned)c, s, g, mx, my);
}

template <typename T, typename Out, bool kBack>
cudaError_t run_tiles(const Mx4Args& a, cudaStream_t s) {
    if (!encode_fn()) return cudaErrorNotSupported;
    using Cfg = TileCfg<Out, 1>;
    static int known[64][kMaxSplits + 1];
    static bool done[64];
    auto kern = mx4_tile_kernel<T, Out, kBack, 1>;
    const cudaError_t e = allow_smem(kern, Cfg::kSmem, done);  // (before its clusters are counted)
    if (e != cudaSuccess) return e;
    int at_once[kMaxSplits + 1];
    for (int i = 1; i <= kMaxSplits; ++i)  // (as many of the kernel with two chunks a stage, which has the same shared memory)
        at_once[i] = clusters_at_once(kern, Cfg::kThreads, Cfg::kSmem, i, known);
    TileArgs g;
    g.codes = a.codes;
    g.scales = a.scales;
    g.Y = a.Y;
    g.ldy = a.ldy;
    g.blocks = mx4_blocks(a.cols);
    g.rows = a.rows;
    g.F = kBack ? a.cols : a.rows;
    g.tokens = a.tokens;
    g.ftiles = (int32_t)(((int64_t)g.F + 2 * kFeatures - 1) / (2 * kFeatures));
    const int64_t C = kBack ? a.rows : a.cols;
    Shape shape = choose(a.tokens, g.ftiles, (int)((C + kKC - 1) / kKC), Cfg::kParts, at_once);
    if constexpr (Cfg::kParts == 1)
        if (shape.sub == 2) return run_shape<T, Out, kBack, 2>(a, g, shape, s);
    return run_shape<T, Out, kBack, 1>(a, g, shape, s);
}

}  // namespace

cudaError_t launch_mx4_tiles(int dt, bool back, const Mx4Args& a, cudaStream_t s) {
    if (dt == kF32)
        return back ? run_tiles<__nv_bfloat16, float, true>(a, s) : run_tiles<__nv_bfloat16, float, false>(a, s);
    if (dt == kF16) return back ? run_tiles<__half, __half, true>(a, s) : run_tiles<__half, __half, false>(a, s);
    return back ? run_tiles<__nv_bfloat16, __nv_bfloat16, true>(a, s) : run_tiles<__nv_bfloat16, __nv_bfloat16, false>(a, s);
}

}  // namespace spops
