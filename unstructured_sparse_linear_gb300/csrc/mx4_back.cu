// Products with a microscaled 4-bit weight on the tcgen05 tensor cores (rows of whole 16 bytes): the input gradient.
//
// mx4_back_kernel  Y[t, f] = sum over c of X[t, c] W[c, f].
//
// The weight is the A operand (128 features x 64 of the contraction, decoded from 4 bits to X's type by groups of four warps),
// X the B operand (nt tokens x 64, by TMA), so D is features x tokens. Two CTAs form a pair (cta_group::2): 256 features,
// each CTA decodes its own 128 and holds half of the tokens' rows, so a value is decoded once per nt tokens and X is read
// from L2 once per 256 features. A row's codes run along the features, across the contraction: the operand in shared memory is
// MN-major, which takes them as they are decoded (tensor memory has the contraction along its columns, and would need each
// code alone).
// Bounds. Per 64 of the contraction shared memory takes the decoded operand twice (written, read) and X twice: 512 cycles at 256
// tokens, as many as the products (8192 tokens 8192 -> 2048: 91 % of its wavefronts, tensor pipe 82 %). 4096 tokens
// 11008 -> 4096 213 us, 1736 TFLOP/s; 2048 tokens 4096 -> 4096 fp16 47; 64 tokens 24 to 28, the latency of
// a stage's codes, which a decoder asks for one stage ahead (a warp waits for loads in 6.2 of the 15 cycles between two of its
// instructions; issue 36 %, integer pipe 28 %), on the 96 SMs that have a tile.
// fp32: the weight's values are bf16 numbers, and X is the sum of three bf16 parts (mx4_split_kernel), which multiply the same
// decoded weight; the first part's products have an accumulator of their own. 700 tokens 4096 -> 6136 75 us, 2048
// tokens 4096 -> 4096 172 (1.4 and 1.6 of their operations' time).
#include "mx4_pair.cuh"

namespace spops {
namespace {

constexpr uint32_t kWBytes = kFeatures * 128;  // of 64 of the contraction
constexpr uint32_t kRing = 6 * (kWBytes + kMaxTokens / 2 * 128);
constexpr int kMaxStages = 10;
constexpr int kAheadL2 = 6;
constexpr uint32_t kOutAt = kRing;

// A stage holds kSub times 64 of the contraction: one, or two where the products of 64 take less time than the messages of a
// stage (up to 128 tokens), and X in kParts parts. Warps 0 to 3 finish (a TMEM lane quarter each), then kGroups groups of
// four decode, one warp loads X, one multiplies.
template <typename Out, int kSub>
struct BackCfg {
    static constexpr int kParts = sizeof(Out) == 4 ? 3 : 1;
    static constexpr int kGroups = kSub == 1 && kParts == 1 ? 6 : 4;
    static constexpr int kLoadWarp = 4 + 4 * kGroups, kMmaWarp = kLoadWarp + 1, kThreads = 32 * (kMmaWarp + 1);
    static constexpr int kOutBufs = kParts == 1 ? 4 : 2;  // (what fits)
    static constexpr int kTokens = kSub == 1 && kParts == 1 ? kMaxTokens : kMaxTokens / 2;  // at most
    static constexpr uint32_t kOutBytes = kOutTokens * 32 * sizeof(Out), kBarsAt = kOutAt + 4 * kOutBufs * kOutBytes, kSmem = kBarsAt + 1024;
    static_assert(kGroups <= (int)(kRing / (kSub * (kWBytes + kParts * kTokens * 64))), "a group's next stage is at most one round of the ring away");
    static_assert(kTokens * kFeatures * 4u <= kRing, "the partial sums fit");
};

template <typename T, typename Out, int kSub>
__global__ void __launch_bounds__(BackCfg<Out, kSub>::kThreads, 1)
mx4_back_kernel(const TileArgs g, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ CUtensorMap map_y) {
    using Cfg = BackCfg<Out, kSub>;
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
    const Share me(g);
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
    // Codes are asked for in pieces of 64 bytes a row, by threads that wait for them: for the first token tile, which is the
    // first to read them, the loader has them fetched into L2 kAheadL2 stages before (64 tokens 11008 -> 4096, weight not in
    // L2: 23.6 us, 27.5 without; in it 21.2 and 20.7).
    auto fetch = [&](int f0, int c) {
        if (c < me.c1)
            asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&map_w)),
                         "r"(f0 / 2), "r"(c * kSub * kKC)
                         : "memory");
    };
    if (tid == 32 * kLoadWarp && me.mine > 0) {
        const Place at = place_of(g, me.cid, me.half);
        if (at.t0 == 0)
            for (int d = 0; d < kAheadL2; ++d) fetch(at.f0, me.c0 + d);
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
        // (the whole warp walks the stages and one thread issues: what its copies take lies in uniform registers then)
        const bool issues = elect_one();
        const uint32_t full = cluster_map(smem_u32(&sh.full[0]), me.lead);  // the barriers count both CTAs' bytes
        uint32_t s = 0, ph = 1;
        for (int i = 0; i < me.mine; ++i) {
            const Place at = place_of(g, me.cid + i * me.ncl, me.half);
            for (int c = me.c0; c < me.c1; ++c) {
                const bool ok = wait(smem_u32(&sh.empty[s]), ph);
                if (issues && at.t0 == 0) fetch(at.f0, c + kAheadL2);
                if (issues && ok) {
                    if (me.half == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[s]), 2 * kSub * kParts * x_bytes);
#pragma unroll
                    for (int h = 0; h < kSub * kParts; ++h)  // (the parts of X lie one behind the other)
                        pair_tma_load_2d(sbase + s * stage_bytes + kSub * kWBytes + h * x_bytes, &map_x,
                                         kParts == 1 ? (c * kSub + h) * kKC : c * kKC + h * g.part, at.t0 + me.half * (g.nt / 2),
                                         full + s * 8);
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // The whole warp walks the stages and one thread issues: what the products take then lies in uniform registers (a
        // loop of one thread took 650 cycles a stage, more than its products). A wait that has run out of time is not
        // looked at: the products of whatever is there end, and the error is recorded.
        if (me.half == 0) {
            const uint32_t mask = 3u << me.lead;
            const uint64_t a0 = tc::smem_desc_sw128(sbase, 8192, 1024);
            const uint64_t b0 = tc::smem_desc_sw128(sbase + kSub * kWBytes, 0, 1024);
            constexpr uint32_t kStepA = 2048 / 16, kStepB = 32 / 16;  // 16 of the contraction
            const bool issues = elect_one();
            uint32_t s = 0, ph = 0, buf = 0, acc_ph = 1;
            for (int i = 0; i < me.mine; ++i) {
                const uint32_t d = tmem + buf * kMaxTokens;
                wait(smem_u32(&sh.acc_empty[buf]), acc_ph);
                tc::fence_after_sync();
                for (int c = 0; c < me.per; ++c) {
                    wait(smem_u32(&sh.full[s]), ph);
                    acquire_pair_smem();
                    tc::fence_after_sync();
                    if (issues) {
                        const uint32_t off = s * (stage_bytes / 16);
#pragma unroll
                        for (int h = 0; h < kSub * kParts; ++h)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                pair_mma_f16(kParts > 1 && h > 0 ? d + (uint32_t)g.nt : d, a0 + off + (kParts == 1 ? h : 0) * (kWBytes / 16) + k * kStepA,
                                             b0 + off + h * (x_bytes / 16) + k * kStepB, g.idesc,
                                             c > 0 || k > 0 || h > (kParts == 1 ? 0 : 1));
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
        // stores' fence, the message) overlap with those of others. A thread has row r of each 64 of the contraction, block
        // `sub` of both 64-feature halves, which are operand blocks of their own.
        const int id = tid & 127, sub = id & 1, r = id >> 1, group = (warp - 4) >> 2;
        const uint32_t to = sbase + (uint32_t)(r >> 3) * 1024u + (uint32_t)(r & 7) * 128u;
        const uint32_t flip = (uint32_t)(4 * sub ^ (r & 7)) << 4;  // the first 16 bytes' place in their row; the others: ^ k
        const uint32_t full = cluster_map(smem_u32(&sh.full[0]), me.lead);
        // The next stage to ask for: number ac of tile ai. A thread's blocks lie at pc and pc + 2 blocks.
        const int64_t next64 = (int64_t)kKC * g.blocks;  // from 64 of the contraction to the next
        int ai = 0, ac = group;
        int64_t row = 0;
        const uint8_t *pc = g.codes, *ps = g.scales;
        bool in0 = false, in1 = false;
        auto aim = [&]() {
            while (ac >= me.per && ai < me.mine) {
                ac -= me.per;
                ++ai;
            }
            if (ai >= me.mine) {
                in0 = in1 = false;
                return;
            }
            const int64_t blk = place_of(g, me.cid + ai * me.ncl, me.half).f0 / kMx4Block + sub;
            row = (int64_t)(me.c0 + ac) * kSub * kKC + r;
            in0 = blk < g.blocks;
            in1 = blk + 2 < g.blocks;
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
                    if (row + h * kKC < g.rows && (x ? in1 : in0)) {
                        const int64_t at = h * next64 + x * 2;
                        k.w[2 * h + x] = ld_v4(pc + at * 16);
                        k.b[2 * h + x] = ps[at];
                    }
                }
            }
            ac += kGroups;
            row += kGroups * kSub * kKC;
            pc += kGroups * kSub * next64 * 16;
            ps += kGroups * kSub * next64;
            if (ac >= me.per) aim();
        };
        Blocks next;
        ask(next);
        uint32_t s = group, ph = 1;
        for (int64_t left = (int64_t)me.mine * me.per - group; left > 0; left -= kGroups) {
            const bool ok = wait(smem_u32(&sh.empty[s]), ph);
            if (ok) {
#pragma unroll
                for (int x = 0; x < kBlocks; ++x) {
                    const uint32_t w[4] = {next.w[x].x, next.w[x].y, next.w[x].z, next.w[x].w}, b = next.b[x];
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
            ask(next);  // (behind the message, which the multiplying warp waits for)
            s += kGroups;
            if (s >= stages) {
                s -= stages;
                ph ^= 1;
            }
        }
    } else {
        finish_tiles<Out, Cfg::kOutBufs>(g, me, map_y, wait, sh.acc_full, sh.acc_empty, sbase, kOutAt, tmem, kMaxTokens, warp, lane);
    }
    if (me.splits > 1) {
        cluster_sync();
        if (!sh.failed && me.mine > 0) add_splits<Out>(g, me, sbase, kThreads);
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

// Tokens per tile and splits of the contraction with the least estimated time in us, fitted to sweeps over both (384 to
// 11008 features, 6 to 172 chunks, 9 to 8192 tokens; the choice is within a tenth of the best of a sweep): 64 of the
// contraction take 0.265 with two of them a stage and 0.3 with one, or their products; a pass without splits 4.4 beside
// that, and its tiles follow each other; with splits, every wave of clusters begins anew and adds its sums.
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

template <typename T, typename Out, int kSub>
cudaError_t run_shape(const Mx4Args& a, Shape shape, cudaStream_t s) {
    using Cfg = BackCfg<Out, kSub>;
    static bool done[64];
    auto kern = mx4_back_kernel<T, Out, kSub>;
    const cudaError_t e = allow_smem(kern, Cfg::kSmem, done);
    if (e != cudaSuccess) return e;
    TileArgs g{};
    CUtensorMap mw, mx, my;
    if (!tile_args<T, Out>(g, a, a.cols, a.rows, shape, Cfg::kParts, &mx, &my) ||
        !encode_matrix<uint8_t>(&mw, a.codes, a.rows, g.blocks * 16, g.blocks * 16, kFeatures / 2, kSub * kKC, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    g.bufs = 2;
    g.stages = min((int)(kRing / (kSub * (kWBytes + Cfg::kParts * shape.nt * 64))), kMaxStages);
    g.idesc = tc::instr_desc_f16(std::is_same<T, __nv_bfloat16>::value ? 1u : 0u, 1u, 0u, 2 * kFeatures, (uint32_t)shape.nt);
    const int c = 2 * shape.splits, clusters = shape.splits > 1 || g.tiles < shape.at_once ? g.tiles : shape.at_once;
    count_launches(1);
    return launch_pdl_cluster(kern, dim3((unsigned)(clusters * c)), dim3(Cfg::kThreads), Cfg::kSmem, (unsigned)c, s, g, mw, mx, my);
}

template <typename T, typename Out>
cudaError_t run_tiles(const Mx4Args& a, cudaStream_t s) {
    using Cfg = BackCfg<Out, 1>;
    static int known[64][kMaxSplits + 1];
    static bool done[64];
    int at_once[kMaxSplits + 1];
    // (as many of the kernel with two 64s a stage, which has the same shared memory)
    const cudaError_t e = count_clusters(mx4_back_kernel<T, Out, 1>, Cfg::kThreads, Cfg::kSmem, at_once, known, done);
    if (e != cudaSuccess) return e;
    const Shape shape = choose(a.tokens, ((int64_t)a.cols + 2 * kFeatures - 1) / (2 * kFeatures),
                               (int)(((int64_t)a.rows + kKC - 1) / kKC), Cfg::kParts, at_once);
    if constexpr (Cfg::kParts == 1)
        if (shape.sub == 2) return run_shape<T, Out, 2>(a, shape, s);
    return run_shape<T, Out, 1>(a, shape, s);
}

}  // namespace

cudaError_t launch_mx4_backward(int dt, const Mx4Args& a, cudaStream_t s) {
    if (dt == kF32) return run_tiles<__nv_bfloat16, float>(a, s);
    return dt == kF16 ? run_tiles<__half, __half>(a, s) : run_tiles<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace spops
