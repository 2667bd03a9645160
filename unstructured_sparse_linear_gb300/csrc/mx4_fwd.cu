// Products with a microscaled 4-bit weight on the tcgen05 tensor cores (rows of whole 16 bytes): forward.
//
// mx4_fwd_kernel  Y[t, f] = sum over c of X[t, c] W[f, c].
//
// The weight is the A operand, decoded from 4 bits to X's type into tensor memory; X is the B operand (nt tokens x 64 of the
// contraction in shared memory, by TMA), so D is features x tokens. Two CTAs form a pair (cta_group::2): 256 features, each CTA
// decodes its own 128 and holds half of the tokens' rows, so a value is decoded once per nt tokens and X is read from L2 once
// per 256 features. Codes come by TMA as well: a thread decodes its own row (a TMEM lane), 16 bytes of it at a time.
// A weight that is decoded into shared memory is written and read there again by each product, and shared memory's bandwidth is
// then what bounds the kernel at every size; in tensor memory neither takes any of it (64 tokens 4096 -> 11008 22.4 us so and
// 14.1 here, 1037 tokens 4096 -> 4096 fp16 40 and 25.4).
// Bounds. 128 features x 256 of the contraction are 128 warps' words of 8 codes, 32 a scheduler: 22 cycles of its integer pipe each in
// bf16 (conversions, byte moves), 14 in fp16, which with the messages makes a stage 1000 cycles: what small products take (64
// tokens: 14.1 us for 22.5 MB of codes, 12.2 in fp16). From 160 tokens a tile on the products take longer: 8192 tokens
// 2048 -> 8192 149 us, 1840 TFLOP/s.
// fp32: the weight's values are bf16 numbers, and X is the sum of three bf16 parts (mx4_split_kernel), which multiply the same
// decoded weight; the first part's products have an accumulator of their own (relative error 4e-8 at 384 of the contraction,
// 2e-7 at 4096; 1.2e-6 at 384 with one accumulator).
#include "mx4_pair.cuh"

namespace spops {
namespace {

constexpr int kCodeBoxes = 4;           // of 256 of the contraction: whole 128-byte lines
constexpr int kMaxSlots = kCodeBoxes;  // stages of X and of the decoded weight: a stage's box lies at most a round of boxes before it
constexpr uint32_t kXRing = 128 * 1024;
constexpr int kTmemCols = 512;

// A stage holds kSub times 64 of the contraction (four, or two, which leaves room for tiles of more than 128 tokens; fp32: two, or
// one), and X in kParts parts. Warps 0 to 3 finish (a TMEM lane quarter each), then
// groups of four decode, one warp loads X, one multiplies, one loads codes.
template <typename Out, int kSub_>
struct FwdCfg {
    static constexpr int kParts = sizeof(Out) == 4 ? 3 : 1, kSub = kSub_;
    static constexpr int kAccs = kParts == 1 ? 1 : 2;  // of a tile
    static constexpr int kGroups = 4;  // at most
    static constexpr int kOutBufs = kParts == 1 ? 4 : 2;  // (what fits)
    static constexpr int kLoadWarp = 4 + 4 * kGroups, kMmaWarp = kLoadWarp + 1, kCodeWarp = kLoadWarp + 2, kThreads = 32 * (kCodeWarp + 1);
    static constexpr int kBoxStages = 4 / kSub;
    static constexpr uint32_t kBoxBytes = kFeatures * 128, kCodesAt = kXRing, kOutAt = kCodesAt + kCodeBoxes * kBoxBytes;
    static constexpr uint32_t kOutBytes = kOutTokens * 32 * sizeof(Out), kBarsAt = kOutAt + 4 * kOutBufs * kOutBytes, kSmem = kBarsAt + 1024;
    static_assert((kParts == 1 ? kMaxTokens : kMaxTokens / 2) * kFeatures * 4u <= kXRing, "the partial sums fit");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// D (+)= A B^T over both CTAs of the pair, A [128 features x 16 of the contraction] of each in its tensor memory.
__device__ __forceinline__ void pair_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_codes(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// 16 columns of the thread's lane; tmem_stored waits for all of them.
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void mbar_arrive_count(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <typename T, typename Out, int kSub>
__global__ void __launch_bounds__(FwdCfg<Out, kSub>::kThreads, 1)
mx4_fwd_kernel(const TileArgs g, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const __grid_constant__ CUtensorMap map_y) {
    using Cfg = FwdCfg<Out, kSub>;
    constexpr int kLoadWarp = Cfg::kLoadWarp, kMmaWarp = Cfg::kMmaWarp, kCodeWarp = Cfg::kCodeWarp, kParts = Cfg::kParts;
    constexpr int kBlocks = 2 * kSub, kWords = (kBlocks + 3) / 4;  // of a row and stage; words of its scales
    // No static shared memory, so the dynamic part starts on the 1 KB boundary that the swizzled tiles need (checked).
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    struct Shared {
        uint64_t full[kMaxSlots], empty[kMaxSlots], codes_full[kCodeBoxes], codes_empty[kCodeBoxes], acc_full[2], acc_empty[2];
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
    const uint32_t stages = g.stages, x_bytes = (uint32_t)g.nt * 64, stage_bytes = kSub * kParts * x_bytes;
    const Share me(g);
    const uint32_t a_col = (uint32_t)(g.bufs * Cfg::kAccs * g.nt);  // the decoded weight's columns lie behind the accumulators'
    if (tid == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 2 * 4 + 1);  // decoding warps of the pair, the loader
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < kCodeBoxes; ++i) {
            mbar_init(smem_u32(&sh.codes_full[i]), 1);
            mbar_init(smem_u32(&sh.codes_empty[i]), 4 * Cfg::kBoxStages);  // a group's warps for each stage
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_empty[i]), 2 * 4);  // finishing warps of the pair
        }
        sh.failed = 0;
        fence_mbar_init();
    }
    if (tid == 32 * kCodeWarp) {
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_x);
        tma_prefetch_map(&map_y);
    }
    __syncthreads();
    pdl_wait();
    if (warp == kMmaWarp) pair_alloc(smem_u32(&sh.tmem), kTmemCols);
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
                if (issues && ok) {
                    if (me.half == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[s]), 2 * kSub * kParts * x_bytes);
#pragma unroll
                    for (int h = 0; h < kSub * kParts; ++h)  // (the parts of X lie one behind the other)
                        pair_tma_load_2d(sbase + s * stage_bytes + h * x_bytes, &map_x,
                                         (c * kSub + h % kSub) * kKC + h / kSub * g.part, at.t0 + me.half * (g.nt / 2), full + s * 8);
                }
                __syncwarp();
                if (++s == stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp == kCodeWarp) {
        const bool issues = elect_one();
        uint32_t s = 0, ph = 1;
        for (int i = 0; i < me.mine; ++i) {
            const Place at = place_of(g, me.cid + i * me.ncl, me.half);
            for (int c = me.c0; c < me.c1; c += Cfg::kBoxStages) {
                const bool ok = wait(smem_u32(&sh.codes_empty[s]), ph);
                if (issues && ok) {
                    const uint32_t bar = smem_u32(&sh.codes_full[s]);
                    mbar_arrive_expect_tx(bar, Cfg::kBoxBytes);
                    tma_load_codes(sbase + Cfg::kCodesAt + s * Cfg::kBoxBytes, &map_w, c * (32 * kSub), at.f0, bar);
                }
                __syncwarp();
                if (++s == kCodeBoxes) {
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
            const uint64_t b0 = tc::smem_desc_sw128(sbase, 0, 1024);
            const bool issues = elect_one();
            uint32_t s = 0, ph = 0, acc_ph = 1;
            int buf = 0;
            for (int i = 0; i < me.mine; ++i) {
                const uint32_t d = tmem + (uint32_t)(buf * Cfg::kAccs * g.nt);
                wait(smem_u32(&sh.acc_empty[buf]), acc_ph);
                tc::fence_after_sync();
                for (int c = 0; c < me.per; ++c) {
                    wait(smem_u32(&sh.full[s]), ph);
                    tc::fence_after_sync();
                    if (issues) {
                        const uint32_t a = tmem + a_col + s * (32 * kSub);
                        const uint64_t b = b0 + s * (stage_bytes / 16);
#pragma unroll
                        for (int h = 0; h < kSub * kParts; ++h)
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // 16 of the contraction: 8 columns, 32 bytes
                                pair_mma_f16_ts(h < kSub ? d : d + (uint32_t)g.nt, a + h % kSub * 32 + k * 8, b + h * (x_bytes / 16) + k * 2,
                                                g.idesc, c > 0 || k > 0 || (h != 0 && h != kSub));
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
                if (++buf == g.bufs) {
                    buf = 0;
                    acc_ph ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4 && (warp - 4) >> 2 < g.groups) {
        // A group of four warps takes every g.groups-th stage, so that the steps of one stage (codes that arrive, decoding,
        // the stores, the message) overlap with those of others. A thread has a row of the 128.
        const int r = tid & 127, group = (warp - 4) >> 2, groups = g.groups;
        const uint32_t from = sbase + Cfg::kCodesAt + (uint32_t)r * 128u, flip = (uint32_t)(r & 7);  // (the codes' swizzle)
        const uint32_t to = tmem + a_col + ((uint32_t)(warp & 3) << 21);
        const uint32_t full = cluster_map(smem_u32(&sh.full[0]), me.lead);
        // The next stage to ask scales for: number ac of tile ai; a row or a block that is not there has codes of zeros, and a
        // scale of one here.
        constexpr uint32_t kOnes = 0x7f7f7f7fu;
        const bool whole = ((g.blocks | (int64_t)reinterpret_cast<uintptr_t>(g.scales)) & (kBlocks - 1)) == 0;
        int ai = 0, ac = group;
        const uint8_t* ps = g.scales;
        bool in = false;
        auto aim = [&]() {
            while (ac >= me.per && ai < me.mine) {
                ac -= me.per;
                ++ai;
            }
            in = false;
            if (ai >= me.mine) return;
            const int row = place_of(g, me.cid + ai * me.ncl, me.half).f0 + r;
            in = row < g.rows;
            ps = g.scales + (int64_t)row * g.blocks + (int64_t)(me.c0 + ac) * kBlocks;
        };
        struct Scales {
            uint32_t w[kWords];
        };
        auto ask = [&]() {
            Scales b;
#pragma unroll
            for (int k = 0; k < kWords; ++k) b.w[k] = kOnes;
            if (in) {
                if (whole) {
                    if constexpr (kSub == 4) {
                        const uint2 v = *reinterpret_cast<const uint2*>(ps);
                        b.w[0] = v.x;
                        b.w[1] = v.y;
                    } else if constexpr (kSub == 2) {
                        b.w[0] = *reinterpret_cast<const uint32_t*>(ps);
                    } else {
                        b.w[0] = kOnes << 16 | *reinterpret_cast<const uint16_t*>(ps);
                    }
                } else {
                    const int64_t blk = (int64_t)(me.c0 + ac) * kBlocks;
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x)
                        if (blk + x < g.blocks)
                            b.w[x / 4] = (b.w[x / 4] & ~(255u << (8 * (x % 4)))) | (uint32_t)ps[x] << (8 * (x % 4));
                }
            }
            ac += groups;
            ps += groups * kBlocks;
            if (ac >= me.per) aim();
            return b;
        };
        aim();
        Scales b = ask();
        uint32_t s = group, ph = 1;
        // The stage at hand: number c of this pair's tile; the boxes of codes before its tile.
        const uint32_t tile_boxes = (uint32_t)(me.per - 1) / Cfg::kBoxStages + 1;
        uint32_t boxes = 0;
        int c = group;
        for (int64_t left = (int64_t)me.mine * me.per - group; left > 0; left -= groups) {
            while (c >= me.per) {
                c -= me.per;
                boxes += tile_boxes;
            }
            const uint32_t box = boxes + (uint32_t)c / Cfg::kBoxStages, cs = box % kCodeBoxes, in_box = (uint32_t)c % Cfg::kBoxStages;
            // The slot first: then the stage before it there has been multiplied, so all stages up to that one had their codes, those
            // of the box before this one in its place among them (kMaxSlots), and the parity can mean no earlier phase. (Boxes
            // arrive in any order: with the codes first, a box that was not there passed for one.)
            const bool free = wait(smem_u32(&sh.empty[s]), ph);
            const bool ok = __all_sync(0xffffffffu, free && wait(smem_u32(&sh.codes_full[cs]), box / kCodeBoxes & 1));
            if (ok) {
                tc::fence_after_sync();
                const uint32_t codes = from + cs * Cfg::kBoxBytes, first = in_box * kBlocks, col = to + s * (32 * kSub);
                uint32_t rare = 0;  // scales but 2^-14 to 2
#pragma unroll
                for (int k = 0; k < kWords; ++k) rare |= (b.w[k] - 0x71717171u) & 0xf0f0f0f0u;
                if (__all_sync(0xffffffffu, rare == 0)) {
#pragma unroll
                    for (int x = 0; x < kBlocks; ++x) {
                        const uint4 w = ld_shared_v4(codes + ((flip ^ (first + x)) << 4));
                        const uint32_t f = __byte_perm(b.w[x / 4] - 0x70707070u, 0, 0x0404 | (x % 4) << 12 | (x % 4) << 4) << 2;  // as fp16
                        uint32_t v[16];
                        mx4::decode8<T>(w.x, f, reinterpret_cast<uint32_t(&)[4]>(v[0]));
                        mx4::decode8<T>(w.y, f, reinterpret_cast<uint32_t(&)[4]>(v[4]));
                        mx4::decode8<T>(w.z, f, reinterpret_cast<uint32_t(&)[4]>(v[8]));
                        mx4::decode8<T>(w.w, f, reinterpret_cast<uint32_t(&)[4]>(v[12]));
                        tmem_put16(col + x * 16, v);
                    }
                } else {
#pragma unroll 1
                    for (int x = 0; x < kBlocks; ++x) {
                        const uint4 w = ld_shared_v4(codes + ((flip ^ (first + x)) << 4));
                        const uint32_t e = ((kWords > 1 && x >= 4 ? b.w[kWords - 1] : b.w[0]) >> (8 * (x & 3))) & 255u;
                        uint32_t v[16];
                        const bool plain = mx4::plain(e) || (e != 255 && (w.x | w.y | w.z | w.w) == 0);  // (or nothing but zeros)
                        if (__all_sync(0xffffffffu, plain)) {
                            const uint32_t f = mx4::plain(e) ? mx4::factor2(e) : 0;
                            mx4::decode8<T>(w.x, f, reinterpret_cast<uint32_t(&)[4]>(v[0]));
                            mx4::decode8<T>(w.y, f, reinterpret_cast<uint32_t(&)[4]>(v[4]));
                            mx4::decode8<T>(w.z, f, reinterpret_cast<uint32_t(&)[4]>(v[8]));
                            mx4::decode8<T>(w.w, f, reinterpret_cast<uint32_t(&)[4]>(v[12]));
                        } else {
                            mx4::decode8_any<T>(w.x, e, reinterpret_cast<uint32_t(&)[4]>(v[0]));
                            mx4::decode8_any<T>(w.y, e, reinterpret_cast<uint32_t(&)[4]>(v[4]));
                            mx4::decode8_any<T>(w.z, e, reinterpret_cast<uint32_t(&)[4]>(v[8]));
                            mx4::decode8_any<T>(w.w, e, reinterpret_cast<uint32_t(&)[4]>(v[12]));
                        }
                        tmem_put16(col + x * 16, v);
                    }
                }
                tmem_stored();
                tc::fence_before_sync();
            }
            __syncwarp();
            if (lane == 0 && ok) {
                pair_arrive(full + s * 8);
                // (for the stages that the tile's last box has not, as well)
                mbar_arrive_count(smem_u32(&sh.codes_empty[cs]), c == me.per - 1 ? Cfg::kBoxStages - in_box : 1);
            }
            __syncwarp();
            b = ask();  // (behind the message, which the multiplying warp waits for)
            s += groups;
            if (s >= stages) {
                s -= stages;
                ph ^= 1;
            }
            c += groups;
        }
    } else if (warp < 4) {
        finish_tiles<Out, Cfg::kOutBufs>(g, me, map_y, wait, sh.acc_full, sh.acc_empty, sbase, Cfg::kOutAt, tmem, Cfg::kAccs * g.nt, warp, lane);
    }
    if (me.splits > 1) {
        cluster_sync();
        if (!sh.failed && me.mine > 0) add_splits<Out>(g, me, sbase, Cfg::kThreads);
    }
    if (sh.failed)  // copies and products that are still in flight
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < kDrainNs;) {
        }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // the pair's products are done, nobody reads this CTA's memory any more
    if (warp == kMmaWarp) pair_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side

// Stages that X's ring and the columns that `bufs` tiles' accumulators leave have room for.
template <typename Cfg>
int slots(int nt, int bufs) {
    const int cols = (kTmemCols - bufs * Cfg::kAccs * nt) / (32 * Cfg::kSub), x = (int)(kXRing / (Cfg::kSub * Cfg::kParts * nt * 64));
    const int n = cols < x ? cols : x;
    return n < kMaxSlots ? n : kMaxSlots;
}
// A second accumulator, so that a tile's sums leave while the next one's products run: where a pair has several tiles and the
// weight keeps three stages (8192 tokens, 2048 -> 8192: 150 us with 160 tokens a tile and two, 165 with 256 and one).
template <typename Cfg>
bool two_buffers(int nt, int splits, int64_t tiles, int64_t at_once) {
    return splits == 1 && tiles > at_once && slots<Cfg>(nt, 2) >= 3;
}

// Tokens per tile, splits of the contraction and 64s of it in a stage with the least estimated time in us, fitted to sweeps over
// them (384 to 11008 features, 6 to 172 times 64 of the contraction, 9 to 8192 tokens): a stage takes its decoding and its
// messages (kLeast), or its products, and 15 % more where the ring has three of 128; tiles follow each other, with one accumulator after
// its sums have left; with splits, every wave of clusters begins anew and adds its sums. (Stages of 256 as those of 128, 64 tokens
// 4096 -> 11008: 14.5 us and 16.3, fp16 12.6 and 14.7, 128 tokens 16.0 and 17.2; 160 tokens leave no room for three.)
template <typename Cfg>
void choose(int64_t tokens, int64_t F, int64_t C, const int (&at_once)[kMaxSplits + 1], double& least, Shape& best) {
    constexpr int kSub = Cfg::kSub;
    constexpr double kLeast = kSub == 1 ? 0.335 : Cfg::kParts > 1 ? 0.5 : kSub == 2 ? 0.335 : 0.535;
    const int most = Cfg::kParts > 1 ? (kSub == 1 ? 128 : 96) : kSub == 2 ? kMaxTokens : 128;
    const int64_t ftiles = (F + 2 * kFeatures - 1) / (2 * kFeatures), stages = (C + kSub * kKC - 1) / (kSub * kKC);
    for (int nt = 32; nt <= most; nt += 32) {
        const double products = kSub * (Cfg::kParts == 1 ? 0.00111 : 0.0042) * nt, stage = products > kLeast ? products : kLeast;
        for (int s = 1; s <= kMaxSplits && s <= stages; ++s) {
            const int64_t tiles = ftiles * ((tokens + nt - 1) / nt);
            const double waves = (double)((tiles + at_once[s] - 1) / at_once[s]), steps = (double)((stages + s - 1) / s);
            double t;
            if (s > 1) {
                t = waves * (4.4 + 0.3 * s + 0.015 * nt + steps * stage);
            } else {
                const bool two = two_buffers<Cfg>(nt, 1, tiles, at_once[1]);
                t = 3.8 + 0.0095 * nt + waves * steps * stage * (two && kSub == 2 && slots<Cfg>(nt, 2) == 3 ? 1.15 : 1.0) +
                    (waves - 1) * (two ? 0.25 : 0.4 + 0.009 * nt);
            }
            if (t < least) {
                least = t;
                best = {nt, s, kSub, at_once[s]};
            }
        }
    }
}

template <typename T, typename Out, int kSub>
cudaError_t run_shape(const Mx4Args& a, Shape shape, cudaStream_t s) {
    using Cfg = FwdCfg<Out, kSub>;
    auto kern = mx4_fwd_kernel<T, Out, kSub>;
    static bool done[64];
    const cudaError_t e = allow_smem(kern, Cfg::kSmem, done);
    if (e != cudaSuccess) return e;
    TileArgs g{};
    CUtensorMap mw, mx, my;
    if (!tile_args<T, Out>(g, a, a.rows, a.cols, shape, Cfg::kParts, &mx, &my) ||
        !encode_matrix<uint8_t>(&mw, a.codes, a.rows, g.blocks * 16, g.blocks * 16, 128, kFeatures, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    g.bufs = two_buffers<Cfg>(shape.nt, shape.splits, g.tiles, shape.at_once) ? 2 : 1;
    g.stages = slots<Cfg>(shape.nt, g.bufs);
    g.groups = min(g.stages, Cfg::kGroups);  // (a group's next stage is at most one round of the ring away)
    g.idesc = tc::instr_desc_f16(std::is_same<T, __nv_bfloat16>::value ? 1u : 0u, 0u, 0u, 2 * kFeatures, (uint32_t)shape.nt);
    const int c = 2 * shape.splits, clusters = shape.splits > 1 || g.tiles < shape.at_once ? g.tiles : shape.at_once;
    count_launches(1);
    return launch_pdl_cluster(kern, dim3((unsigned)(clusters * c)), dim3(Cfg::kThreads), Cfg::kSmem, (unsigned)c, s, g, mw, mx, my);
}

template <typename T, typename Out>
cudaError_t run_tiles(const Mx4Args& a, cudaStream_t s) {
    constexpr int kSub = sizeof(Out) == 4 ? 1 : 2;
    using Cfg = FwdCfg<Out, kSub>;
    static int known[64][kMaxSplits + 1];
    static bool done[64];
    int at_once[kMaxSplits + 1];
    // (as many of the kernel with other stages: one CTA fills an SM)
    const cudaError_t e = count_clusters(mx4_fwd_kernel<T, Out, kSub>, Cfg::kThreads, Cfg::kSmem, at_once, known, done);
    if (e != cudaSuccess) return e;
    double least = 1e300;
    Shape shape{};
    choose<Cfg>(a.tokens, a.rows, a.cols, at_once, least, shape);
    choose<FwdCfg<Out, 2 * kSub>>(a.tokens, a.rows, a.cols, at_once, least, shape);
    if (shape.sub == kSub) return run_shape<T, Out, kSub>(a, shape, s);
    return run_shape<T, Out, 2 * kSub>(a, shape, s);
}

}  // namespace

cudaError_t launch_mx4_forward(int dt, const Mx4Args& a, cudaStream_t s) {
    if (dt == kF32) return run_tiles<__nv_bfloat16, float>(a, s);
    return dt == kF16 ? run_tiles<__half, __half>(a, s) : run_tiles<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace spops
