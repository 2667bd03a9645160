// Low-rank adapters of many requests: the plan of a batch (which tokens use which adapter)
// and the launchers of the operators that walk it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace spops {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraTile = 128;  // rows of one adapter in a tensor-core tile
constexpr int kLoraRows = 8;    // rows of one adapter in a tile of the general kernels

// One tile: `rows` consecutive positions of the plan's order, all of one adapter (-1: tokens
// without one). tok0 is the first token when the tile's tokens are consecutive, else -1.
struct LoraTile {
    int32_t adapter, pos0, rows, tok0;
};

// A tile of the general kernels, with its tokens in place: these serve small batches too, where
// every dependent load counts.
struct alignas(16) LoraSmall {
    int32_t adapter, rows;
    int32_t tok[kLoraRows];
    int32_t pad[2];
};

constexpr int kLoraHdr = 16;  // header words: counts[kLoraCnt...]
enum LoraCount { kLoraCntTiles = 0, kLoraCntSmall = 1, kLoraCntWith = 2 };

// Views of a plan buffer (16-byte aligned). order: the tokens sorted by adapter (stable;
// tokens without an adapter last); off[a] .. off[a + 1]: adapter a's positions (off[n] = tokens
// that have one); tiles: tiles of up to kLoraTile rows, adapters only; small: tiles of up to
// kLoraRows rows, then those of the tokens without an adapter.
struct LoraPlanView {
    int32_t* counts;
    int32_t* order;
    int32_t* tmp;     // [tokens] scratch of the sort
    int32_t* off;     // [n + 2]
    int32_t* tstart;  // [n + 2] scratch: first tile of each adapter
    int32_t* aorder;  // [n] the adapters, those with the most tokens first
    LoraTile* tiles;
    LoraSmall* small;
    int32_t tokens, n;
};

// The most tiles of up to `rows` rows that `tokens` tokens in `groups` groups can give: each group
// that has a token may end with a tile of one row.
inline int64_t lora_tiles_most(int32_t tokens, int64_t groups, int rows) {
    const int64_t m = tokens < groups ? tokens : groups;
    return (tokens - m) / rows + m;
}
// Slots of the two lists: adapters, and for the small tiles the tokens without one too.
inline int64_t lora_tiles_cap(int32_t tokens, int32_t n, int rows) {
    return lora_tiles_most(tokens, rows == kLoraRows ? (int64_t)n + 1 : n, rows);
}
inline size_t lora_words4(int64_t words) { return (size_t)((words + 3) / 4 * 4); }

inline size_t lora_plan_bytes(int32_t tokens, int32_t n) {
    return 4 * (kLoraHdr + 2 * lora_words4(tokens) + 3 * lora_words4((int64_t)n + 2)) +
           sizeof(LoraTile) * (size_t)lora_tiles_cap(tokens, n, kLoraTile) +
           sizeof(LoraSmall) * (size_t)lora_tiles_cap(tokens, n, kLoraRows);
}

inline LoraPlanView lora_plan_view(const void* plan, int32_t tokens, int32_t n) {
    int32_t* p = static_cast<int32_t*>(const_cast<void*>(plan));
    LoraPlanView v;
    v.counts = p;
    v.order = p + kLoraHdr;
    v.tmp = v.order + lora_words4(tokens);
    v.off = v.tmp + lora_words4(tokens);
    v.tstart = v.off + lora_words4((int64_t)n + 2);
    v.aorder = v.tstart + lora_words4((int64_t)n + 2);
    v.tiles = reinterpret_cast<LoraTile*>(v.aorder + lora_words4((int64_t)n + 2));
    v.small = reinterpret_cast<LoraSmall*>(v.tiles + lora_tiles_cap(tokens, n, kLoraTile));
    v.tokens = tokens;
    v.n = n;
    return v;
}

// O[t, :] = base[t, :] + s_a (U[t, :] W1_a) W2_a for every token t of adapter a, and
// P[t, :] = U[t, :] W1_a (unscaled). kb: back = false, the forward product (W1_a = A_a^T,
// W2_a = B_a^T); back = true, the input gradient (U = dY, W1_a = B_a, W2_a = A_a).
// O == nullptr: P only. base == nullptr: zeros. Tokens without an adapter: O = base, P = 0.
struct LoraArgs {
    const void* U = nullptr;
    int64_t ldu = 0;
    int32_t K = 0;           // columns of U
    const void* A = nullptr;  // [n, rank, in]
    const void* B = nullptr;  // [n, out, rank]
    const float* scale = nullptr;
    float scale_all = 1.f;
    int32_t rank = 0;
    const void* base = nullptr;
    int64_t ldb = 0;
    void* O = nullptr;
    int64_t ldo = 0;
    int32_t N = 0;        // columns of base and O
    float* P = nullptr;   // [tokens, rank]
};

// G_a[j, x] (or its transpose) = s_a sum over adapter a's tokens t of P[t, j] U[t, x].
struct LoraWgradArgs {
    const void* U = nullptr;
    int64_t ldu = 0;
    int32_t N = 0;            // columns of U
    const float* P = nullptr;  // [tokens, rank]
    void* G = nullptr;         // [n, rank, N], or [n, N, rank] when rank_minor
    bool rank_minor = false;
    bool dependent = false;  // P is written by the launch directly before (else by an earlier one)
};

cudaError_t launch_lora_plan(const int32_t* ids, const LoraPlanView& v, cudaStream_t s);
// General kernels: any type, size and alignment.
cudaError_t launch_lora_rows(int dt, bool back, const LoraArgs& a, const LoraPlanView& v, cudaStream_t s);
cudaError_t launch_lora_wgrad_rows(int dt, const LoraWgradArgs* w, int nw, int32_t rank, const float* scale,
                                   float scale_all, const LoraPlanView& v, cudaStream_t s);

// Tensor-core kernels (fp16 / bf16, 16-byte rows).
bool lora_tiles_ok(int dt, const LoraArgs& a, const LoraPlanView& v);
cudaError_t launch_lora_tiles(int dt, bool back, const LoraArgs& a, const LoraPlanView& v, cudaStream_t s);
bool lora_wgrad_tiles_ok(int dt, const LoraWgradArgs* w, int nw);
cudaError_t launch_lora_wgrad_tiles(int dt, const LoraWgradArgs* w, int nw, int32_t rank, const float* scale,
                                    float scale_all, const LoraPlanView& v, bool after_lora, cudaStream_t s);

// Operators (the dispatch between the kernels). after_lora: launch_lora was the launch before
// this one, on the same stream and in the same call.
cudaError_t launch_lora(int dt, bool back, const LoraArgs& a, const LoraPlanView& v, cudaStream_t s);
cudaError_t launch_lora_wgrad(int dt, const LoraWgradArgs* w, int nw, int32_t rank, const float* scale,
                              float scale_all, const LoraPlanView& v, bool after_lora, cudaStream_t s);

}  // namespace spops
