// Microscaled 4-bit weights: launchers of their conversion and of their products.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace spops {

constexpr int kMx4Block = 32;  // values that share a scale

inline int64_t mx4_blocks(int64_t cols) { return (cols + kMx4Block - 1) / kMx4Block; }

// Y[t, f] = sum over c of X[t, c] V(f, c): V(f, c) = W[f, c] (back = false: X W^T, F = rows, C = cols),
// or W[c, f] (back = true: X W, F = cols, C = rows). W [rows, cols] as codes (16 bytes a block of 32) and
// scales (one byte a block).
struct Mx4Args {
    const void* X = nullptr;
    int64_t ldx = 0;
    const uint8_t* codes = nullptr;
    const uint8_t* scales = nullptr;
    void* Y = nullptr;
    int64_t ldy = 0;
    int32_t tokens = 0, rows = 0, cols = 0;
};

cudaError_t launch_mx4_quantize(int dt, const void* X, int64_t ldx, int32_t rows, int32_t cols, uint8_t* codes,
                                uint8_t* scales, cudaStream_t s);
cudaError_t launch_mx4_dequantize(int dt, const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t cols,
                                  void* Y, int64_t ldy, cudaStream_t s);

// fp16 / bf16. Forward for one token, and for up to eight (any alignment):
cudaError_t launch_mx4_vec(int dt, const Mx4Args& a, cudaStream_t s);
cudaError_t launch_mx4_rows(int dt, const Mx4Args& a, cudaStream_t s);
// On the tcgen05 tensor cores, where mx4_tile_rows holds for X and Y. fp32: X is its three bf16 parts, mx4_split_cols
// columns, each part's behind the others'.
cudaError_t launch_mx4_forward(int dt, const Mx4Args& a, cudaStream_t s);
cudaError_t launch_mx4_backward(int dt, const Mx4Args& a, cudaStream_t s);

// Rows as TMA loads and stores them: rows and addresses on 16-byte boundaries, whole 16 bytes (a store writes no less).
inline bool mx4_tile_rows(const void* p, int64_t ld, int64_t cols, int64_t es) {
    return cols * es % 16 == 0 && ld * es % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld < (1ll << 37);
}
inline int64_t mx4_split_cols(int64_t cols) { return 3 * ((cols + 127) / 128 * 128); }
// Bytes of a copy of Y [tokens, cols] with such rows, and of X (fp32: of its parts).
inline size_t mx4_y_bytes(int64_t tokens, int64_t cols, int64_t es) {
    return ((size_t)tokens * (size_t)((cols * es + 15) / 16 * 16) + 255) / 256 * 256;
}
inline size_t mx4_x_bytes(int64_t tokens, int64_t cols, int64_t es) {
    return es == 4 ? mx4_y_bytes(tokens, mx4_split_cols(cols), 2) : mx4_y_bytes(tokens, cols, es);
}

// The dispatch between the kernels. workspace: for the operands that need a copy (mx4_needs_copies).
bool mx4_needs_copies(int dt, bool back, const Mx4Args& a);
cudaError_t launch_mx4_product(int dt, bool back, const Mx4Args& a, void* workspace, cudaStream_t s);

// dropout.cu: Y = base + keep * X * factor. state (device, two words) replaces seed and call.
struct DropoutArgs {
    const void* X = nullptr;
    const void* base = nullptr;
    void* Y = nullptr;
    int64_t ldx = 0, ldb = 0, ldy = 0;
    const uint64_t* state = nullptr;
    uint64_t seed = 0, call = 0;
    uint32_t threshold = 0;  // of 65536: numbers below it are dropped
    int32_t rows = 0, cols = 0;
};
cudaError_t launch_dropout(int dt, const DropoutArgs& a, cudaStream_t s);

}  // namespace spops
