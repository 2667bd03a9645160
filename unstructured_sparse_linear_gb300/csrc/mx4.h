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

// General kernel: any type, size and alignment.
cudaError_t launch_mx4_general(int dt, bool back, const Mx4Args& a, cudaStream_t s);

// Tensor-core kernel (fp16 / bf16, rows of X and Y that begin on 16-byte boundaries).
bool mx4_tiles_ok(int dt, const Mx4Args& a);
cudaError_t launch_mx4_tiles(int dt, bool back, const Mx4Args& a, cudaStream_t s);

// The dispatch between the kernels.
cudaError_t launch_mx4_product(int dt, bool back, const Mx4Args& a, cudaStream_t s);

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
