// Products with a microscaled 4-bit weight in fp32, any size and alignment, on the CUDA cores.
//
// mx4_general_kernel  Y = X W^T (forward) or X W (back), fp32 sums. A CTA has 64 tokens x 64 features and walks the
// contraction in steps of 32: the weight's values and X go to shared memory, a thread
// holds 4 x 4 sums. Bound by the FMA pipe and its operands' shared-memory reads.
#include "internal.h"
#include "mx4.cuh"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kTile = 64, kStep = 32, kThreads = 256;
constexpr int kPitch = kTile + 4;  // fp32 words of a shared row: 16-byte aligned, columns on other banks

template <bool kBack>
__global__ void __launch_bounds__(kThreads) mx4_general_kernel(Mx4Args g) {
    __shared__ __align__(16) float xs[kStep][kPitch], ws[kStep][kPitch];
    const int tid = threadIdx.x;
    const int F = kBack ? g.cols : g.rows, C = kBack ? g.rows : g.cols;
    const int64_t nb = (g.cols + kMx4Block - 1) / kMx4Block;
    const int64_t ft = ((int64_t)F + kTile - 1) / kTile, tt = ((int64_t)g.tokens + kTile - 1) / kTile;
    const float* X = static_cast<const float*>(g.X);
    float* Y = static_cast<float*>(g.Y);
    pdl_trigger();
    pdl_wait();
    for (int64_t tile = blockIdx.x; tile < ft * tt; tile += gridDim.x) {
        const int64_t f0 = tile % ft * kTile, t0 = tile / ft * kTile;
        const int ti = tid / 16 * 4, fi = tid % 16 * 4;
        float acc[4][4] = {};
        for (int64_t c0 = 0; c0 < C; c0 += kStep) {
            // eight codes a thread
            const int r = kBack ? tid / 8 : tid / 4, e = (kBack ? tid % 8 : tid % 4) * 8;
            const int64_t row = (kBack ? c0 : f0) + r, col = (kBack ? f0 : c0) + e;
            uint32_t code = 0, b = 0;
            if (row < g.rows && col < g.cols) {
                code = *reinterpret_cast<const uint32_t*>(g.codes + row * nb * 16 + col / 2);
                b = g.scales[row * nb + col / kMx4Block];
            }
            const float s = mx4::scale_f32(b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = mx4::value_f32(code >> (4 * i), s);
                if (kBack) ws[r][e + i] = v;
                else ws[e + i][r] = v;
            }
#pragma unroll
            for (int i = 0; i < kTile * kStep / kThreads; ++i) {
                const int t = tid / 32 + 8 * i, c = tid % 32;
                const bool in = t0 + t < g.tokens && c0 + c < C;
                xs[c][t] = in ? X[(t0 + t) * g.ldx + c0 + c] : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < kStep; ++c) {
                const float4 x = *reinterpret_cast<const float4*>(&xs[c][ti]);
                const float4 w = *reinterpret_cast<const float4*>(&ws[c][fi]);
                const float xv[4] = {x.x, x.y, x.z, x.w}, wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv[i], wv[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t0 + ti + i < g.tokens && f0 + fi + j < F)
                    Y[(t0 + ti + i) * g.ldy + f0 + fi + j] = acc[i][j];
    }
}

}  // namespace

cudaError_t launch_mx4_general(bool back, const Mx4Args& a, cudaStream_t s) {
    const int64_t F = back ? a.cols : a.rows;
    const int64_t tiles = ((F + kTile - 1) / kTile) * (((int64_t)a.tokens + kTile - 1) / kTile);
    const unsigned grid = (unsigned)min64(tiles, 1 << 20);
    count_launches(1);
    return back ? launch_pdl(mx4_general_kernel<true>, dim3(grid), dim3(kThreads), 0, s, a)
                : launch_pdl(mx4_general_kernel<false>, dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace spops
