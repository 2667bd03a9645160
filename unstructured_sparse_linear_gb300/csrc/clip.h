// The global 2-norm of many gradients and their scaling by it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace spops {

// Bytes of one tensor that a CTA takes at a time: with the bytes before and behind it in their
// 16-byte granules at most 32 KB.
constexpr int kClipChunk = 32768 - 16;
constexpr int kClipMaxCtas = 1024;  // partial sums

// One gradient of a set. out == in: scaled in place. first: its first chunk in the set.
struct ClipEntry {
    const void* in;
    void* out;
    int64_t count;
    int64_t first;
    int32_t dtype;
    int32_t pad;
};

inline int64_t clip_chunks(int64_t count, size_t esize) {
    const int64_t per = kClipChunk / (int64_t)esize;
    return (count + per - 1) / per;
}
// A set: the count of CTAs that have come to the wait between the passes, then the entries.
constexpr size_t kGradSetHead = 64;
inline size_t grad_set_bytes(int64_t tensors) { return kGradSetHead + sizeof(ClipEntry) * (size_t)(tensors > 0 ? tensors : 1); }
inline unsigned long long* grad_set_arrived(void* set) { return static_cast<unsigned long long*>(set); }
inline ClipEntry* grad_set_entries(void* set) {
    return reinterpret_cast<ClipEntry*>(static_cast<char*>(set) + kGradSetHead);
}
inline size_t grad_norm_ws_bytes() { return sizeof(double) * kClipMaxCtas; }

constexpr int kClipFill = 64;  // entries per fill launch (kernel parameters)
struct ClipFill {
    ClipEntry e[kClipFill];
};

cudaError_t launch_grad_set_fill(void* set, int64_t at, const ClipFill& f, int n, cudaStream_t s);
// norm_out = the 2-norm of the set's inputs; scale: also out = in * min(1, max_norm / (norm + 1e-6)).
cudaError_t launch_grad_norm(void* set, int32_t tensors, int64_t chunks, bool in_place, bool scale,
                             double max_norm, float* norm_out, double* partial, cudaStream_t s);

}  // namespace spops
