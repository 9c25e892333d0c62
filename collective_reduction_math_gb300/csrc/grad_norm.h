// grad_norm.h -- parameters of the gradient norm and the clipping, shared by
// the C ABI (grad_norm_api.cu) and the kernels (grad_norm_kernel.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mr_internal.h"

namespace mr {

// A launch takes up to kListTensors tensors; longer lists take several.
constexpr int kListTensors = 512;

// A tensor is cut into tiles of kTileBytes, counted from its start rounded
// down to 16 bytes.  8 vectors a thread and 4 CTAs an SM: 1.5e9 bf16 in 427 us
// (105 % of the copy rate; with chains of multiply-adds for sums it was 435, with
// 4 vectors 483, and with 6 CTAs an SM besides 692).
constexpr uint32_t kTileVectors = 8;        // 16-byte vectors a thread
constexpr uint32_t kTileBytes = kThreads * kTileVectors * 16;
constexpr int kNormCtas = 4;                // CTAs an SM

struct TensorList {
    const void* in[kListTensors];
    void* out[kListTensors];                // clipping: where the clipped tensor goes (may be in)
    uint64_t n[kListTensors];               // elements; bit 63: bf16
    uint32_t tile0[kListTensors + 1];       // tiles of the tensors before
    int count;
};
constexpr uint64_t kIsBf16 = 1ull << 63;

// A sum as two floats: the sum, and what its additions lost.
struct SumPair {
    float hi, lo;
};
// What a thread, a CTA or all have summed, each element in one of the three: x^2, (x 2^-90)^2 or (x 2^90)^2.
struct NormPart {
    SumPair mid, big, small;
};
constexpr int kMostNormGrid = 1024;         // parts of a launch at most
// Up to as many parts every CTA of the clipping joins for itself, while its first
// tile is on its way; more, which only lists of several launches have, one CTA
// joins in a launch before.  Else a call's time grew with the square of its list
// (tensors of 2000 bf16: 1400 of them 49 us without that launch and 48 with it,
// 2048 66 and 62, 4096 142 and 115, 10000 470 and 277; 1024, at this limit, 34 and 35).
constexpr int kMostOwnJoin = kMostNormGrid;

struct NormOfParts {
    const NormPart* parts;
    int count;
    float max_norm;
    float* norm;        // may be null
    NormPart* all;      // where the join puts them together; may be null, and the first of them
};

cudaError_t launch_norm_parts(const TensorList& L, NormPart* parts, dim3 grid, cudaStream_t s);
cudaError_t launch_norm_join(const NormOfParts& N, cudaStream_t s);
cudaError_t launch_clip(const TensorList& L, const NormOfParts& N, dim3 grid, cudaStream_t s);

}  // namespace mr
