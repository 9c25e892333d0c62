// adjust.h -- the adjusted scores' parameters, shared by the C ABI
// (adjust_api.cu) and the kernels (adjust_kernel.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mr_internal.h"

namespace mr {

struct AdjustParams {
    const void* x[kMaxRanks];       // the scores of rank r's columns
    const void* in[kMaxRanks];      // what is changed: the scores, or (gradient) what comes back to the adjusted ones
    void* out[kMaxRanks];
    uint64_t ldx[kMaxRanks];        // elements from a row to the next
    uint64_t ldi[kMaxRanks];
    uint64_t ldo[kMaxRanks];
    uint32_t col0[kMaxRanks + 1];   // first column of each rank
    uint64_t rows;
    int W;
    uint32_t vocab;
    uint32_t window;                // columns a CTA takes of a row at a time
    uint32_t windows;               // windows a row
    // the history of each row (null: none)
    const long long* history;
    uint64_t ld_history;            // entries a row
    const long long* n_history;     // null: ld_history
    const long long* n_prompt;      // null: 0
    const float* repetition;        // null: 1
    const float* frequency;         // null: 0
    const float* presence;          // null: 0
    // biases (null: none)
    const long long* bias_ids;
    const float* bias;
    uint32_t K;
    const uint32_t* mask;           // null: every token is allowed
    uint64_t ld_mask;               // 32-bit words from a row to the next
    uint32_t listed;                // columns of a window that the lists may name, at most
    float ranks_per_col;            // W / vocab
};

// Where a column of the window stands in the history: bit 31, it is there;
// bit 30, it has a bias; below, how often the model has said it.
constexpr uint32_t kSeen = 1u << 31, kBiased = 1u << 30, kTimes = kBiased - 1;

// The listed columns of a window are kept in a hash table in shared memory: a
// key, a word and a place in the list of the slots taken (at most four fifths),
// beside the window's mask.  Windows are a multiple of 1024 columns.  Up to
// kMostListed entries of a row's lists, of which each may name another column,
// two CTAs fit an SM and wide windows are faster; longer lists take windows of
// kNarrowWindow columns, each of which has a place (512 x 131072 bf16: histories
// of 4096 94 us in windows of 32768, 230 in windows of 4096; of 8192 179 and 302;
// of 12000, one CTA an SM, 379 and 370).
constexpr uint32_t kMostListed = 8448, kNarrowWindow = 4096;
__host__ __device__ constexpr uint32_t adjust_slots(uint32_t listed) { return (listed * 5 / 4 + 2) / 2 * 2; }
constexpr size_t adjust_smem(uint32_t listed, uint32_t window) { return (size_t)10 * adjust_slots(listed) + window / 8; }

// CTAs an SM, and vectors whose loads a thread has in flight.  4096 x 131072
// bf16 with lists and a mask: 439 us at 6 CTAs with 2 vectors, 430 at 5 with 4,
// 461 at 4 with 4; with a mask alone 344 at 6 with 2, 372 at 5 with 4.
__host__ __device__ constexpr int adjust_ctas(bool lists) { return lists ? 5 : 6; }
__host__ __device__ constexpr uint32_t adjust_ahead(bool lists) { return lists ? 4 : 2; }
cudaError_t launch_adjust(const AdjustParams& P, int dtype, bool grad, dim3 grid, cudaStream_t s);

}  // namespace mr
