// embedding.h -- the embedding lookup's and its gradient's parameters, shared
// by the C ABI (embedding_api.cu) and the kernels (embedding_kernel.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mr_internal.h"

namespace mr {

// A table [vocab, hidden] whose row v lies in the buffer of the rank whose
// chunk [floor(r*vocab/W), floor((r+1)*vocab/W)) it falls in.
struct TableRows {
    void* row0[kMaxRanks];          // rank r's first row
    uint64_t ld[kMaxRanks];         // elements from a row to the next
    uint32_t first[kMaxRanks + 1];  // that row's number
    int W;
    uint32_t vocab;
    float ranks_per_row;            // W / vocab
};

struct EmbeddingParams {
    TableRows table;
    const long long* ids;
    uint64_t rows, hidden;
    float scale;
    void* out;
    uint64_t ld_out;
    uint64_t parts;                 // warps a row
};

struct EmbeddingGradParams {
    TableRows grad;
    const void* g;
    uint64_t ld_g;
    const long long* ids;
    uint64_t rows, hidden;
    float scale;
    int accumulate;
    uint64_t slabs;                 // warps a row: kSlab columns each
};

constexpr int kLookupVectors = 4;   // 16-byte vectors a lane takes of a row at a time
constexpr int kSlab = 256;          // columns that a warp of the gradient sums

// vec: every row of the table and of the output starts on a 16-byte boundary
// and holds whole vectors.
cudaError_t launch_embedding(const EmbeddingParams& P, int dtype, bool vec, dim3 grid, cudaStream_t s);
cudaError_t launch_embedding_grad(const EmbeddingGradParams& P, int g_dtype, int table_dtype, bool vec, dim3 grid, cudaStream_t s);

}  // namespace mr
