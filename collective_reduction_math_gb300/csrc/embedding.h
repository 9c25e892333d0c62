// embedding.h -- the embedding lookup's and its gradient's parameters, shared
// by the C ABI (embedding_api.cu) and the kernels (embedding_kernel.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mr_internal.h"
#include "sort_plan.h"

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

// The gradient's tokens are sorted by their row and cut into units: runs of
// positions of one row, at most kUnit long, which a warp sums.
constexpr uint32_t kUnit = 32;
constexpr int kSortDigit = 10;          // bits sorted in a pass at most
struct Unit {
    uint32_t start;     // first position; kPart: one of several units of its row, kFirst: the first of them
    uint32_t row;
};
constexpr uint32_t kPart = 1u << 31, kFirst = 1u << 30, kStart = kFirst - 1;
struct SortCounts {
    uint32_t units, longs;      // units; rows of more than one
};

struct EmbeddingGradParams {
    TableRows grad;
    const void* g;
    uint64_t ld_g;
    const long long* ids;
    uint32_t rows;
    uint64_t hidden;
    float scale;
    int accumulate;
    uint32_t slabs;                 // warps a unit: kSlab columns each
    uint32_t passes, digit;         // of the sort, and bits in each
    uint32_t ahead;                 // rows of g asked for from L2 while the sort runs
    uint32_t cleared;               // table rows cleared meanwhile, a multiple of 8
    // the workspace
    SortCounts* counts;
    uint32_t* tokens;               // by position: the token
    Unit* units;                    // and one more, which starts behind the last position
    uint32_t* longs;                // first units of rows that have several
    uint32_t* present;              // a bit a row: it has a token
    float* partial;                 // sums of units of such rows: [slot][ld_partial]
    uint64_t ld_partial;
};
// The slot of a unit that is one of several.  Such units that are not first
// start kUnit apart, and so do first ones: two slots for each kUnit positions.
__host__ __device__ constexpr uint32_t partial_slot(uint32_t start, bool first) { return start / kUnit * 2 + (first ? 1 : 0); }

constexpr int kLookupVectors = 4;   // 16-byte vectors a lane takes of a row at a time
constexpr int kSlab = 256;          // columns that a warp of the gradient sums
constexpr uint32_t kFillBytes = 4096;   // of a row without tokens, that a warp clears at a time

// The buffer row of table row v (v < vocab): an estimate of its rank, put right.
#ifdef __CUDACC__
__device__ __forceinline__ char* row_of(const TableRows& T, uint32_t v, int bytes) {
    int r = 0;
    if (T.W > 1) {
        r = min(T.W - 1, (int)((float)v * T.ranks_per_row));
        while (T.first[r] > v) --r;
        while (T.first[r + 1] <= v) ++r;
    }
    return static_cast<char*>(T.row0[r]) + (uint64_t)(v - T.first[r]) * T.ld[r] * bytes;
}
#endif

// vec: every row of the table and of the output starts on a 16-byte boundary
// and holds whole vectors.
cudaError_t launch_embedding(const EmbeddingParams& P, int dtype, bool vec, dim3 grid, cudaStream_t s);
// CTAs that the current device takes in a cluster of the sort, at most.
int most_sort_cluster();
// Sorts P.rows tokens as planned and cuts them into units.
cudaError_t launch_token_sort(const EmbeddingGradParams& P, int g_dtype, int table_dtype, const SortPlan& plan, cudaStream_t s);
cudaError_t launch_embedding_sum(const EmbeddingGradParams& P, int g_dtype, int table_dtype, bool vec, dim3 grid, cudaStream_t s);
cudaError_t launch_embedding_join(const EmbeddingGradParams& P, int table_dtype, dim3 grid, cudaStream_t s);

}  // namespace mr
