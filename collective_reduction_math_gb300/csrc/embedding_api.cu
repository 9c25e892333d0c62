// embedding_api.cu -- the C ABI of the embedding lookup and its gradient:
// argument checks, alias checks and dispatch.  See include/mr.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "embedding.h"
#include "mr.h"
#include "mr_internal.h"
#include "order.cuh"
#include "spans.h"

namespace {

using mr::misaligned;
using mr::report_error;

constexpr size_t kMostStride = (size_t)1 << 40;
using Spans = mr::Spans<MR_MAX_RANKS + 4>;

mr_status_t check_float(const char* what, mr_dtype_t dtype) {
    if (dtype != MR_FP32 && dtype != MR_BF16 && dtype != MR_INT32)
        return report_error(MR_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)dtype);
    if (dtype == MR_INT32) return report_error(MR_ERR_UNSUPPORTED, "%s takes fp32 and bf16 rows", what);
    return MR_OK;
}
size_t bytes_of(mr_dtype_t dtype) { return dtype == MR_BF16 ? 2 : 4; }

// rows of `hidden` elements every `ld` elements: a rank's part of the table, or the tokens' rows
mr_status_t check_rows(const char* what, const char* name, const void* p, size_t rows, size_t hidden, size_t ld, size_t b) {
    if (!p) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s is NULL", what, name);
    if (misaligned(p, b)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s is not aligned to its element", what, name);
    if (ld < hidden || ld > kMostStride)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s's rows are %zu elements apart: below hidden = %zu, or over 2^40", what, name, ld, hidden);
    if ((unsigned __int128)rows * ld * b >> 62) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s is too large", what, name);
    return MR_OK;
}

// Whether every row starts on a 16-byte boundary.
bool on_vectors(const void* p, size_t rows, size_t ld, size_t b) { return !misaligned(p, 16) && (rows <= 1 || ld * b % 16 == 0); }

// The table's buffers, and whether all their rows start on 16-byte boundaries.
mr_status_t check_table(const char* what, const char* name, void* const* rank, const size_t* ld, int W, size_t vocab, size_t hidden,
                        mr_dtype_t dtype, bool written, mr::TableRows& T, Spans& spans, bool& vec) {
    if (W < 1 || W > MR_MAX_RANKS) return report_error(MR_ERR_INVALID_ARGUMENT, "W = %d is outside [1, %d]", W, MR_MAX_RANKS);
    mr_status_t st = check_float(what, dtype);
    if (st != MR_OK) return st;
    if (!rank) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: the %s pointer array is NULL", what, name);
    if (vocab < 1 || vocab >= ((size_t)1 << 31))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: vocab = %zu is outside [1, 2^31)", what, vocab);
    if (hidden < 1 || hidden >= ((size_t)1 << 31))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: hidden = %zu is outside [1, 2^31)", what, hidden);
    const size_t b = bytes_of(dtype);
    T.W = W;
    T.vocab = (uint32_t)vocab;
    T.ranks_per_row = (float)W / (float)vocab;
    for (int r = 0; r < W; ++r) {
        const size_t lo = mr::chunk_lo(W, vocab, r), n = mr::chunk_lo(W, vocab, r + 1) - lo;
        T.row0[r] = rank[r];
        T.ld[r] = ld ? ld[r] : hidden;
        T.first[r] = (uint32_t)lo;
        if (n == 0) continue;       // fewer rows than ranks: never looked at
        char at[48];
        snprintf(at, sizeof(at), "%s[%d]", name, r);
        if ((st = check_rows(what, at, rank[r], n, hidden, T.ld[r], b)) != MR_OK) return st;
        spans.add_rows(rank[r], n, T.ld[r] * b, hidden * b, name, r, written);
        vec = vec && on_vectors(rank[r], n, T.ld[r], b);
    }
    T.first[W] = (uint32_t)vocab;
    return MR_OK;
}

mr_status_t check_ids(const char* what, const long long* ids, size_t rows, Spans& spans) {
    if (rows >= ((size_t)1 << 31)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: rows = %zu is outside [0, 2^31)", what, rows);
    if (rows == 0) return MR_OK;
    if (!ids || misaligned(ids, 8)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: ids is NULL or not aligned to its element", what);
    spans.add(ids, rows * sizeof(long long), "ids", false);
    return MR_OK;
}

mr_status_t check_scale(const char* what, float scale) {
    if (!isfinite(scale)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: scale must be finite", what);
    return MR_OK;
}

// The workspace's parts from `base` on; its size.
size_t workspace_of(mr::EmbeddingGradParams& P, void* base, size_t rows, size_t vocab, size_t hidden) {
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return static_cast<char*>(base) + here;
    };
    const size_t longs = rows / (mr::kUnit + 1);        // rows with more than one unit, at most
    P.counts = reinterpret_cast<mr::SortCounts*>(take(sizeof(mr::SortCounts)));
    P.tokens = reinterpret_cast<uint32_t*>(take(rows * sizeof(uint32_t)));
    P.units = reinterpret_cast<mr::Unit*>(take((rows + 1) * sizeof(mr::Unit)));
    P.longs = reinterpret_cast<uint32_t*>(take(longs * sizeof(uint32_t)));
    P.present = reinterpret_cast<uint32_t*>(take((vocab + 31) / 32 * sizeof(uint32_t)));
    P.ld_partial = (hidden + 3) / 4 * 4;
    P.partial = reinterpret_cast<float*>(take(longs ? (rows + mr::kUnit - 1) / mr::kUnit * 2 * P.ld_partial * sizeof(float) : 0));
    return at;
}

dim3 warp_grid(uint64_t units, unsigned per_sm) {
    const uint64_t per = mr::kThreads / 32, ctas = (units + per - 1) / per;
    return dim3((unsigned)std::max<uint64_t>(1, std::min(ctas, (uint64_t)mr::device_sms() * per_sm)), 1, 1);
}

}  // namespace

extern "C" {

mr_status_t mr_embedding(const void* const* table, const size_t* ld, int W, size_t vocab, size_t hidden, mr_dtype_t dtype,
                         float scale, const long long* ids, size_t rows, void* out, size_t ld_out, void* stream) {
    const char* what = "mr_embedding";
    mr::clear_error();
    mr::EmbeddingParams P{};
    Spans spans;
    bool vec = true;
    mr_status_t st = check_table(what, "table", (void* const*)table, ld, W, vocab, hidden, dtype, false, P.table, spans, vec);
    if (st == MR_OK) st = check_scale(what, scale);
    if (st == MR_OK) st = check_ids(what, ids, rows, spans);
    if (st != MR_OK || rows == 0) return st;
    const size_t b = bytes_of(dtype);
    P.ld_out = ld_out ? ld_out : hidden;
    if ((st = check_rows(what, "out", out, rows, hidden, P.ld_out, b)) != MR_OK) return st;
    spans.add_rows(out, rows, P.ld_out * b, hidden * b, "out", -1, true);
    if ((st = check_spans(spans)) != MR_OK) return st;
    vec = vec && on_vectors(out, rows, P.ld_out, b) && hidden * b % 16 == 0;
    P.ids = ids;
    P.rows = rows;
    P.hidden = hidden;
    P.scale = scale;
    P.out = out;
    const size_t part = 32 * mr::kLookupVectors * 16 / b;
    P.parts = (hidden + part - 1) / part;
    const dim3 grid = warp_grid(P.rows * P.parts, 64);
    const cudaError_t e = mr::launch_embedding(P, dtype, vec, grid, (cudaStream_t)stream);
    if (e != cudaSuccess) return report_error(MR_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
    mr::count_launch();
    if (mr::debug_log_level() > 0)
        fprintf(stderr, "[mr] %s dtype=%s W=%d rows=%zu hidden=%zu vocab=%zu vec=%d grid=%u\n", what, dtype == MR_BF16 ? "bf16" : "fp32", W,
                rows, hidden, vocab, (int)vec, grid.x);
    return MR_OK;
}

size_t mr_embedding_grad_workspace_bytes(size_t rows, size_t vocab, size_t hidden) {
    if (rows > MR_MAX_EMBEDDING_GRAD_ROWS || vocab >= ((size_t)1 << 31) || hidden >= ((size_t)1 << 31)) return 0;      // no such call
    mr::EmbeddingGradParams P{};
    return workspace_of(P, nullptr, rows, vocab, hidden);
}

mr_status_t mr_embedding_grad(const void* g_out, size_t ld_g, mr_dtype_t dtype, const long long* ids, size_t rows, float scale,
                              void* const* grad, const size_t* ld_grad, int W, size_t vocab, size_t hidden,
                              mr_dtype_t grad_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    const char* what = "mr_embedding_grad";
    mr::clear_error();
    mr::EmbeddingGradParams P{};
    Spans spans;
    bool vec = true;
    mr_status_t st = check_table(what, "grad", grad, ld_grad, W, vocab, hidden, grad_dtype, true, P.grad, spans, vec);
    if (st == MR_OK) st = check_float(what, dtype);
    if (st == MR_OK) st = check_scale(what, scale);
    if (st == MR_OK) st = check_ids(what, ids, rows, spans);
    if (st != MR_OK) return st;
    if (accumulate != 0 && accumulate != 1) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: accumulate = %d is neither 0 nor 1", what, accumulate);
    if (rows == 0 && accumulate) return MR_OK;
    if (rows > MR_MAX_EMBEDDING_GRAD_ROWS)
        return report_error(MR_ERR_UNSUPPORTED, "%s takes at most %d rows a call", what, MR_MAX_EMBEDDING_GRAD_ROWS);
    const size_t b = bytes_of(dtype), need = workspace_of(P, workspace, rows, vocab, hidden);
    P.ld_g = ld_g ? ld_g : hidden;
    if (rows > 0) {
        if ((st = check_rows(what, "g_out", g_out, rows, hidden, P.ld_g, b)) != MR_OK) return st;
        spans.add_rows(g_out, rows, P.ld_g * b, hidden * b, "g_out", -1, false);
        vec = vec && on_vectors(g_out, rows, P.ld_g, b);
    }
    if (!workspace || misaligned(workspace, 16))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: workspace is NULL or not on a 16-byte boundary", what);
    if (workspace_bytes < need)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes, %zu are needed", what, workspace_bytes, need);
    spans.add(workspace, need, "workspace", true);
    if ((st = check_spans(spans)) != MR_OK) return st;
    vec = vec && hidden % 8 == 0;
    P.g = g_out;
    P.ids = ids;
    P.rows = (uint32_t)rows;
    P.hidden = hidden;
    P.scale = scale;
    P.accumulate = accumulate;
    P.slabs = (uint32_t)((hidden + mr::kSlab - 1) / mr::kSlab);
    // keys 0 .. vocab
    uint32_t bits = 1;
    while (vocab >> bits) ++bits;
    P.passes = (bits + mr::kSortDigit - 1) / mr::kSortDigit;
    P.digit = (bits + P.passes - 1) / P.passes;
    const mr::SortPlan plan = mr::plan_sort(rows, vocab, hidden, b, bytes_of(grad_dtype), accumulate, mr::device_sms(),
                                            rows > 32768 ? mr::most_sort_cluster() : mr::kMostSortCluster / 2);
    if (plan.cluster == 0)
        return report_error(MR_ERR_UNSUPPORTED, "%s: this device's clusters sort fewer than %zu rows a call", what, rows);
    P.ahead = plan.ahead;
    P.cleared = plan.cleared;
    cudaError_t e = mr::launch_token_sort(P, dtype, grad_dtype, plan, (cudaStream_t)stream);
    if (e == cudaSuccess) {
        mr::count_launch();
        const uint64_t most = rows * P.slabs + (accumulate ? 0 : vocab);
        const dim3 grid = warp_grid(most, 8);
        e = mr::launch_embedding_sum(P, dtype, grad_dtype, vec, grid, (cudaStream_t)stream);
        if (mr::debug_log_level() > 0)
            fprintf(stderr, "[mr] %s dtype=%s grad=%s W=%d rows=%zu hidden=%zu vocab=%zu accumulate=%d vec=%d sort=%dx%d grid=%u\n", what,
                    dtype == MR_BF16 ? "bf16" : "fp32", grad_dtype == MR_BF16 ? "bf16" : "fp32", W, rows, hidden, vocab, accumulate, (int)vec,
                    plan.cluster, plan.items, grid.x);
    }
    if (e == cudaSuccess) {
        mr::count_launch();
        const size_t longs = rows / (mr::kUnit + 1);
        if (longs == 0) return MR_OK;
        const uint64_t most = longs * ((hidden + 127) / 128);
        e = mr::launch_embedding_join(P, grad_dtype, dim3((unsigned)std::min<uint64_t>(most, (uint64_t)mr::device_sms() * 8), 1, 1), (cudaStream_t)stream);
        if (e == cudaSuccess) mr::count_launch();
    }
    return e == cudaSuccess ? MR_OK : report_error(MR_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
}

}  // extern "C"
