// adjust_api.cu -- the C ABI of the adjusted scores: argument checks, alias
// checks, windows and dispatch.  See include/mr.h.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "adjust.h"
#include "mr.h"
#include "mr_internal.h"
#include "order.cuh"
#include "spans.h"

namespace {

using mr::misaligned;
using mr::report_error;

constexpr size_t kMostRows = (size_t)1 << 36, kMostStride = (size_t)1 << 40;

struct Call {
    const char* what;
    mr::AdjustParams P;
    mr::Spans<3 * MR_MAX_RANKS + 12> spans;
    size_t rows = 0, b = 4;
    mr_dtype_t dtype = MR_FP32;
};

mr_status_t check_shape(Call& c, int W, size_t rows, size_t vocab, mr_dtype_t dtype) {
    if (W < 1 || W > MR_MAX_RANKS) return report_error(MR_ERR_INVALID_ARGUMENT, "W = %d is outside [1, %d]", W, MR_MAX_RANKS);
    if (dtype != MR_FP32 && dtype != MR_BF16 && dtype != MR_INT32)
        return report_error(MR_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)dtype);
    if (dtype == MR_INT32) return report_error(MR_ERR_UNSUPPORTED, "%s takes fp32 and bf16 scores", c.what);
    if (vocab < 1 || vocab >= ((size_t)1 << 31))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: vocab = %zu is outside [1, 2^31)", c.what, vocab);
    if (rows > kMostRows) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: rows = %zu is more than 2^36", c.what, rows);
    c.rows = rows;
    c.dtype = dtype;
    c.b = dtype == MR_BF16 ? 2 : 4;
    c.P.rows = rows;
    c.P.W = W;
    c.P.vocab = (uint32_t)vocab;
    for (int r = 0; r <= W; ++r) c.P.col0[r] = (uint32_t)mr::chunk_lo(W, vocab, r);
    return MR_OK;
}

// W rank buffers of the call's shape.
mr_status_t check_shards(Call& c, const char* name, const void* const* rank, const size_t* ld, const void** to, uint64_t* to_ld,
                         bool written, bool own_rank) {
    if (!rank) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: the %s pointer array is NULL", c.what, name);
    for (int r = 0; r < c.P.W; ++r) {
        const size_t width = c.P.col0[r + 1] - c.P.col0[r];
        to[r] = rank[r];
        to_ld[r] = ld ? ld[r] : width;
        if (width == 0 || c.rows == 0) continue;        // fewer columns than ranks: never looked at
        if (!rank[r] || misaligned(rank[r], c.b))
            return report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s[%d] is NULL or not aligned to its element", c.what, name, r);
        if (to_ld[r] < width || to_ld[r] > kMostStride || (unsigned __int128)c.rows * to_ld[r] * c.b >> 62)
            return report_error(MR_ERR_INVALID_ARGUMENT, "%s: rows of %s[%d] are %zu elements apart: below the rank's %zu columns, or too large",
                                c.what, name, r, (size_t)to_ld[r], width);
        c.spans.add_rows(rank[r], c.rows, to_ld[r] * c.b, width * c.b, name, own_rank ? r : -1, written);
    }
    return MR_OK;
}

template <class T>
mr_status_t per_row(Call& c, const T* p, size_t per, const char* name) {
    if (misaligned(p, sizeof(T))) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s is not aligned to its element", c.what, name);
    c.spans.add(p, c.rows * per * sizeof(T), name, false);
    return MR_OK;
}

mr_status_t check_adjust(Call& c, const mr_adjust_t* a, bool grad) {
    if (!a) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: adjust is NULL", c.what);
    mr::AdjustParams& P = c.P;
    if (!a->history != (a->history_len == 0))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: history and history_len go together", c.what);
    if (a->history_len >= ((size_t)1 << 30))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: history_len = %zu is outside [0, 2^30)", c.what, a->history_len);
    if (!a->history && (a->n_history || a->n_prompt || a->repetition || a->frequency || a->presence))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: lengths and penalties need a history", c.what);
    if (a->bias_count < 0 || a->bias_count > MR_MAX_BIAS)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: bias_count = %d is outside [0, %d]", c.what, a->bias_count, MR_MAX_BIAS);
    if ((a->bias_count > 0) != (a->bias_ids != nullptr) || (a->bias_count > 0) != (a->bias != nullptr))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: bias_count, bias_ids and bias go together", c.what);
    const size_t words = ((size_t)P.vocab + 31) / 32;
    P.ld_mask = a->ld_mask ? a->ld_mask : words;
    if (a->mask && (P.ld_mask < words || P.ld_mask > kMostStride || (unsigned __int128)c.rows * P.ld_mask >> 58))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: ld_mask = %zu is below the %zu words of a row, or too large", c.what, (size_t)P.ld_mask, words);
    if ((unsigned __int128)c.rows * a->history_len >> 58 || (unsigned __int128)c.rows * (size_t)a->bias_count >> 58)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: the lists are too large", c.what);
    if (c.rows == 0) return MR_OK;
    mr_status_t st = per_row(c, a->history, a->history_len, "history");
    if (st == MR_OK) st = per_row(c, a->n_history, 1, "n_history");
    if (st == MR_OK) st = per_row(c, a->n_prompt, 1, "n_prompt");
    if (st == MR_OK) st = per_row(c, a->repetition, 1, "repetition");
    if (st == MR_OK) st = per_row(c, a->frequency, 1, "frequency");
    if (st == MR_OK) st = per_row(c, a->presence, 1, "presence");
    if (st == MR_OK) st = per_row(c, a->bias_ids, (size_t)a->bias_count, "bias_ids");
    if (st == MR_OK) st = per_row(c, a->bias, (size_t)a->bias_count, "bias");
    if (st != MR_OK) return st;
    if (a->mask) {
        if (misaligned(a->mask, 4)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: mask is not aligned to its element", c.what);
        c.spans.add_rows(a->mask, c.rows, P.ld_mask * 4, words * 4, "mask", -1, false);
    }
    // what this direction has no use for is not looked at on the GPU
    const bool penalties = a->repetition || (!grad && (a->frequency || a->presence));
    P.history = penalties ? a->history : nullptr;
    P.ld_history = a->history_len;
    P.n_history = a->n_history;
    P.n_prompt = a->n_prompt;
    P.repetition = a->repetition;
    P.frequency = a->frequency;
    P.presence = a->presence;
    P.K = grad ? 0 : (uint32_t)a->bias_count;
    P.bias_ids = a->bias_ids;
    P.bias = a->bias;
    P.mask = a->mask;
    return MR_OK;
}

// Columns a CTA takes at a time, and how many of them the lists may name.  Wide
// windows read the history less often and lose L2 for what they write: 128 KiB
// of scores, or 64 KiB of gradients, beside which scores are read (4096 x 131072
// bf16, histories of 1024 to 2048, windows of 64, 128 and 192 KiB: 417, 390 and
// 407 us, the gradient 413, 422 and 442; 1024 x 131072 fp32 in 128 and 256 KiB:
// 173 and 184).  Few rows are cut finer, as far as the device would hold the windows
// at once with short lists (64 rows: 13 windows of 10240 columns, 19.5 us; 16 of
// 8192, more than it holds, 22.6); lists beyond some 3000 entries a window leave
// room for fewer CTAs than are counted with here.  The lists count by the room
// that their rows have (history_len), whatever n_history says: a row's length is
// known on the device alone.  For long lists see kMostListed.
void plan_windows(mr::AdjustParams& P, size_t b, bool grad) {
    const uint64_t listed = (P.history ? P.ld_history : 0) + P.K;
    const uint64_t held = (uint64_t)mr::device_sms() * mr::adjust_ctas(listed > 0) / P.rows;        // windows of a row
    P.window = listed > mr::kMostListed ? mr::kNarrowWindow : (grad ? 1u << 16 : 1u << 17) / (uint32_t)b;
    if (held > 0) P.window = (uint32_t)std::min<uint64_t>(P.window, ((P.vocab + held - 1) / held + 1023) / 1024 * 1024);
    P.windows = (P.vocab + P.window - 1) / P.window;
    P.listed = (uint32_t)std::min<uint64_t>(listed, P.window);
    P.ranks_per_col = (float)P.W / (float)P.vocab;
}

// Ranks whose columns lie behind one another in every buffer (column slices of
// one) are taken as one: a window's walk is then not cut at their borders (256 x
// 8192 fp32 in 8 slices: 7.6 us against 13.3 cut).
void join_ranks(mr::AdjustParams& P, size_t b) {
    int last = -1;
    for (int r = 0; r < P.W; ++r) {
        if (P.col0[r] == P.col0[r + 1]) continue;       // a rank without a column
        const auto behind = [&](const void* a, uint64_t lda, const void* n, uint64_t ldn) {
            return lda == ldn && (const char*)n == (const char*)a + (size_t)(P.col0[r] - P.col0[last]) * b;
        };
        const bool joins = last >= 0 && behind(P.in[last], P.ldi[last], P.in[r], P.ldi[r]) &&
                           behind(P.out[last], P.ldo[last], P.out[r], P.ldo[r]) &&
                           (!P.x[r] || behind(P.x[last], P.ldx[last], P.x[r], P.ldx[r]));
        if (joins) continue;
        ++last;
        P.x[last] = P.x[r], P.in[last] = P.in[r], P.out[last] = P.out[r];
        P.ldx[last] = P.ldx[r], P.ldi[last] = P.ldi[r], P.ldo[last] = P.ldo[r];
        P.col0[last] = P.col0[r];
    }
    P.W = last + 1;
    P.col0[P.W] = P.vocab;
}

mr_status_t run(Call& c, bool grad, void* stream) {
    mr_status_t st = check_spans(c.spans);
    if (st != MR_OK) return st;
    mr::AdjustParams& P = c.P;
    join_ranks(P, c.b);
    plan_windows(P, c.b, grad);
    const dim3 grid((unsigned)std::min<uint64_t>(P.rows * P.windows, (uint64_t)1 << 30), 1, 1);
    const cudaError_t e = mr::launch_adjust(P, c.dtype, grad, grid, (cudaStream_t)stream);
    if (e != cudaSuccess) return report_error(MR_ERR_CUDA, "%s launch failed: %s", c.what, cudaGetErrorString(e));
    mr::count_launch();
    if (mr::debug_log_level() > 0)
        fprintf(stderr, "[mr] %s dtype=%s W=%d rows=%zu vocab=%u window=%u listed=%u grid=%u\n", c.what, c.dtype == MR_BF16 ? "bf16" : "fp32",
                P.W, c.rows, P.vocab, P.window, P.listed, grid.x);
    return MR_OK;
}

}  // namespace

extern "C" {

mr_status_t mr_adjust_logits(const void* const* logits, const size_t* ld, int W, size_t rows, size_t vocab, mr_dtype_t dtype,
                             const mr_adjust_t* adjust, void* const* out, const size_t* ld_out, void* stream) {
    mr::clear_error();
    Call c{"mr_adjust_logits", {}, {}};
    mr_status_t st = check_shape(c, W, rows, vocab, dtype);
    if (st == MR_OK) st = check_shards(c, "logits", logits, ld, c.P.x, c.P.ldx, false, true);
    if (st == MR_OK) st = check_shards(c, "out", out, ld_out, (const void**)c.P.out, c.P.ldo, true, true);
    if (st == MR_OK) st = check_adjust(c, adjust, false);
    if (st != MR_OK || rows == 0) return st;
    std::copy(c.P.x, c.P.x + W, c.P.in);
    std::copy(c.P.ldx, c.P.ldx + W, c.P.ldi);
    return run(c, false, stream);
}

mr_status_t mr_adjust_logits_grad(const void* const* logits, const size_t* ld, int W, size_t rows, size_t vocab, mr_dtype_t dtype,
                                  const mr_adjust_t* adjust, const void* const* g_out, const size_t* ld_g, void* const* grad,
                                  const size_t* ld_grad, void* stream) {
    mr::clear_error();
    Call c{"mr_adjust_logits_grad", {}, {}};
    mr_status_t st = check_shape(c, W, rows, vocab, dtype);
    const bool scores = adjust && adjust->repetition;
    // the gradients may replace those that came back, not the scores, which are still looked at
    if (st == MR_OK && scores) st = check_shards(c, "logits", logits, ld, c.P.x, c.P.ldx, false, false);
    if (st == MR_OK) st = check_shards(c, "g_out", g_out, ld_g, c.P.in, c.P.ldi, false, true);
    if (st == MR_OK) st = check_shards(c, "grad", grad, ld_grad, (const void**)c.P.out, c.P.ldo, true, true);
    if (st == MR_OK) st = check_adjust(c, adjust, true);
    if (st != MR_OK || rows == 0) return st;
    return run(c, true, stream);
}

}  // extern "C"
