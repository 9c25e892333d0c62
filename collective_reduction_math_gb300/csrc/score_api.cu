// score_api.cu -- the C ABI of the token-score operators: argument checks,
// alias checks, the split of rows over CTAs and dispatch.  See include/mr.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <mutex>

#include "mr.h"
#include "mr_internal.h"
#include "order.cuh"

namespace {

using mr::report_error;
using mr::ScoreParams;

constexpr float kLeastScale = 5.421010862427522e-20f;       // 2^-64
constexpr size_t kMostRows = (size_t)1 << 36, kMostStride = (size_t)1 << 40;

// A byte range of the call, or (ld > 0) rows of `width` bytes every `ld` bytes from lo.
struct Span {
    uintptr_t lo, hi;
    size_t ld, width;
    const char* name;
    int rank;       // -1: not a rank buffer
    bool written;
};

struct Spans {
    Span s[2 * MR_MAX_RANKS + 8];
    int n = 0;
    void add(const void* p, size_t bytes, const char* name, bool written) {
        if (p && bytes) s[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, 0, 0, name, -1, written};
    }
    void add_rows(const void* p, size_t rows, size_t ld, size_t width, const char* name, int rank, bool written) {
        if (width) s[n++] = {(uintptr_t)p, (uintptr_t)p + (rows - 1) * ld + width, ld, width, name, rank, written};
    }
};

// Whether two overlapping ranges never share a byte: rows of one stride whose
// columns lie beside each other (column slices of one buffer).
bool beside(const Span& a, const Span& b) {
    if (!a.ld || a.ld != b.ld) return false;
    const Span &x = a.lo <= b.lo ? a : b, &y = a.lo <= b.lo ? b : a;
    const size_t d = (y.lo - x.lo) % x.ld;      // where y's columns start within x's rows
    return d >= x.width && d + y.width <= x.ld;
}

mr_status_t check_spans(Spans& v) {
    std::sort(v.s, v.s + v.n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    int open[2 * MR_MAX_RANKS + 8];
    int nopen = 0;
    for (int i = 0; i < v.n; ++i) {
        const Span& b = v.s[i];
        int keep = 0;
        for (int j = 0; j < nopen; ++j) {
            const Span& a = v.s[open[j]];
            if (a.hi <= b.lo) continue;
            open[keep++] = open[j];
            if (!a.written && !b.written) continue;
            // in place: a rank's gradients over its own scores, row by row
            const bool in_place = a.rank >= 0 && a.rank == b.rank && a.written != b.written && a.lo == b.lo && a.ld == b.ld;
            if (!in_place && !beside(a, b))
                return report_error(MR_ERR_ALIAS, "%s[%d] overlaps %s[%d] in a form that is not an allowed in-place one",
                                    a.name, std::max(0, a.rank), b.name, std::max(0, b.rank));
        }
        nopen = keep;
        open[nopen++] = i;
    }
    return MR_OK;
}

struct Call {
    const char* what;
    ScoreParams P;
    Spans spans;
    size_t rows = 0;
    mr_dtype_t dtype = MR_FP32;
    size_t esize = 4;
    uint32_t nsb = 0;
};

bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Shapes, rank buffers and strides of the scores (and of the gradients).
mr_status_t check_scores(Call& c, const void* const* logits, const size_t* ld, void* const* grad, const size_t* ld_grad,
                         bool with_grad, int W, size_t rows, size_t vocab, mr_dtype_t dtype, float scale) {
    const char* w = c.what;
    if (W < 1 || W > MR_MAX_RANKS) return report_error(MR_ERR_INVALID_ARGUMENT, "W = %d is outside [1, %d]", W, MR_MAX_RANKS);
    if (dtype != MR_FP32 && dtype != MR_BF16 && dtype != MR_INT32)
        return report_error(MR_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)dtype);
    if (dtype == MR_INT32) return report_error(MR_ERR_UNSUPPORTED, "%s takes fp32 and bf16 scores", w);
    if (!logits || (with_grad && !grad)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: logits or grad pointer array is NULL", w);
    if (vocab < 1 || vocab >= ((size_t)1 << 31))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: vocab = %zu is outside [1, 2^31)", w, vocab);
    if (rows > kMostRows) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: rows = %zu is more than 2^36", w, rows);
    if (!(scale >= kLeastScale && scale <= 1.0f / kLeastScale))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: scale must lie in [2^-64, 2^64]", w);
    ScoreParams& P = c.P;
    const size_t b = dtype == MR_BF16 ? 2 : 4;
    c.dtype = dtype;
    c.esize = b;
    c.rows = rows;
    P.rows = rows;
    P.W = W;
    P.vocab = (uint32_t)vocab;
    P.shards_per_col = (float)W / (float)vocab;
    P.scale = scale;
    P.c = (float)((double)scale * 1.4426950408889634);
    const uint32_t sb = mr::kSuperblockBytes / b;       // scores in a superblock
    uint32_t nsb = 0;
    for (int r = 0; r < W; ++r) {
        const size_t lo = mr::chunk_lo(W, vocab, r), width = mr::chunk_lo(W, vocab, r + 1) - lo;
        P.col0[r] = (uint32_t)lo;
        P.sb0[r] = nsb;
        P.x[r] = logits[r];
        P.ld[r] = ld ? ld[r] : width;
        P.g[r] = with_grad ? grad[r] : nullptr;
        P.ldg[r] = ld_grad ? ld_grad[r] : width;
        if (width == 0) continue;       // fewer columns than ranks: never read
        if (rows == 0) continue;
        if (!logits[r]) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: logits[%d] is NULL", w, r);
        if (misaligned(logits[r], b)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: logits[%d] is not aligned to its element", w, r);
        if (P.ld[r] < width || P.ld[r] > kMostStride)
            return report_error(MR_ERR_INVALID_ARGUMENT, "%s: ld[%d] = %zu is below the rank's %zu columns (or over 2^40)", w, r,
                                (size_t)P.ld[r], width);
        if ((unsigned __int128)rows * P.ld[r] * b >> 62)
            return report_error(MR_ERR_INVALID_ARGUMENT, "%s: rows * ld[%d] is too large", w, r);
        c.spans.add_rows(logits[r], rows, P.ld[r] * b, width * b, "logits", r, false);
        if (with_grad) {
            if (!grad[r] || misaligned(grad[r], b))
                return report_error(MR_ERR_INVALID_ARGUMENT, "%s: grad[%d] is NULL or not aligned to its element", w, r);
            if (P.ldg[r] < width || P.ldg[r] > kMostStride || (unsigned __int128)rows * P.ldg[r] * b >> 62)
                return report_error(MR_ERR_INVALID_ARGUMENT, "%s: ld_grad[%d] = %zu is below the rank's %zu columns, or too large", w, r,
                                    (size_t)P.ldg[r], width);
            c.spans.add_rows(grad[r], rows, P.ldg[r] * b, width * b, "grad", r, true);
        }
        // places before the row's start on its 16-byte boundary, over all rows
        const size_t most = (uintptr_t)logits[r] % 16 == 0 && (rows == 1 || P.ld[r] * b % 16 == 0) ? 0
                          : rows == 1 ? (uintptr_t)logits[r] % 16 / b : 16 / b - 1;
        nsb += (uint32_t)((width + most + sb - 1) / sb);
    }
    P.col0[W] = (uint32_t)vocab;
    P.sb0[W] = nsb;
    c.nsb = nsb;
    return MR_OK;
}

// A per-row array: alignment, and its range.
template <class T>
mr_status_t per_row(Call& c, const T* p, size_t per, const char* name, bool written, bool required) {
    if (!p) return required ? report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s is NULL", c.what, name) : MR_OK;
    if (misaligned(p, sizeof(T))) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: %s is not aligned to its element", c.what, name);
    c.spans.add(p, c.rows * per * sizeof(T), name, written);
    return MR_OK;
}

// Clusters of C CTAs of a forward kernel that the current device holds at
// once.  The answer (the driver's, some 10 us) is kept: it depends on the
// kernel, C and the shared memory alone.  Asking beats dividing: clusters do
// not cross the borders between groups of SMs, and 114 clusters of 4 where
// 110 fit left the last four to a second wave (loss and gradient of 1140 rows
// 1.5 times as long).
int resident_clusters(int dev, mr::ScoreKernel kernel, int C, size_t smem) {
    struct Known {
        mr::ScoreKernel kernel;
        size_t smem;
        int C, dev, n;
    };
    constexpr int kMost = 256;      // the oldest gives way
    static Known known[kMost];
    static unsigned count = 0;
    static std::mutex mutex;
    std::lock_guard<std::mutex> lock(mutex);
    for (unsigned i = 0; i < std::min(count, (unsigned)kMost); ++i)
        if (known[i].kernel == kernel && known[i].smem == smem && known[i].C == C && known[i].dev == dev) return known[i].n;
    int n = 0;
    cudaError_t e = mr::allow_score_kernel(kernel, C, smem);
    if (e == cudaSuccess && C == 1) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, mr::kScoreThreads, smem);
        n *= mr::device_sms();
    } else if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)C, 1, 1);
        cfg.blockDim = dim3(mr::kScoreThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)C;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return 0;       // not kept: the launch will say what is wrong
    }
    known[count++ % kMost] = {kernel, smem, C, dev, n};
    return n;
}

struct Plan {
    int C, clusters;
    size_t smem;
};
// What a forward kernel takes of shared memory at a cluster size, and the
// share of the row that it reads twice from beyond it; false: no such choice.
using Needs = bool (*)(const Call&, int C, int choice, size_t* smem, double* again);

// CTAs per row (a cluster), from the modelled time of the whole call: rounds
// of rows over the resident clusters, each a CTA's part of a row at its share
// of the bandwidth (26 GB/s alone) and the cost of the row's start and join.
// `pick_us` is what the top alternatives take the row warp, one row after
// another: a round is not shorter than that, so many rows take small clusters
// (513 rows of 131072 with 20 alternatives: 56 us on clusters of 1, 58 on 2, 87
// on 4; 37 rows: 23, 18, 15).
Plan plan_forward(const Call& c, mr::ScoreKernel kernel, Needs needs, double passes, double join_us, double pick_us) {
    constexpr double kRowUs = 1.0;
    Plan best{0, 1, 0};
    double best_us = 1e300;
    int dev = 0;
    cudaGetDevice(&dev);
    for (int C = 1; C <= mr::kMaxScoreCluster; C *= 2) {
        if (C > 1 && (uint32_t)C * mr::kThreads / 32 > c.nsb + 7) break;        // a superblock for every warp
        size_t bytes = 0;
        double again = 0.0;
        for (int choice = 0; needs(c, C, choice, &bytes, &again); ++choice) {
            if (bytes > mr::kMostDynamicSmem) continue;
            const int clusters = resident_clusters(dev, kernel, C, bytes);
            if (clusters < 1) continue;
            const double rounds = ceil((double)c.rows / clusters);
            const double active = std::min<double>(clusters, c.rows) * C;
            const double gbs = std::min(26.0, 6600.0 / active);
            const double row_us = (double)c.nsb * mr::kSuperblockBytes * (passes + again) / C / (gbs * 1e3) + kRowUs +
                                  (C == 1 ? 0.0 : join_us);
            const double us = row_us + (rounds - 1.0) * std::max(row_us, pick_us);
            if (us < best_us) {
                best_us = us;
                best = {C, clusters, bytes};
            }
        }
    }
    return best;
}

bool plain_needs(const Call&, int, int choice, size_t* smem, double*) {
    *smem = 0;
    return choice == 0;
}
bool top_needs(const Call& c, int, int choice, size_t* smem, double*) {
    *smem = mr::score_top_smem(c.nsb * mr::kSbRuns, c.P.top_k);
    return choice == 0;
}
// The CTA's part of a row, or all but its last round, which may hold a
// superblock or two and keep a third CTA off the SM.
bool step_needs(const Call& c, int C, int choice, size_t* smem, double* again) {
    const uint32_t warps = mr::kThreads / 32, part = (c.nsb + C - 1) / C;
    const uint32_t rounds = (part + warps - 1) / warps, kept = rounds - (uint32_t)choice;
    if (choice > 1 || kept < 1) return false;
    *smem = kept * mr::kStepRoundBytes;
    *again = part > kept * warps ? (double)(part - kept * warps) / part : 0.0;
    return true;
}

// Warps per row of an elementwise kernel, each of `most` superblocks or, where
// there are few rows, fewer, and the grid.  The distillation's units read the
// row's list: 16 superblocks each (4096 x 128000 bf16, 100 entries, units of 4,
// 8, 12, 16, 24: 406, 360, 353, 349, 360 us); the log probabilities' read
// next to nothing and keep the GPU's window on memory smaller with 4 (8192 x
// 131072: 623, 635, 642, 653, 657 us).
dim3 grad_grid(Call& c, uint32_t most) {
    const size_t warps = (size_t)mr::device_sms() * 3 * (mr::kThreads / 32);
    uint32_t s = most;
    while (s > 1 && c.rows * ((c.nsb + s - 1) / s) < 2 * warps) s /= 2;
    c.P.part_sb = s;
    c.P.parts = (int)((c.nsb + s - 1) / s);
    const size_t ctas = (c.rows * c.P.parts + mr::kThreads / 32 - 1) / (mr::kThreads / 32);
    return dim3((unsigned)std::min(ctas, (size_t)mr::device_sms() * 3), 1, 1);
}

mr_status_t launched(const Call& c, cudaError_t e, dim3 grid, size_t smem) {
    if (e != cudaSuccess) return report_error(MR_ERR_CUDA, "%s launch failed: %s", c.what, cudaGetErrorString(e));
    mr::count_launch();
    if (mr::debug_log_level() > 0)
        fprintf(stderr, "[mr] %s dtype=%s W=%d rows=%zu vocab=%u superblocks=%u grid=%u cluster=%d smem=%zu parts=%d\n", c.what,
                c.dtype == MR_BF16 ? "bf16" : "fp32", c.P.W, c.rows, c.P.vocab, c.nsb, grid.x, c.P.csize, smem, c.P.parts);
    return MR_OK;
}

// The teacher's list.
mr_status_t check_teacher(Call& c, int K, const long long* ids, const float* val, mr_distill_t mode, float teacher_scale) {
    if (K < 1 || K > MR_MAX_TEACHER)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: K = %d is outside [1, %d]", c.what, K, MR_MAX_TEACHER);
    if (mode != MR_DISTILL_RENORM && mode != MR_DISTILL_TAIL)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: unknown mode %d", c.what, (int)mode);
    if (!(teacher_scale > 0.0f) || !isfinite(teacher_scale))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: teacher_scale must be positive and finite", c.what);
    if (mode == MR_DISTILL_TAIL && teacher_scale != 1.0f)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: MR_DISTILL_TAIL takes log probabilities as they are (teacher_scale 1)", c.what);
    mr_status_t st = per_row(c, ids, (size_t)K, "teacher_ids", false, c.rows > 0);
    if (st == MR_OK) st = per_row(c, val, (size_t)K, "teacher_val", false, c.rows > 0);
    c.P.K = K;
    c.P.tail = mode == MR_DISTILL_TAIL;
    c.P.teacher_scale = teacher_scale;
    c.P.t_ids = ids;
    c.P.t_val = val;
    return st;
}

mr_status_t run_forward(Call& c, mr::ScoreKernel kernel, const Plan& plan, void* stream) {
    c.P.csize = plan.C;
    const dim3 grid((unsigned)(std::min<size_t>(c.rows, plan.clusters) * plan.C), 1, 1);
    cudaError_t e = mr::allow_score_kernel(kernel, plan.C, plan.smem);
    if (e == cudaSuccess)
        e = mr::launch_kernel_of(mr::kScoreThreads, kernel, grid, plan.smem, (cudaStream_t)stream, plan.C > 1 ? plan.C : 0, c.P);
    return launched(c, e, grid, plan.smem);
}

mr_status_t run_distill(Call& c, bool step, void* stream) {
    const mr::ScoreKernel kernel = mr::distill_forward(c.dtype, step);
    Plan plan = plan_forward(c, kernel, step ? step_needs : plain_needs, step ? 2.0 : 1.0, step ? 2.0 : 1.0, 0.0);
    if (plan.C == 0) {
        // no GPU to ask, or a row too long for sixteen CTAs' shared memory:
        // what does not fit is read again
        plan = {step ? mr::kMaxScoreCluster : 1, 1, step ? 4 * mr::kStepRoundBytes : 0};
        int dev = 0;
        cudaGetDevice(&dev);
        plan.clusters = std::max(1, resident_clusters(dev, kernel, plan.C, plan.smem));
    }
    c.P.cache_rounds = (uint32_t)(plan.smem / mr::kStepRoundBytes);
    return run_forward(c, kernel, plan, stream);
}

}  // namespace

extern "C" {

mr_status_t mr_logprob(const void* const* logits, const size_t* ld, int W, size_t rows, size_t vocab, mr_dtype_t dtype,
                       float scale, const long long* ids, int top_k, float* logprob, float* entropy, float* stats,
                       long long* top_ids, float* top_logprob, void* stream) {
    mr::clear_error();
    Call c{"mr_logprob", {}, {}};
    mr_status_t st = check_scores(c, logits, ld, nullptr, nullptr, false, W, rows, vocab, dtype, scale);
    if (st != MR_OK) return st;
    if (top_k < 0 || top_k > MR_MAX_TOP || (size_t)top_k > vocab)
        return report_error(MR_ERR_INVALID_ARGUMENT, "mr_logprob: top_k = %d is outside [0, min(%d, vocab)]", top_k, MR_MAX_TOP);
    if (top_k > 0 && vocab > MR_MAX_TOP_VOCAB)
        return report_error(MR_ERR_UNSUPPORTED, "mr_logprob: top_k takes a vocab of at most %d", MR_MAX_TOP_VOCAB);
    if ((top_k > 0) != (top_ids || top_logprob))
        return report_error(MR_ERR_INVALID_ARGUMENT, "mr_logprob: top_k and top_ids / top_logprob go together");
    if (logprob && !ids) return report_error(MR_ERR_INVALID_ARGUMENT, "mr_logprob: logprob needs ids");
    if (!logprob && !entropy && !stats && !top_k) return report_error(MR_ERR_INVALID_ARGUMENT, "mr_logprob: no output is asked for");
    if (rows == 0) return MR_OK;
    if ((st = per_row(c, ids, 1, "ids", false, false)) != MR_OK) return st;
    if ((st = per_row(c, logprob, 1, "logprob", true, false)) != MR_OK) return st;
    if ((st = per_row(c, entropy, 1, "entropy", true, false)) != MR_OK) return st;
    if ((st = per_row(c, stats, 2, "stats", true, false)) != MR_OK) return st;
    if ((st = per_row(c, top_ids, (size_t)top_k, "top_ids", true, false)) != MR_OK) return st;
    if ((st = per_row(c, top_logprob, (size_t)top_k, "top_logprob", true, false)) != MR_OK) return st;
    if ((st = check_spans(c.spans)) != MR_OK) return st;
    c.P.ids = ids;
    c.P.top_k = top_k;
    c.P.logprob = logprob;
    c.P.entropy = entropy;
    c.P.stats = stats;
    c.P.top_ids = top_ids;
    c.P.top_logprob = top_logprob;
    const mr::ScoreKernel kernel = mr::logprob_forward(c.P, dtype);
    Plan plan = plan_forward(c, kernel, top_k ? top_needs : plain_needs, 1.0, 1.0, top_k ? 14.0 + 0.22 * top_k : 0.0);
    if (plan.C == 0) plan = {1, 1, top_k ? mr::score_top_smem(c.nsb * mr::kSbRuns, top_k) : 0};       // no GPU to ask: the launch will fail
    return run_forward(c, kernel, plan, stream);
}

mr_status_t mr_logprob_grad(const void* const* logits, const size_t* ld, int W, size_t rows, size_t vocab, mr_dtype_t dtype,
                            float scale, const long long* ids, const float* stats, const float* entropy,
                            const float* g_logprob, const float* g_entropy, void* const* grad, const size_t* ld_grad,
                            void* stream) {
    mr::clear_error();
    Call c{"mr_logprob_grad", {}, {}};
    mr_status_t st = check_scores(c, logits, ld, grad, ld_grad, true, W, rows, vocab, dtype, scale);
    if (st != MR_OK) return st;
    if (!g_logprob && !g_entropy) return report_error(MR_ERR_INVALID_ARGUMENT, "mr_logprob_grad: neither g_logprob nor g_entropy is given");
    if (rows == 0) return MR_OK;
    if ((st = per_row(c, ids, 1, "ids", false, g_logprob != nullptr)) != MR_OK) return st;
    if ((st = per_row(c, stats, 2, "stats", false, true)) != MR_OK) return st;
    if ((st = per_row(c, entropy, 1, "entropy", false, g_entropy != nullptr)) != MR_OK) return st;
    if ((st = per_row(c, g_logprob, 1, "g_logprob", false, false)) != MR_OK) return st;
    if ((st = per_row(c, g_entropy, 1, "g_entropy", false, false)) != MR_OK) return st;
    if ((st = check_spans(c.spans)) != MR_OK) return st;
    c.P.ids = ids;
    c.P.stats_in = stats;
    c.P.entropy_in = entropy;
    c.P.g_row = g_logprob;
    c.P.g_entropy = g_entropy;
    const dim3 grid = grad_grid(c, 4);
    return launched(c, mr::launch_logprob_grad(c.P, dtype, grid, (cudaStream_t)stream), grid, 0);
}

mr_status_t mr_distill_topk(const void* const* logits, const size_t* ld, int W, size_t rows, size_t vocab, mr_dtype_t dtype,
                            float scale, int K, const long long* teacher_ids, const float* teacher_val, mr_distill_t mode,
                            float teacher_scale, float* loss, float* stats, void* stream) {
    mr::clear_error();
    Call c{"mr_distill_topk", {}, {}};
    mr_status_t st = check_scores(c, logits, ld, nullptr, nullptr, false, W, rows, vocab, dtype, scale);
    if (st == MR_OK) st = check_teacher(c, K, teacher_ids, teacher_val, mode, teacher_scale);
    if (st != MR_OK) return st;
    if (!loss && !stats) return report_error(MR_ERR_INVALID_ARGUMENT, "mr_distill_topk: no output is asked for");
    if (rows == 0) return MR_OK;
    if ((st = per_row(c, loss, 1, "loss", true, false)) != MR_OK) return st;
    if ((st = per_row(c, stats, 4, "stats", true, false)) != MR_OK) return st;
    if ((st = check_spans(c.spans)) != MR_OK) return st;
    c.P.loss = loss;
    c.P.stats = stats;
    return run_distill(c, false, stream);
}

mr_status_t mr_distill_topk_grad(const void* const* logits, const size_t* ld, int W, size_t rows, size_t vocab,
                                 mr_dtype_t dtype, float scale, int K, const long long* teacher_ids, const float* teacher_val,
                                 mr_distill_t mode, float teacher_scale, const float* stats, const float* g_loss,
                                 void* const* grad, const size_t* ld_grad, void* stream) {
    mr::clear_error();
    Call c{"mr_distill_topk_grad", {}, {}};
    mr_status_t st = check_scores(c, logits, ld, grad, ld_grad, true, W, rows, vocab, dtype, scale);
    if (st == MR_OK) st = check_teacher(c, K, teacher_ids, teacher_val, mode, teacher_scale);
    if (st != MR_OK) return st;
    if (rows == 0) return MR_OK;
    if ((st = per_row(c, stats, 4, "stats", false, true)) != MR_OK) return st;
    if ((st = per_row(c, g_loss, 1, "g_loss", false, true)) != MR_OK) return st;
    if ((st = check_spans(c.spans)) != MR_OK) return st;
    c.P.stats_in = stats;
    c.P.g_row = g_loss;
    const dim3 grid = grad_grid(c, 16);
    return launched(c, mr::launch_distill_grad(c.P, dtype, grid, (cudaStream_t)stream), grid, 0);
}

mr_status_t mr_distill_topk_step(const void* const* logits, const size_t* ld, int W, size_t rows, size_t vocab,
                                 mr_dtype_t dtype, float scale, int K, const long long* teacher_ids, const float* teacher_val,
                                 mr_distill_t mode, float teacher_scale, const float* weight, float* loss,
                                 void* const* grad, const size_t* ld_grad, void* stream) {
    mr::clear_error();
    Call c{"mr_distill_topk_step", {}, {}};
    mr_status_t st = check_scores(c, logits, ld, grad, ld_grad, true, W, rows, vocab, dtype, scale);
    if (st == MR_OK) st = check_teacher(c, K, teacher_ids, teacher_val, mode, teacher_scale);
    if (st != MR_OK) return st;
    if (rows == 0) return MR_OK;
    if ((st = per_row(c, weight, 1, "weight", false, true)) != MR_OK) return st;
    if ((st = per_row(c, loss, 1, "loss", true, false)) != MR_OK) return st;
    if ((st = check_spans(c.spans)) != MR_OK) return st;
    c.P.g_row = weight;
    c.P.loss = loss;
    return run_distill(c, true, stream);
}

}  // extern "C"
