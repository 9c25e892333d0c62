// grad_norm_api.cu -- the C ABI of the gradient norm and the clipping:
// argument checks, alias checks, the lists and dispatch.  See include/mr.h.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <algorithm>
#include <memory>
#include <new>

#include "grad_norm.h"
#include "mr.h"
#include "mr_internal.h"
#include "spans.h"

namespace {

using mr::misaligned;
using mr::report_error;
using mr::TensorList;

constexpr size_t kMostElements = (size_t)1 << 40;
constexpr int kMostTensors = 1 << 20;

int launches(int count) { return (count + mr::kListTensors - 1) / mr::kListTensors; }

struct Call {
    const char* what;
    const void* const* in;
    void* const* out;       // null: no clipping
    const size_t* n;
    const mr_dtype_t* dtype;
    int count;
    float* norm;
    void* workspace;
};

size_t element_bytes(mr_dtype_t dtype) { return dtype == MR_BF16 ? 2 : 4; }

mr_status_t check(const Call& c, size_t workspace_bytes) {
    if (c.count < 0 || c.count > kMostTensors)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: count = %d is outside [0, 2^20]", c.what, c.count);
    if (c.count > 0 && (!c.in || !c.n || !c.dtype)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: grad, n or dtype is NULL", c.what);
    const size_t need = mr_grad_norm_workspace_bytes(c.count);
    if (!c.workspace || misaligned(c.workspace, 8))
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: workspace is NULL or not on an 8-byte boundary", c.what);
    if (workspace_bytes < need)
        return report_error(MR_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes, %zu are needed", c.what, workspace_bytes, need);
    if (misaligned(c.norm, 4)) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: norm is not aligned to its element", c.what);
    const size_t most = (size_t)c.count * (c.out ? 2 : 1) + 2;
    const std::unique_ptr<mr::Span[]> s(new (std::nothrow) mr::Span[most]);
    const std::unique_ptr<int[]> open(new (std::nothrow) int[most]);
    if (!s || !open) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: no memory on the host to check %d tensors", c.what, c.count);
    int k = 0;
    uint64_t tiles = 0;
    for (int i = 0; i < c.count; ++i) {
        const mr_dtype_t d = c.dtype[i];
        if (d != MR_FP32 && d != MR_BF16 && d != MR_INT32)
            return report_error(MR_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d of tensor %d", c.what, (int)d, i);
        if (d == MR_INT32) return report_error(MR_ERR_UNSUPPORTED, "%s takes fp32 and bf16 tensors", c.what);
        if (c.n[i] > kMostElements) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: tensor %d has %zu elements: more than 2^40", c.what, i, c.n[i]);
        if (c.n[i] == 0) continue;
        const size_t b = element_bytes(d), bytes = c.n[i] * b;
        if (!c.in[i] || misaligned(c.in[i], b))
            return report_error(MR_ERR_INVALID_ARGUMENT, "%s: grad[%d] is NULL or not aligned to its element", c.what, i);
        s[k++] = {(uintptr_t)c.in[i], (uintptr_t)c.in[i] + bytes, bytes, bytes, "grad", i, false};
        tiles += bytes / mr::kTileBytes + 2;
        if (!c.out) continue;
        if (!c.out[i] || misaligned(c.out[i], b))
            return report_error(MR_ERR_INVALID_ARGUMENT, "%s: out[%d] is NULL or not aligned to its element", c.what, i);
        s[k++] = {(uintptr_t)c.out[i], (uintptr_t)c.out[i] + bytes, bytes, bytes, "out", i, true};
    }
    if (tiles >> 30) return report_error(MR_ERR_INVALID_ARGUMENT, "%s: the tensors are too large together", c.what);
    s[k++] = {(uintptr_t)c.workspace, (uintptr_t)c.workspace + need, 0, 0, "workspace", -1, true};
    if (c.norm) s[k++] = {(uintptr_t)c.norm, (uintptr_t)c.norm + sizeof(float), 0, 0, "norm", -1, true};
    return mr::check_spans(s.get(), open.get(), k);
}

// The tensors [first, first + kListTensors) of the call; the number of tiles.
uint32_t fill(TensorList& L, const Call& c, int first) {
    uint32_t tiles = 0;
    L.count = 0;
    for (int i = first; i < std::min(c.count, first + mr::kListTensors); ++i) {
        if (c.n[i] == 0) continue;
        const size_t b = element_bytes(c.dtype[i]);
        const int k = L.count++;
        L.in[k] = c.in[i];
        L.out[k] = c.out ? c.out[i] : nullptr;
        L.n[k] = c.n[i] | (c.dtype[i] == MR_BF16 ? mr::kIsBf16 : 0);
        L.tile0[k] = tiles;
        tiles += (uint32_t)(((uintptr_t)c.in[i] % 16 + c.n[i] * b + mr::kTileBytes - 1) / mr::kTileBytes);
    }
    L.tile0[L.count] = tiles;
    return tiles;
}

mr_status_t failed(const Call& c, cudaError_t e) {
    return report_error(MR_ERR_CUDA, "%s launch failed: %s", c.what, cudaGetErrorString(e));
}

mr_status_t run(const Call& c, float max_norm, cudaStream_t s) {
    TensorList L;
    mr::NormPart* parts = static_cast<mr::NormPart*>(c.workspace);
    mr::NormOfParts N{parts, 0, max_norm, c.norm, nullptr};
    for (int j = 0; j < launches(c.count); ++j) {
        const uint32_t tiles = fill(L, c, j * mr::kListTensors);
        if (tiles == 0) continue;
        const unsigned ctas = std::min<unsigned>({tiles, (unsigned)(mr::device_sms() * mr::kNormCtas), (unsigned)mr::kMostNormGrid});
        const cudaError_t e = mr::launch_norm_parts(L, parts + N.count, dim3(ctas, 1, 1), s);
        if (e != cudaSuccess) return failed(c, e);
        mr::count_launch();
        N.count += (int)ctas;
        if (mr::debug_log_level() > 0)
            fprintf(stderr, "[mr] %s tensors=%d of %d tiles=%u grid=%u\n", c.what, L.count, c.count, tiles, ctas);
    }
    bool told = false;      // the norm: by a launch of its own or the clipping's first
    if (c.out && N.count > mr::kMostOwnJoin) {
        N.all = parts;
        const cudaError_t e = mr::launch_norm_join(N, s);
        if (e != cudaSuccess) return failed(c, e);
        mr::count_launch();
        N.count = 1;
        told = true;
    }
    for (int j = 0; c.out && j < launches(c.count); ++j) {
        const uint32_t tiles = fill(L, c, j * mr::kListTensors);
        if (tiles == 0) continue;
        N.norm = told ? nullptr : c.norm;
        told = true;
        // Of six CTAs an SM four are resident, and the others take over as these end
        // (290 tensors, 7e8 mixed, 853 us, with four CTAs 860; 40 tensors of 9e6 18.8 and
        // 19.0; but in place below the limit, where none has much to do, 6.7e7 fp32 50.5 and 48.8).
        const unsigned ctas = std::min<unsigned>(tiles, (unsigned)mr::device_sms() * 6);
        const cudaError_t e = mr::launch_clip(L, N, dim3(ctas, 1, 1), s);
        if (e != cudaSuccess) return failed(c, e);
        mr::count_launch();
    }
    if (told || !c.norm) return MR_OK;
    const cudaError_t e = mr::launch_norm_join(N, s);
    if (e != cudaSuccess) return failed(c, e);
    mr::count_launch();
    return MR_OK;
}

}  // namespace

extern "C" {

size_t mr_grad_norm_workspace_bytes(int count) {
    return (size_t)std::max(1, launches(std::min(std::max(count, 0), kMostTensors))) * mr::kMostNormGrid * sizeof(mr::NormPart);
}

mr_status_t mr_grad_norm(const void* const* grad, const size_t* n, const mr_dtype_t* dtype, int count, float* norm,
                         void* workspace, size_t workspace_bytes, void* stream) {
    mr::clear_error();
    const Call c{"mr_grad_norm", grad, nullptr, n, dtype, count, norm, workspace};
    if (!norm) return report_error(MR_ERR_INVALID_ARGUMENT, "mr_grad_norm: norm is NULL");
    const mr_status_t st = check(c, workspace_bytes);
    return st != MR_OK ? st : run(c, 0.0f, (cudaStream_t)stream);
}

mr_status_t mr_clip_grad_norm(const void* const* grad, void* const* out, const size_t* n, const mr_dtype_t* dtype, int count,
                              float max_norm, float* norm, void* workspace, size_t workspace_bytes, void* stream) {
    mr::clear_error();
    const Call c{"mr_clip_grad_norm", grad, out, n, dtype, count, norm, workspace};
    if (!(max_norm >= 0.0f)) return report_error(MR_ERR_INVALID_ARGUMENT, "mr_clip_grad_norm: max_norm must be a number and not negative");
    if (count > 0 && !out) return report_error(MR_ERR_INVALID_ARGUMENT, "mr_clip_grad_norm: out is NULL");
    const mr_status_t st = check(c, workspace_bytes);
    return st != MR_OK ? st : run(c, max_norm, (cudaStream_t)stream);
}

}  // extern "C"
