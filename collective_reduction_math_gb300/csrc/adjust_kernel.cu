// adjust_kernel.cu -- penalties for repeated tokens, biases and token masks on
// rows of scores that W simulated ranks hold in shards, and the way back.
//
// A CTA has a window of a row's columns, which may lie in several shards.  It
// counts the row's history in shared memory (a word a column), streams the
// window through with the mask, and then sets the columns of the history and
// of the biases right, each once: an entry of a list takes its column's word
// and leaves 0, so the next one with the same token finds nothing to do, and
// the words are all 0 again for the next window.
#include "adjust.h"
#include "elements.cuh"

namespace mr {
namespace {

__device__ __forceinline__ uint64_t clamped(const long long* n, uint64_t row, uint64_t most, uint64_t none) {
    if (!n) return none;
    const long long v = n[row];
    return v < 0 ? 0 : min((uint64_t)v, most);
}

__device__ __forceinline__ int rank_of(const AdjustParams& P, uint32_t col) {
    int r = 0;
    while (P.col0[r + 1] <= col) ++r;
    return r;
}

// Bits [col, col + 32) of a row's mask, as far as `last` (the last column wanted).
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* mask, uint32_t col, uint32_t last) {
    const uint32_t w = col / 32, lo = mask[w], hi = w < last / 32 ? mask[w + 1] : 0;
    return __funnelshift_r(lo, hi, col % 32);
}

template <int DT, bool GRAD>
__device__ __forceinline__ void dense(const AdjustParams& P, uint64_t row, const uint32_t* mask, uint32_t lo, uint32_t hi) {
    using E = Element<DT>;
    using Raw = typename E::Raw;
    constexpr uint32_t V = E::kLanes;
    const Raw masked = GRAD ? (Raw)0 : (Raw)E::kMinusInf;
    for (int r = rank_of(P, lo); r < P.W && P.col0[r] < hi; ++r) {
        const uint32_t a = max(lo, P.col0[r]), b = min(hi, P.col0[r + 1]);
        if (a >= b) continue;
        const Raw* from = static_cast<const Raw*>(P.in[r]) + row * P.ldi[r] + (a - P.col0[r]);
        Raw* to = static_cast<Raw*>(P.out[r]) + row * P.ldo[r] + (a - P.col0[r]);
        const bool in_place = from == to;
        if (in_place && !mask) continue;
        const uint32_t n = b - a;
        const uint32_t at = (uint32_t)((uintptr_t)from % 16) / E::kBytes;
        const bool vec = (uintptr_t)from % 16 == (uintptr_t)to % 16;
        const uint32_t head = vec ? min(n, (V - at) % V) : n, vectors = (n - head) / V, tail = head + vectors * V;
        for (uint32_t i = threadIdx.x; i < head + (n - tail); i += kThreads) {
            const uint32_t c = i < head ? i : tail + (i - head);
            const bool keep = !mask || (mask[(a + c) / 32] >> ((a + c) % 32) & 1);
            if (!keep) to[c] = masked;
            else if (!in_place) to[c] = from[c];
        }
        for (uint32_t i = threadIdx.x; i < vectors; i += kThreads) {
            const uint32_t c = head + i * V;
            const uint32_t bits = mask ? mask_bits(mask, a + c, a + c + V - 1) & ((1u << V) - 1) : (1u << V) - 1;
            if (bits == (1u << V) - 1 && in_place) continue;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (bits) v = load16_once(from + c);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (V == 4) {
                    if (!(bits >> k & 1)) w[k] = masked;
                } else {
                    if (!(bits >> (2 * k) & 1)) w[k] = (w[k] & 0xffff0000u) | masked;
                    if (!(bits >> (2 * k + 1) & 1)) w[k] = (w[k] & 0xffffu) | (uint32_t)masked << 16;
                }
            }
            store16(to + c, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

// Column col's word, taken; its score or gradient set right.
template <int DT, bool GRAD>
__device__ __forceinline__ void fix(const AdjustParams& P, uint64_t row, const uint32_t* mask, uint32_t col, uint32_t* word) {
    using E = Element<DT>;
    const uint32_t v = atomicExch(word, 0);
    if (!v || (mask && !(mask[col / 32] >> (col % 32) & 1))) return;
    const int r = rank_of(P, col);
    const uint64_t c = col - P.col0[r];
    const float x = P.x[r] ? E::get(P.x[r], row * P.ldx[r] + c) : 0.0f;
    const uint32_t times = v & kTimes;
    float y = GRAD ? E::get(P.in[r], row * P.ldi[r] + c) : x;
    if ((v & kSeen || times) && P.repetition) {
        const float rep = P.repetition[row];
        y = (x > 0.0f) ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
    }
    if constexpr (!GRAD) {
        if (times) {
            if (P.frequency) y = __fsub_rn(y, __fmul_rn(P.frequency[row], (float)times));
            if (P.presence) y = __fsub_rn(y, P.presence[row]);
        }
        if (v & kBiased) {
            float sum = 0.0f;       // a token listed twice has the sum, in the list's order
            for (uint32_t k = 0; k < P.K; ++k)
                if (P.bias_ids[row * P.K + k] == (long long)col) sum = __fadd_rn(sum, P.bias[row * P.K + k]);
            y = __fadd_rn(y, sum);
        }
    }
    E::put(P.out[r], row * P.ldo[r] + c, y);
}

template <int DT, bool GRAD>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ AdjustParams P) {
    extern __shared__ uint32_t words[];
    const bool lists = P.history || P.K;
    if (lists)
        for (uint32_t i = threadIdx.x; i < P.window; i += kThreads) words[i] = 0;
    pdl_enter();
    const uint64_t units = P.rows * P.windows;
    for (uint64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const uint64_t row = u / P.windows;
        const uint32_t lo = (uint32_t)(u - row * P.windows) * P.window, hi = min(P.vocab, lo + P.window);
        const uint32_t* mask = P.mask ? P.mask + row * P.ld_mask : nullptr;
        const long long* history = P.history ? P.history + row * P.ld_history : nullptr;
        const uint64_t n = history ? clamped(P.n_history, row, P.ld_history, P.ld_history) : 0;
        if (lists) {
            const uint64_t prompt = history ? clamped(P.n_prompt, row, n, 0) : 0;
            __syncthreads();
            for (uint64_t i = threadIdx.x; i < n; i += kThreads) {
                const uint64_t c = (uint64_t)history[i] - lo;
                if (c >= hi - lo) continue;
                if (i < prompt) atomicOr(&words[c], kSeen);
                else atomicAdd(&words[c], 1u);
            }
            for (uint32_t k = threadIdx.x; k < P.K; k += kThreads) {
                const uint64_t c = (uint64_t)P.bias_ids[row * P.K + k] - lo;
                if (c < hi - lo) atomicOr(&words[c], kBiased);
            }
        }
        dense<DT, GRAD>(P, row, mask, lo, hi);
        if (lists) {
            __syncthreads();
            for (uint64_t i = threadIdx.x; i < n; i += kThreads) {
                const uint64_t c = (uint64_t)history[i] - lo;
                if (c < hi - lo) fix<DT, GRAD>(P, row, mask, lo + (uint32_t)c, &words[c]);
            }
            for (uint32_t k = threadIdx.x; k < P.K; k += kThreads) {
                const uint64_t c = (uint64_t)P.bias_ids[row * P.K + k] - lo;
                if (c < hi - lo) fix<DT, GRAD>(P, row, mask, lo + (uint32_t)c, &words[c]);
            }
        }
    }
}

template <int DT, bool GRAD>
cudaError_t launch(const AdjustParams& P, dim3 grid, size_t smem, cudaStream_t s) {
    const cudaError_t e = allow_dynamic_smem(adjust_kernel<DT, GRAD>, smem);
    return e != cudaSuccess ? e : launch_kernel(adjust_kernel<DT, GRAD>, grid, smem, s, 0, P);
}

}  // namespace

cudaError_t launch_adjust(const AdjustParams& P, int dtype, bool grad, dim3 grid, size_t smem, cudaStream_t s) {
    if (dtype == MR_BF16) return grad ? launch<MR_BF16, true>(P, grid, smem, s) : launch<MR_BF16, false>(P, grid, smem, s);
    return grad ? launch<MR_FP32, true>(P, grid, smem, s) : launch<MR_FP32, false>(P, grid, smem, s);
}

}  // namespace mr
