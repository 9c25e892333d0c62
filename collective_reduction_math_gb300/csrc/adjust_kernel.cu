// adjust_kernel.cu -- penalties for repeated tokens, biases and token masks on
// rows of scores that W simulated ranks hold in shards, and the way back.
//
// A CTA has a window of a row's columns, which may lie in several shards.  It
// puts the history's and the biases' columns that lie there into a hash table in
// shared memory, with the times each occurs; reads their scores, each once, and
// works out what they become; streams the window through with the mask; and then
// writes the listed columns over it.  Their scores are read first because the
// stream finds them in L2 then: after it, they had left L2 again.  A row's
// history is read once for each of its windows, from L2 after the first.
#include "adjust.h"
#include "elements.cuh"

namespace mr {
namespace {

// Entries of the history, and listed columns, whose loads a thread has in
// flight (4096 x 131072 bf16: 417 us with one column, 420 with two; the gradient,
// which reads two values a column, 437 and 413).
constexpr int kEntries = 4;
__host__ __device__ constexpr int gathers(bool grad) { return grad ? 2 : 1; }

__device__ __forceinline__ uint64_t clamped(const long long* n, uint64_t row, uint64_t most, uint64_t none) {
    if (!n) return none;
    const long long v = n[row];
    return v < 0 ? 0 : min((uint64_t)v, most);
}

__device__ __forceinline__ int rank_of(const AdjustParams& P, uint32_t col) {
    if (P.W == 1) return 0;
    int r = min(P.W - 1, (int)((float)col * P.ranks_per_col));      // nearly
    while (P.col0[r] > col) --r;
    while (P.col0[r + 1] <= col) ++r;
    return r;
}

// Bytes that each repeat the head bit of the byte the selector names (8 + its number).
__device__ __forceinline__ uint32_t spread_heads(uint32_t v, uint32_t selector) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(v), "r"(selector));
    return r;
}
// The words of a vector of which the mask allows no place but those of `bits`.
// Multiplying four bits by 2^7 + 2^14 + 2^21 + 2^28 puts one at the head of each
// byte; a byte permutation that spreads heads makes them masks.
template <int DT, bool GRAD>
__device__ __forceinline__ void apply_mask(uint32_t (&w)[4], uint32_t bits) {
    constexpr uint32_t kSpread = 0x10204080u;
    uint32_t m[4];
    if constexpr (DT == MR_BF16) {
        const uint32_t lo = (bits & 15u) * kSpread, hi = (bits >> 4) * kSpread;
        m[0] = spread_heads(lo, 0x9988);
        m[1] = spread_heads(lo, 0xbbaa);
        m[2] = spread_heads(hi, 0x9988);
        m[3] = spread_heads(hi, 0xbbaa);
    } else {
        const uint32_t all = bits * kSpread;
        m[0] = spread_heads(all, 0x8888);
        m[1] = spread_heads(all, 0x9999);
        m[2] = spread_heads(all, 0xaaaa);
        m[3] = spread_heads(all, 0xbbbb);
    }
    constexpr uint32_t kMasked = GRAD ? 0u : DT == MR_BF16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (w[k] & m[k]) | (kMasked & ~m[k]);
}

// The mask's bits of a thread's vectors: kThreads vectors on, the same place in
// other words.
template <uint32_t V>
struct VectorBits {
    const uint32_t* word;
    uint32_t shift;
    static constexpr uint32_t kAll = (1u << V) - 1, kStep = kThreads * V / 32;
    __device__ __forceinline__ VectorBits(const uint32_t* words, uint32_t col) : word(words + col / 32), shift(col % 32) {}
    // of the vector j * kThreads on
    __device__ __forceinline__ uint32_t at(uint32_t j) const {
        uint32_t b = word[j * kStep] >> shift;
        if (shift + V > 32) b |= word[j * kStep + 1] << (32 - shift);
        return b & kAll;
    }
};
__device__ __forceinline__ bool is_allowed(const uint32_t* mask, uint32_t col) { return !mask || (mask[col / 32] >> (col % 32) & 1); }

// mask: the bits from column mask0 on (null: all are allowed).
template <int DT, bool GRAD, uint32_t kAhead>
__device__ __forceinline__ void stream(const AdjustParams& P, uint64_t row, const uint32_t* mask, uint32_t mask0, uint32_t lo, uint32_t hi) {
    using E = Element<DT>;
    using Raw = typename E::Raw;
    constexpr uint32_t V = E::kLanes, kAll = VectorBits<V>::kAll;
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
            if (!is_allowed(mask, a + c - mask0)) to[c] = masked;
            else if (!in_place) to[c] = from[c];
        }
        const uint32_t first = head + threadIdx.x * V;
        const uint32_t mine = threadIdx.x < vectors ? (vectors - threadIdx.x + kThreads - 1) / kThreads : 0;    // this thread's vectors
        const VectorBits<V> allowed(mask, a + first - mask0);
        from += first;
        to += first;
        uint32_t keep[kAhead];      // a round ahead
#pragma unroll
        for (uint32_t j = 0; j < kAhead; ++j) keep[j] = mask && j < mine ? allowed.at(j) : kAll;
        for (uint32_t i = 0; i < mine; i += kAhead) {
            uint32_t next[kAhead];
            uint4 v[kAhead];
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) {
                // masked as a whole, or left as it is: not read
                if (i + j < mine && keep[j] && !(in_place && keep[j] == kAll)) v[j] = load16_once(from + (i + j) * (kThreads * V));
                else v[j] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) next[j] = mask && i + kAhead + j < mine ? allowed.at(i + kAhead + j) : kAll;
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) {
                if (i + j < mine && !(in_place && keep[j] == kAll)) {
                    uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                    if (mask) apply_mask<DT, GRAD>(w, keep[j]);
                    store16(to + (i + j) * (kThreads * V), make_uint4(w[0], w[1], w[2], w[3]));
                }
                keep[j] = next[j];
            }
        }
    }
}

// The listed columns of the window.
struct Table {
    uint32_t* key;      // column + 1; 0: free
    uint32_t* word;
    uint16_t* taken;    // the slots that are not free
    uint32_t slots;
    // a column's word, of a slot that is taken if it has none
    __device__ __forceinline__ uint32_t* put(uint32_t c, uint32_t* count) const {
        for (uint32_t h = __umulhi(c * 2654435769u, slots);; h = h + 1 < slots ? h + 1 : 0) {
            uint32_t k = *(volatile uint32_t*)(key + h);
            if (k == 0) {
                k = atomicCAS(key + h, 0u, c + 1);
                if (k == 0) {
                    taken[atomicAdd(count, 1u)] = (uint16_t)h;
                    return word + h;
                }
            }
            if (k == c + 1) return word + h;
        }
    }
};

// What a row's listed columns become.
template <bool GRAD>
struct Penalties {
    const AdjustParams& P;
    uint64_t row;
    float repetition, frequency, presence;
    __device__ __forceinline__ Penalties(const AdjustParams& P_, uint64_t row_) : P(P_), row(row_) {
        repetition = P.repetition ? P.repetition[row] : 1.0f;
        frequency = !GRAD && P.frequency ? P.frequency[row] : 0.0f;
        presence = !GRAD && P.presence ? P.presence[row] : 0.0f;
    }
    // y: the column's score, or the gradient that came back to it; x: its score; v: its word
    __device__ __forceinline__ float of(uint32_t col, uint32_t v, float x, float y) const {
        const uint32_t times = v & kTimes;
        if (P.repetition && (v & kSeen || times)) y = x > 0.0f ? __fdiv_rn(y, repetition) : __fmul_rn(y, repetition);
        if constexpr (!GRAD) {
            if (times) {
                if (P.frequency) y = __fsub_rn(y, __fmul_rn(frequency, (float)times));
                if (P.presence) y = __fsub_rn(y, presence);
            }
            if (v & kBiased) {
                float sum = 0.0f;       // a token listed twice has the sum, in the list's order
                for (uint32_t k = 0; k < P.K; ++k)
                    if (P.bias_ids[row * P.K + k] == (long long)col) sum = __fadd_rn(sum, P.bias[row * P.K + k]);
                y = __fadd_rn(y, sum);
            }
        }
        return y;
    }
};

// A listed column's value; a NaN keeps its bits (a column that a prompt names and
// no penalty changes is as it was).
template <int DT>
__device__ __forceinline__ void put_listed(void* p, uint64_t i, uint32_t value) {
    using E = Element<DT>;
    const float v = __uint_as_float(value);
    if (DT == MR_BF16 && isnan(v)) static_cast<typename E::Raw*>(p)[i] = (typename E::Raw)(value >> 16);
    else E::put(p, i, v);
}

template <int DT, bool GRAD, bool LISTS>
__global__ void __launch_bounds__(kThreads, adjust_ctas(LISTS)) adjust_kernel(const __grid_constant__ AdjustParams P) {
    using E = Element<DT>;
    constexpr int kGathers = gathers(GRAD);
    extern __shared__ uint4 dynamic[];
    uint32_t* const words = reinterpret_cast<uint32_t*>(dynamic);
    __shared__ uint32_t count;
    const uint32_t slots = adjust_slots(P.listed);
    const Table table{words, words + slots, reinterpret_cast<uint16_t*>(words + 2 * slots), slots};
    uint32_t* const bits = words + 2 * slots + slots / 2;      // the window's mask
    const uint64_t units = P.rows * P.windows;
    const auto clear = [&] {
        for (uint32_t i = threadIdx.x; i < slots / 2; i += kThreads) dynamic[i] = make_uint4(0, 0, 0, 0);     // keys and words
        if (threadIdx.x == 0) count = 0;
    };
    if constexpr (LISTS) clear();
    pdl_enter();
    for (uint64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const uint64_t row = u / P.windows;
        const uint32_t lo = (uint32_t)(u - row * P.windows) * P.window, width = min(P.vocab - lo, P.window);
        const uint32_t* mask = P.mask ? P.mask + row * P.ld_mask : nullptr;
        if constexpr (LISTS) {
            if (u != blockIdx.x) {
                __syncthreads();        // the last window's listed columns are written
                clear();
            }
            // the stream would wait for the mask each time it asks for scores (4096 x 131072
            // bf16: 468 us, with the window's mask in shared memory 439)
            if (mask)
                for (uint32_t i = threadIdx.x; i < (width + 31) / 32; i += kThreads) bits[i] = mask[lo / 32 + i];
            const Penalties<GRAD> penalties(P, row);
            __syncthreads();
            if (P.history) {
                const long long* history = P.history + row * P.ld_history;
                const uint64_t n = clamped(P.n_history, row, P.ld_history, P.ld_history), prompt = clamped(P.n_prompt, row, n, 0);
                for (uint64_t i0 = threadIdx.x; i0 < n; i0 += kEntries * kThreads) {
                    uint64_t c[kEntries];
#pragma unroll
                    for (int j = 0; j < kEntries; ++j) {
                        const uint64_t i = i0 + j * kThreads;
                        c[j] = i < n ? (uint64_t)history[i] - lo : ~0ull;
                    }
#pragma unroll
                    for (int j = 0; j < kEntries; ++j) {
                        if (c[j] >= width) continue;
                        uint32_t* word = table.put((uint32_t)c[j], &count);
                        if (i0 + j * kThreads < prompt) atomicOr(word, kSeen);
                        else atomicAdd(word, 1u);
                    }
                }
            }
            for (uint32_t k = threadIdx.x; k < P.K; k += kThreads) {
                const uint64_t c = (uint64_t)P.bias_ids[row * P.K + k] - lo;
                if (c < width) atomicOr(table.put((uint32_t)c, &count), kBiased);
            }
            __syncthreads();
            for (uint32_t i0 = threadIdx.x; i0 < count; i0 += kGathers * kThreads) {
                uint32_t h[kGathers], col[kGathers];
                float x[kGathers], y[kGathers];
#pragma unroll
                for (int j = 0; j < kGathers; ++j) {
                    if (i0 + j * kThreads >= count) continue;
                    h[j] = table.taken[i0 + j * kThreads];
                    col[j] = lo + table.key[h[j]] - 1;
                    const int r = rank_of(P, col[j]);
                    const uint64_t c = col[j] - P.col0[r];
                    x[j] = P.x[r] ? E::get(P.x[r], row * P.ldx[r] + c) : 0.0f;
                    y[j] = GRAD ? E::get(P.in[r], row * P.ldi[r] + c) : x[j];
                }
#pragma unroll
                for (int j = 0; j < kGathers; ++j)
                    if (i0 + j * kThreads < count)
                        table.word[h[j]] = __float_as_uint(penalties.of(col[j], table.word[h[j]], x[j], y[j]));
            }
        }
        if constexpr (!LISTS) {
            stream<DT, GRAD, adjust_ahead(false)>(P, row, mask, 0, lo, lo + width);
        } else {
            stream<DT, GRAD, adjust_ahead(true)>(P, row, mask ? bits : nullptr, lo, lo, lo + width);
            __syncthreads();        // the window is written
            for (uint32_t i = threadIdx.x; i < count; i += kThreads) {
                const uint32_t h = table.taken[i], col = lo + table.key[h] - 1;
                if (!is_allowed(mask ? bits : nullptr, col - lo)) continue;
                const int r = rank_of(P, col);
                put_listed<DT>(P.out[r], row * P.ldo[r] + (col - P.col0[r]), table.word[h]);
            }
        }
    }
}

template <int DT, bool GRAD, bool LISTS>
cudaError_t launch(const AdjustParams& P, dim3 grid, cudaStream_t s) {
    const size_t smem = LISTS ? adjust_smem(P.listed, P.window) : 0;
    const cudaError_t e = allow_dynamic_smem(adjust_kernel<DT, GRAD, LISTS>, smem);
    return e != cudaSuccess ? e : launch_kernel(adjust_kernel<DT, GRAD, LISTS>, grid, smem, s, 0, P);
}
template <int DT, bool GRAD>
cudaError_t launch(const AdjustParams& P, dim3 grid, cudaStream_t s) {
    return P.listed ? launch<DT, GRAD, true>(P, grid, s) : launch<DT, GRAD, false>(P, grid, s);
}

}  // namespace

cudaError_t launch_adjust(const AdjustParams& P, int dtype, bool grad, dim3 grid, cudaStream_t s) {
    if (dtype == MR_BF16) return grad ? launch<MR_BF16, true>(P, grid, s) : launch<MR_BF16, false>(P, grid, s);
    return grad ? launch<MR_FP32, true>(P, grid, s) : launch<MR_FP32, false>(P, grid, s);
}

}  // namespace mr
