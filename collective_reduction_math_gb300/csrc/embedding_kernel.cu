// embedding_kernel.cu -- the embedding lookup and its gradient.
//
//   lookup:    out[t] = scale * table[ids[t]]
//   gradient:  grad[v] (+)= scale * sum over t with ids[t] = v of g[t]
//
// Both move rows; neither has arithmetic to speak of.
#include <algorithm>

#include "elements.cuh"
#include "embedding.h"

namespace mr {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// The buffer row of table row v (v < vocab): an estimate of its rank, put right.
__device__ __forceinline__ char* row_of(const TableRows& T, uint32_t v, int bytes) {
    int r = 0;
    if (T.W > 1) {
        r = min(T.W - 1, (int)((float)v * T.ranks_per_row));
        while (T.first[r] > v) --r;
        while (T.first[r + 1] <= v) ++r;
    }
    return static_cast<char*>(T.row0[r]) + (uint64_t)(v - T.first[r]) * T.ld[r] * bytes;
}

// ---------------------------------------------------------------------------
// Lookup: a warp takes 32 lanes x 4 vectors of 16 bytes (2 KiB) of a row.  A
// row is left out by a negative id (zeros), and NaN past the vocabulary.
// ---------------------------------------------------------------------------
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const __grid_constant__ EmbeddingParams P) {
    using E = Element<DT>;
    constexpr int V = VEC ? E::kLanes : 1, kPart = 32 * kLookupVectors * E::kLanes, N = kPart / (32 * V);
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t warps = (uint64_t)gridDim.x * (kThreads / 32), units = P.rows * P.parts;
    pdl_enter();
    for (uint64_t u = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u < units; u += warps) {
        const uint64_t t = P.parts == 1 ? u : u / P.parts;
        const uint64_t c0 = (u - t * P.parts) * kPart;
        const long long id = P.ids[t];
        const bool there = id >= 0 && id < (long long)P.table.vocab;
        const char* from = there ? row_of(P.table, (uint32_t)id, E::kBytes) : nullptr;
        char* to = static_cast<char*>(P.out) + t * P.ld_out * E::kBytes;
        const float other = id < 0 ? 0.0f : __int_as_float(0x7fffffff);
        if constexpr (VEC) {
            uint4 v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint64_t c = c0 + (uint64_t)(j * 32 + lane) * V;
                if (there && c < P.hidden) v[j] = load16(from + c * E::kBytes);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint64_t c = c0 + (uint64_t)(j * 32 + lane) * V;
                if (c >= P.hidden) continue;
                float f[V];
                if (there) E::unpack(v[j], f);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = there ? __fmul_rn(f[i], P.scale) : other;
                store16(to + c * E::kBytes, E::pack(f));
            }
        } else {
#pragma unroll 8
            for (int j = 0; j < N; ++j) {
                const uint64_t c = c0 + (uint64_t)(j * 32 + lane);
                if (c < P.hidden) E::put(to, c, there ? __fmul_rn(E::get(from, c), P.scale) : other);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient.  A warp has a token and kSlab columns.  The first token of its id
// sums the rows of all that have it, in the order of the tokens, in fp32.
// ---------------------------------------------------------------------------
template <int DG, int DT, bool VEC>
struct Slab {
    static constexpr int kPer = kSlab / 32;
    float acc[kPer];
    // column i of lane l: beside one another where they are read in vectors
    static __device__ __forceinline__ uint32_t column(uint32_t lane, int i) { return VEC ? lane * kPer + i : i * 32 + lane; }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
    }
    __device__ __forceinline__ void add(const char* row, uint64_t c0, uint64_t hidden, uint32_t lane) {
        using E = Element<DG>;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kPer; i += E::kLanes) {
                const uint64_t c = c0 + column(lane, i);
                if (c >= hidden) break;
                float f[E::kLanes];
                E::unpack(load16(row + c * E::kBytes), f);
#pragma unroll
                for (int k = 0; k < E::kLanes; ++k) acc[i + k] = __fadd_rn(acc[i + k], f[k]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint64_t c = c0 + column(lane, i);
                if (c < hidden) acc[i] = __fadd_rn(acc[i], E::get(row, c));
            }
        }
    }
    __device__ __forceinline__ void finish(char* row, uint64_t c0, uint64_t hidden, uint32_t lane, float scale, bool accumulate) const {
        using E = Element<DT>;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kPer; i += E::kLanes) {
                const uint64_t c = c0 + column(lane, i);
                if (c >= hidden) break;
                float f[E::kLanes];
                if (accumulate) E::unpack(load16(row + c * E::kBytes), f);
#pragma unroll
                for (int k = 0; k < E::kLanes; ++k) {
                    const float s = __fmul_rn(acc[i + k], scale);
                    f[k] = accumulate ? __fadd_rn(f[k], s) : s;
                }
                store16(row + c * E::kBytes, E::pack(f));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const uint64_t c = c0 + column(lane, i);
                if (c >= hidden) break;
                const float s = __fmul_rn(acc[i], scale);
                E::put(row, c, accumulate ? __fadd_rn(E::get(row, c), s) : s);
            }
        }
    }
};

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) clear_table_kernel(const __grid_constant__ EmbeddingGradParams P) {
    using E = Element<DT>;
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t warps = (uint64_t)gridDim.x * (kThreads / 32);
    pdl_enter();
    for (uint64_t v = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; v < P.grad.vocab; v += warps) {
        char* row = row_of(P.grad, (uint32_t)v, E::kBytes);
        if constexpr (VEC) {
            for (uint64_t c = lane * E::kLanes; c < P.hidden; c += 32 * E::kLanes) store16(row + c * E::kBytes, make_uint4(0, 0, 0, 0));
        } else {
            for (uint64_t c = lane; c < P.hidden; c += 32) E::put(row, c, 0.0f);
        }
    }
}

template <int DG, int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_grad_kernel(const __grid_constant__ EmbeddingGradParams P) {
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t warps = (uint64_t)gridDim.x * (kThreads / 32), units = P.rows * P.slabs;
    const char* g = static_cast<const char*>(P.g);
    pdl_enter();
    for (uint64_t u = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u < units; u += warps) {
        const uint64_t t = u / P.slabs, c0 = (u - t * P.slabs) * kSlab;
        const long long id = P.ids[t];
        if (id < 0 || id >= (long long)P.grad.vocab) continue;
        bool first = true;
        for (uint64_t i = 0; i < t && first; i += 32) first = !__any_sync(kAll, i + lane < t && P.ids[i + lane] == id);
        if (!first) continue;
        Slab<DG, DT, VEC> sum;
        sum.clear();
        for (uint64_t i = t; i < P.rows; i += 32) {
            unsigned same = __ballot_sync(kAll, i + lane < P.rows && P.ids[i + lane] == id);
            for (; same; same &= same - 1) sum.add(g + (i + __ffs(same) - 1) * P.ld_g * Element<DG>::kBytes, c0, P.hidden, lane);
        }
        sum.finish(row_of(P.grad, (uint32_t)id, Element<DT>::kBytes), c0, P.hidden, lane, P.scale, P.accumulate != 0);
    }
}

template <int DG, int DT, bool VEC>
cudaError_t launch_grad(const EmbeddingGradParams& P, dim3 grid, cudaStream_t s) {
    if (!P.accumulate) {
        const dim3 all((unsigned)std::min<uint64_t>(device_sms() * 8, (P.grad.vocab + kThreads / 32 - 1ull) / (kThreads / 32)), 1, 1);
        const cudaError_t e = launch_kernel(clear_table_kernel<DT, VEC>, all, 0, s, 0, P);
        if (e != cudaSuccess) return e;
        count_launch();
    }
    if (P.rows == 0) return cudaSuccess;
    const cudaError_t e = launch_kernel(embedding_grad_kernel<DG, DT, VEC>, grid, 0, s, 0, P);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingParams& P, int dtype, bool vec, dim3 grid, cudaStream_t s) {
    if (dtype == MR_BF16)
        return vec ? launch_kernel(embedding_kernel<MR_BF16, true>, grid, 0, s, 0, P)
                   : launch_kernel(embedding_kernel<MR_BF16, false>, grid, 0, s, 0, P);
    return vec ? launch_kernel(embedding_kernel<MR_FP32, true>, grid, 0, s, 0, P)
               : launch_kernel(embedding_kernel<MR_FP32, false>, grid, 0, s, 0, P);
}

cudaError_t launch_embedding_grad(const EmbeddingGradParams& P, int g_dtype, int table_dtype, bool vec, dim3 grid, cudaStream_t s) {
    if (g_dtype == MR_BF16) {
        if (table_dtype == MR_BF16)
            return vec ? launch_grad<MR_BF16, MR_BF16, true>(P, grid, s) : launch_grad<MR_BF16, MR_BF16, false>(P, grid, s);
        return vec ? launch_grad<MR_BF16, MR_FP32, true>(P, grid, s) : launch_grad<MR_BF16, MR_FP32, false>(P, grid, s);
    }
    if (table_dtype == MR_BF16)
        return vec ? launch_grad<MR_FP32, MR_BF16, true>(P, grid, s) : launch_grad<MR_FP32, MR_BF16, false>(P, grid, s);
    return vec ? launch_grad<MR_FP32, MR_FP32, true>(P, grid, s) : launch_grad<MR_FP32, MR_FP32, false>(P, grid, s);
}

}  // namespace mr
