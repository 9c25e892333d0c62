// embedding_kernel.cu -- the embedding lookup and its gradient.
//
//   lookup:    out[t] = scale * table[ids[t]]
//   gradient:  grad[v] (+)= scale * sum over t with ids[t] = v of g[t]
//
// Both move rows; neither has arithmetic to speak of.
#include <type_traits>

#include "elements.cuh"
#include "embedding.h"

namespace mr {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// A vector of a row, times the scale, or `other` where there is no row.
template <int DT>
__device__ __forceinline__ uint4 scaled(uint4 v, float scale, bool there, float other) {
    using E = Element<DT>;
    float f[E::kLanes];
    E::unpack(v, f);
#pragma unroll
    for (int i = 0; i < E::kLanes; ++i) f[i] = there ? __fmul_rn(f[i], scale) : other;
    return E::pack(f);
}

// ---------------------------------------------------------------------------
// Lookup: a warp takes 32 lanes x 4 vectors of 16 bytes (2 KiB) of a row.  A
// row is left out by a negative id (zeros), and NaN past the vocabulary.
// ---------------------------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const __grid_constant__ EmbeddingParams P) {
    using E = Element<DT>;
    constexpr int V = E::kLanes, kPart = 32 * kLookupVectors * V;
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
        uint4 v[kLookupVectors];
#pragma unroll
        for (int j = 0; j < kLookupVectors; ++j) {
            const uint64_t c = c0 + (uint64_t)(j * 32 + lane) * V;
            if (there && c < P.hidden) v[j] = load16(from + c * E::kBytes);
        }
#pragma unroll
        for (int j = 0; j < kLookupVectors; ++j) {
            const uint64_t c = c0 + (uint64_t)(j * 32 + lane) * V;
            if (c < P.hidden) store16_once(to + c * E::kBytes, scaled<DT>(v[j], P.scale, there, other));
        }
    }
}

// 16 bytes from place m on of two vectors (m is the same in all lanes).
__device__ __forceinline__ uint4 from_place(uint4 a, uint4 b, uint32_t m) {
    const uint32_t s = m % 4 * 8;
    switch (m / 4) {
        case 0: return make_uint4(__funnelshift_r(a.x, a.y, s), __funnelshift_r(a.y, a.z, s), __funnelshift_r(a.z, a.w, s), __funnelshift_r(a.w, b.x, s));
        case 1: return make_uint4(__funnelshift_r(a.y, a.z, s), __funnelshift_r(a.z, a.w, s), __funnelshift_r(a.w, b.x, s), __funnelshift_r(b.x, b.y, s));
        case 2: return make_uint4(__funnelshift_r(a.z, a.w, s), __funnelshift_r(a.w, b.x, s), __funnelshift_r(b.x, b.y, s), __funnelshift_r(b.y, b.z, s));
        default: return make_uint4(__funnelshift_r(a.w, b.x, s), __funnelshift_r(b.x, b.y, s), __funnelshift_r(b.y, b.z, s), __funnelshift_r(b.z, b.w, s));
    }
}

// Rows that start anywhere.  The vectors are the output row's; where the table's
// row lies otherwise past a 16-byte boundary, each is made of the two that it
// lies in.  Those of the first and the last could reach over the row's ends, so
// these two and what is left at the ends, 4 V - 2 elements at most, go one by one,
// an element a lane.  (20000 x 2001 bf16: 43.5 us element by element, 27.5
// so, at four CTAs an SM; 30.8 at three, 41.7 at five, which spill.)
template <int DT>
__global__ void __launch_bounds__(kThreads, 4) embedding_any_kernel(const __grid_constant__ EmbeddingParams P) {
    using E = Element<DT>;
    constexpr uint32_t V = E::kLanes, kPart = 32 * kLookupVectors;      // vectors
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t warps = (uint64_t)gridDim.x * (kThreads / 32), units = P.rows * P.parts;
    pdl_enter();
    for (uint64_t u = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; u < units; u += warps) {
        const uint64_t t = u / P.parts, part = u - t * P.parts;
        const long long id = P.ids[t];
        const bool there = id >= 0 && id < (long long)P.table.vocab;
        char* to = static_cast<char*>(P.out) + t * P.ld_out * E::kBytes;
        const char* from = there ? row_of(P.table, (uint32_t)id, E::kBytes) : to;      // to: never read
        const float other = id < 0 ? 0.0f : __int_as_float(0x7fffffff);
        const uint64_t head = min(P.hidden, (uint64_t)((16 - (uintptr_t)to % 16) % 16 / E::kBytes));
        const uint64_t vectors = (P.hidden - head) / V;
        const uint32_t m = (uint32_t)(((uintptr_t)from + head * E::kBytes) % 16);
        uint64_t lo = 0, hi = vectors;      // the vectors that are moved as such
        if (m) {
            lo = vectors > 2 ? 1 : 0;
            hi = vectors > 2 ? vectors - 1 : 0;
        }
        uint4 v[kLookupVectors], w[kLookupVectors];
#pragma unroll
        for (int j = 0; j < kLookupVectors; ++j) {
            const uint64_t i = part * kPart + j * 32 + lane;
            if (!there || i < lo || i >= hi) continue;
            const char* p = from + (head + i * V) * E::kBytes - m;
            v[j] = load16(p);
            if (m) w[j] = load16(p + 16);
        }
#pragma unroll
        for (int j = 0; j < kLookupVectors; ++j) {
            const uint64_t i = part * kPart + j * 32 + lane;
            if (m) v[j] = from_place(v[j], w[j], m);
            if (i >= lo && i < hi) store16_once(to + (head + i * V) * E::kBytes, scaled<DT>(v[j], P.scale, there, other));
        }
        const uint64_t e = lane < head + lo * V ? lane : lane + (hi - lo) * V;
        if (part == 0 && e < P.hidden) E::put(to, e, there ? __fmul_rn(E::get(from, e), P.scale) : other);
    }
}

// ---------------------------------------------------------------------------
// Gradient.  The tokens come sorted by row and cut into units
// (token_sort_kernel.cu).  A warp has a unit and kSlab columns: it adds up to
// kUnit rows of g in fp32, in the tokens' order, four rows' loads at a time, and
// writes the table's row, or a partial sum where the row has more units; embedding_join_kernel adds those.  Warps without a unit clear
// rows of no token.
// ---------------------------------------------------------------------------
constexpr int kPer = kSlab / 32;    // columns a lane
// CTAs an SM, for 16384 rows of 4096 bf16 added to an fp32 table: 3 of them 99 us
// (with eight rows' loads at a time as with four), 4 83, 5 (which spill) 109;
// reads and writes that leave nothing in L1 and go first from L2, 80.  Measured
// for bf16 rows in vectors alone, which do not spill at 4; the other variants
// spill 20 to 68 bytes a thread.
constexpr int kSumCtas = 4;

// column i of lane l: beside one another where they are read in vectors
template <bool VEC>
__device__ __forceinline__ uint32_t column(uint32_t lane, int i) {
    return VEC ? lane * kPer + i : i * 32 + lane;
}

// A lane's part of a row, as it lies in memory.
template <int DT, bool VEC>
struct Piece {
    using E = Element<DT>;
    static constexpr int kWords = VEC ? kPer / E::kLanes : kPer;
    typename std::conditional<VEC, uint4, float>::type w[kWords];
    __device__ __forceinline__ void load(const char* row, uint64_t c0, uint64_t hidden, uint32_t lane) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint64_t c = c0 + column<VEC>(lane, VEC ? i * E::kLanes : i);
            if constexpr (VEC) {
                w[i] = make_uint4(0, 0, 0, 0);
                if (c < hidden) w[i] = load16_once(row + c * E::kBytes);
            } else {
                w[i] = c < hidden ? E::get(row, c) : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void values(float (&f)[kPer]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (VEC) {
                float part[E::kLanes];
                E::unpack(w[i], part);
#pragma unroll
                for (int k = 0; k < E::kLanes; ++k) f[i * E::kLanes + k] = part[k];
            } else {
                f[i] = w[i];
            }
        }
    }
    static __device__ __forceinline__ void store(char* row, uint64_t c0, uint64_t hidden, uint32_t lane, const float (&f)[kPer]) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint64_t c = c0 + column<VEC>(lane, VEC ? i * E::kLanes : i);
            if (c >= hidden) break;
            if constexpr (VEC) {
                float part[E::kLanes];
#pragma unroll
                for (int k = 0; k < E::kLanes; ++k) part[k] = f[i * E::kLanes + k];
                store16_once(row + c * E::kBytes, E::pack(part));
            } else {
                E::put(row, c, f[i]);
            }
        }
    }
};

// Clears kFillBytes of each of eight rows that no token has.
template <int DT>
__device__ __forceinline__ void fill(const EmbeddingGradParams& P, uint64_t task, uint32_t chunks, uint32_t lane) {
    constexpr int b = Element<DT>::kBytes;
    const uint32_t group = (uint32_t)(task / chunks), chunk = (uint32_t)(task - (uint64_t)group * chunks), first = P.cleared + group * 8;
    const uint32_t there = P.present[first / 32] >> (first % 32) & 0xffu;
    const uint64_t from = (uint64_t)chunk * kFillBytes, upto = min(P.hidden * b, from + kFillBytes);
    for (uint32_t i = 0; i < 8; ++i)
        if (first + i < P.grad.vocab && !(there >> i & 1)) clear_bytes<b>(row_of(P.grad, first + i, b) + from, upto - from, lane);
}

template <int DG, int DT, bool VEC>
__global__ void __launch_bounds__(kThreads, kSumCtas) embedding_sum_kernel(const __grid_constant__ EmbeddingGradParams P) {
    constexpr int kRows = 4;
    const uint32_t lane = threadIdx.x % 32;
    const uint32_t warps = gridDim.x * (kThreads / 32), first = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const char* g = static_cast<const char*>(P.g);
    // from a task to this warp's next: units, and slabs
    const uint32_t unit_step = warps / P.slabs, slab_step = warps % P.slabs;
    uint32_t u = first / P.slabs, slab = first % P.slabs;
    pdl_enter();
    const uint32_t units = P.counts->units;
    for (; u < units; u += unit_step, slab += slab_step) {
        if (slab >= P.slabs) {
            slab -= P.slabs;
            if (++u >= units) break;
        }
        const Unit now = P.units[u];
        const uint32_t start = now.start & kStart, n = (P.units[u + 1].start & kStart) - start;
        const uint32_t token = lane < n ? P.tokens[start + lane] : 0;
        const uint64_t c0 = (uint64_t)slab * kSlab;
        char* row = row_of(P.grad, now.row, Element<DT>::kBytes);
        const bool whole = !(now.start & kPart), add = whole && P.accumulate;
        Piece<DT, VEC> old;
        if (add) old.load(row, c0, P.hidden, lane);
        float acc[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
        for (uint32_t i = 0; i < n; i += kRows) {
            Piece<DG, VEC> piece[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (i + r < n)
                    piece[r].load(g + (uint64_t)__shfl_sync(kAll, token, i + r) * P.ld_g * Element<DG>::kBytes, c0, P.hidden, lane);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (i + r >= n) break;
                float f[kPer];
                piece[r].values(f);
#pragma unroll
                for (int k = 0; k < kPer; ++k) acc[k] = __fadd_rn(acc[k], f[k]);
            }
        }
        if (!whole) {
            float* to = P.partial + partial_slot(start, now.start & kFirst) * P.ld_partial;
            Piece<MR_FP32, VEC>::store(reinterpret_cast<char*>(to), c0, P.hidden, lane, acc);
            continue;
        }
        float was[kPer];
        if (add) old.values(was);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            acc[k] = __fmul_rn(acc[k], P.scale);
            if (add) acc[k] = __fadd_rn(was[k], acc[k]);
        }
        Piece<DT, VEC>::store(row, c0, P.hidden, lane, acc);
    }
    if (P.accumulate) return;
    if (slab >= P.slabs) {
        slab -= P.slabs;
        ++u;
    }
    // rows of no token, of those not cleared yet
    const uint32_t chunks = (uint32_t)((P.hidden * Element<DT>::kBytes + kFillBytes - 1) / kFillBytes);
    const uint64_t tasks = P.cleared < P.grad.vocab ? (uint64_t)((P.grad.vocab - P.cleared + 7) / 8) * chunks : 0;
    for (uint64_t task = (u - units) * (uint64_t)P.slabs + slab; task < tasks; task += warps) fill<DT>(P, task, chunks, lane);
}

// A CTA adds a row's partial sums of 128 columns: each warp a run of them,
// then the warps' sums in their order.
constexpr uint32_t kJoinColumns = 128;
template <int DT>
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(const __grid_constant__ EmbeddingGradParams P) {
    using E = Element<DT>;
    constexpr uint32_t kWarps = kThreads / 32;
    __shared__ float4 sum[kWarps][32];
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    pdl_enter();
    const uint32_t slabs = (uint32_t)((P.hidden + kJoinColumns - 1) / kJoinColumns), units = P.counts->units;
    const uint64_t tasks = (uint64_t)P.counts->longs * slabs;
    for (uint64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
        const uint32_t u = P.longs[task / slabs];
        const uint64_t c = task % slabs * kJoinColumns + lane * 4;
        const uint32_t start = P.units[u].start & kStart, row = P.units[u].row;
        uint32_t parts = 1;     // the units of this row
        for (bool all = true; all && u + parts < units;) {
            const uint32_t at = u + parts + lane, here = __ballot_sync(kAll, at < units && P.units[at].row == row);
            parts += __popc(here);
            all = here == kAll;
        }
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const uint32_t from = (uint32_t)((uint64_t)warp * parts / kWarps), to = (uint32_t)((uint64_t)(warp + 1) * parts / kWarps);
        if (c < P.hidden) {
#pragma unroll 8
            for (uint32_t k = from; k < to; ++k) {
                const float* p = P.partial + partial_slot(start + k * kUnit, k == 0) * P.ld_partial + c;
                const uint4 v = load16(p);
                s.x = __fadd_rn(s.x, __uint_as_float(v.x));
                s.y = __fadd_rn(s.y, __uint_as_float(v.y));
                s.z = __fadd_rn(s.z, __uint_as_float(v.z));
                s.w = __fadd_rn(s.w, __uint_as_float(v.w));
            }
        }
        __syncthreads();    // the last task's sums are read
        sum[warp][lane] = s;
        __syncthreads();
        if (threadIdx.x < kJoinColumns) {
            const uint64_t col = task % slabs * kJoinColumns + threadIdx.x;
            float t = 0.0f;
#pragma unroll
            for (uint32_t w = 0; w < kWarps; ++w) t = __fadd_rn(t, reinterpret_cast<const float*>(sum[w])[threadIdx.x]);
            if (col < P.hidden) {
                char* to_row = row_of(P.grad, row, E::kBytes);
                t = __fmul_rn(t, P.scale);
                E::put(to_row, col, P.accumulate ? __fadd_rn(E::get(to_row, col), t) : t);
            }
        }
    }
}

template <int DG, int DT>
cudaError_t launch_sum(const EmbeddingGradParams& P, bool vec, dim3 grid, cudaStream_t s) {
    return vec ? launch_kernel(embedding_sum_kernel<DG, DT, true>, grid, 0, s, 0, P)
               : launch_kernel(embedding_sum_kernel<DG, DT, false>, grid, 0, s, 0, P);
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingParams& P, int dtype, bool vec, dim3 grid, cudaStream_t s) {
    if (dtype == MR_BF16) return launch_kernel(vec ? embedding_kernel<MR_BF16> : embedding_any_kernel<MR_BF16>, grid, 0, s, 0, P);
    return launch_kernel(vec ? embedding_kernel<MR_FP32> : embedding_any_kernel<MR_FP32>, grid, 0, s, 0, P);
}

cudaError_t launch_embedding_sum(const EmbeddingGradParams& P, int g_dtype, int table_dtype, bool vec, dim3 grid, cudaStream_t s) {
    if (g_dtype == MR_BF16)
        return table_dtype == MR_BF16 ? launch_sum<MR_BF16, MR_BF16>(P, vec, grid, s) : launch_sum<MR_BF16, MR_FP32>(P, vec, grid, s);
    return table_dtype == MR_BF16 ? launch_sum<MR_FP32, MR_BF16>(P, vec, grid, s) : launch_sum<MR_FP32, MR_FP32>(P, vec, grid, s);
}

cudaError_t launch_embedding_join(const EmbeddingGradParams& P, int table_dtype, dim3 grid, cudaStream_t s) {
    return table_dtype == MR_BF16 ? launch_kernel(embedding_join_kernel<MR_BF16>, grid, 0, s, 0, P)
                                  : launch_kernel(embedding_join_kernel<MR_FP32>, grid, 0, s, 0, P);
}

}  // namespace mr
