// grad_norm_kernel.cu -- the L2 norm of a list of tensors, and the tensors
// scaled to a largest norm.
//
//   norm = sqrt(sum x^2),   coef = norm > max ? max / norm : 1,   out = coef * x
//
// Squares of fp32 values leave fp32's range at both ends, so three sums are
// kept: of x^2, of (x 2^-80)^2 and of (x 2^90)^2.  Where the first is finite
// and at least 2^-60, what it lost below 2^-126 is nothing beside it; where
// it overflowed, some |x| is over 2^60 and the second has all that counts;
// below 2^-60 every |x| is below 2^-30 and the third can neither overflow nor
// lose a bit that counts.  A thread's sums are fp32 over a tile, then
// fp32 pairs (the rounding of each addition is kept beside the sum); CTAs and
// the whole list are joined in 64 bits, over a fixed split: the same bits on
// every run.
#include "elements.cuh"
#include "grad_norm.h"

namespace mr {
namespace {

constexpr float kDown = 0x1p-80f, kUp = 0x1p90f;
constexpr unsigned kAll = 0xffffffffu;

struct Sum3 {
    float mid = 0.0f, big = 0.0f, small = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float d = __fmul_rn(x, kDown), u = __fmul_rn(x, kUp);
        mid = __fmaf_rn(x, x, mid);
        big = __fmaf_rn(d, d, big);
        small = __fmaf_rn(u, u, small);
    }
};

// A sum with what its additions lost (nothing once it is no number).
struct Pair {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
        hi = s;
    }
    __device__ __forceinline__ double value() const { return isfinite(hi) ? (double)hi + (double)lo : (double)hi; }
};

// A tile of tensor i: the elements [lo, hi), from a 16-byte boundary where lo > 0.
struct Tile {
    int i;
    uint64_t lo, hi;
};
template <int DT>
__device__ __forceinline__ void tile_range(const TensorList& L, int i, uint32_t tile, uint64_t& lo, uint64_t& hi) {
    constexpr uint64_t per = kTileBytes / Element<DT>::kBytes;
    const uint64_t n = L.n[i] & ~kIsBf16, before = (uintptr_t)L.in[i] % 16 / Element<DT>::kBytes;
    const uint64_t p = (uint64_t)(tile - L.tile0[i]) * per;
    lo = p > before ? p - before : 0;
    hi = min(n, p + per - before);
}

__device__ __forceinline__ int tensor_of(const TensorList& L, uint32_t tile) {
    int lo = 0, hi = L.count;       // tile0[lo] <= tile < tile0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (L.tile0[mid] <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int DT>
__device__ __forceinline__ void sum_tile(const TensorList& L, int i, uint32_t tile, Sum3& s) {
    using E = Element<DT>;
    constexpr uint32_t V = E::kLanes;
    uint64_t lo, hi;
    tile_range<DT>(L, i, tile, lo, hi);
    const char* p = static_cast<const char*>(L.in[i]);
    if (hi - lo == kTileBytes / E::kBytes) {        // whole vectors, on their boundaries
        uint4 v[kTileVectors];
#pragma unroll
        for (uint32_t j = 0; j < kTileVectors; ++j) v[j] = load16_once(p + (lo + (j * kThreads + threadIdx.x) * V) * E::kBytes);
#pragma unroll
        for (uint32_t j = 0; j < kTileVectors; ++j) {
            float f[V];
            E::unpack(v[j], f);
#pragma unroll
            for (uint32_t k = 0; k < V; ++k) s.add(f[k]);
        }
    } else {
        for (uint64_t e = lo + threadIdx.x; e < hi; e += kThreads) s.add(E::get(p, e));
    }
}

// The same on every thread of the CTA (kThreads threads).
__device__ __forceinline__ NormPart join(NormPart v) {
    __shared__ NormPart part[kThreads / 32];
    for (int d = 16; d; d /= 2) {
        v.mid += __shfl_xor_sync(kAll, v.mid, d);
        v.big += __shfl_xor_sync(kAll, v.big, d);
        v.small += __shfl_xor_sync(kAll, v.small, d);
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    NormPart t = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) {
        t.mid += part[w].mid;
        t.big += part[w].big;
        t.small += part[w].small;
    }
    return t;
}

__global__ void __launch_bounds__(kThreads) norm_parts_kernel(const __grid_constant__ TensorList L, NormPart* parts) {
    const uint32_t tiles = L.tile0[L.count];
    Pair mid, big, small;
    pdl_enter();
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int i = tensor_of(L, t);
        Sum3 s;
        if (L.n[i] & kIsBf16) sum_tile<MR_BF16>(L, i, t, s);
        else sum_tile<MR_FP32>(L, i, t, s);
        mid.add(s.mid);
        big.add(s.big);
        small.add(s.small);
    }
    const NormPart all = join({mid.value(), big.value(), small.value()});
    if (threadIdx.x == 0) parts[blockIdx.x] = all;
}

// The norm in 64 bits, on every thread.
__device__ __forceinline__ double norm_of(const NormOfParts& N) {
    NormPart v{0.0, 0.0, 0.0};
    for (int i = threadIdx.x; i < N.count; i += kThreads) {
        const volatile NormPart& p = N.parts[i];
        v.mid += p.mid;
        v.big += p.big;
        v.small += p.small;
    }
    v = join(v);
    if (v.mid >= 0x1p-60 && isfinite(v.mid)) return sqrt(v.mid);
    if (v.mid < 0x1p-60) return sqrt(v.small) * 0x1p-90;
    return isnan(v.mid) ? v.mid : sqrt(v.big) * 0x1p80;
}

__global__ void __launch_bounds__(kThreads) norm_join_kernel(const __grid_constant__ NormOfParts N) {
    pdl_enter();
    const double norm = norm_of(N);
    if (threadIdx.x == 0) *N.norm = (float)norm;
}

template <int DT>
__device__ __forceinline__ void clip_tile(const TensorList& L, int i, uint32_t tile, float coef) {
    using E = Element<DT>;
    constexpr uint32_t V = E::kLanes;
    uint64_t lo, hi;
    tile_range<DT>(L, i, tile, lo, hi);
    const char* p = static_cast<const char*>(L.in[i]);
    char* q = static_cast<char*>(L.out[i]);
    if (hi - lo == kTileBytes / E::kBytes && (uintptr_t)p % 16 == (uintptr_t)q % 16) {
        uint4 v[kTileVectors];
#pragma unroll
        for (uint32_t j = 0; j < kTileVectors; ++j) v[j] = load16_once(p + (lo + (j * kThreads + threadIdx.x) * V) * E::kBytes);
#pragma unroll
        for (uint32_t j = 0; j < kTileVectors; ++j) {
            float f[V];
            E::unpack(v[j], f);
#pragma unroll
            for (uint32_t k = 0; k < V; ++k) f[k] = __fmul_rn(f[k], coef);
            store16_once(q + (lo + (j * kThreads + threadIdx.x) * V) * E::kBytes, E::pack(f));
        }
    } else {
        for (uint64_t e = lo + threadIdx.x; e < hi; e += kThreads) E::put(q, e, __fmul_rn(E::get(p, e), coef));
    }
}

__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ TensorList L, const __grid_constant__ NormOfParts N) {
    const uint32_t tiles = L.tile0[L.count];
    pdl_enter();
    const double norm = norm_of(N);
    if (N.norm && blockIdx.x == 0 && threadIdx.x == 0) *N.norm = (float)norm;
    const float coef = norm <= (double)N.max_norm ? 1.0f : (float)((double)N.max_norm / norm);     // NaN where the norm is
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int i = tensor_of(L, t);
        if (coef == 1.0f && L.in[i] == L.out[i]) continue;
        if (L.n[i] & kIsBf16) clip_tile<MR_BF16>(L, i, t, coef);
        else clip_tile<MR_FP32>(L, i, t, coef);
    }
}

}  // namespace

cudaError_t launch_norm_parts(const TensorList& L, NormPart* parts, dim3 grid, cudaStream_t s) {
    return launch_kernel(norm_parts_kernel, grid, 0, s, 0, L, parts);
}
cudaError_t launch_norm_join(const NormOfParts& N, cudaStream_t s) { return launch_kernel(norm_join_kernel, dim3(1, 1, 1), 0, s, 0, N); }
cudaError_t launch_clip(const TensorList& L, const NormOfParts& N, dim3 grid, cudaStream_t s) {
    return launch_kernel(clip_kernel, grid, 0, s, 0, L, N);
}

}  // namespace mr
