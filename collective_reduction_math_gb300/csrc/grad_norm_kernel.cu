// grad_norm_kernel.cu -- the L2 norm of a list of tensors, and the tensors
// scaled to a largest norm.
//
//   norm = sqrt(sum x^2),   coef = norm > max ? max / norm : 1,   out = coef * x
//
// Squares of fp32 values leave fp32's range at both ends, so three sums are
// kept: of x^2, of (x 2^-90)^2 and of (x 2^90)^2.  Where the first is finite
// and at least 2^-60, what it lost below 2^-126 is nothing beside it.  Where it
// overflowed, the squares add up to 2^128 at least and the second sum to 2^-52:
// it loses less than 2^-149 a term, of 2^44 terms at most (a call's tiles), and
// as many of (2^128 2^-90)^2 = 2^76 do not overflow it.  Below 2^-60 every |x| is
// below 2^-30 and the third can neither overflow nor lose a bit that counts.  A thread's sums are fp32 over a tile; tiles, threads,
// CTAs and launches are joined in pairs of floats (the rounding of each addition
// kept beside the sum), over a fixed split: the same bits on every run.  (In
// 64 bits the joins took longer than small lists' sums: this GPU does some two
// such operations a cycle and SM.)
#include "elements.cuh"
#include "grad_norm.h"
#include "packed.cuh"

namespace mr {
namespace {

constexpr float kDown = 0x1p-90f, kUp = 0x1p90f;
constexpr unsigned kAll = 0xffffffffu;

// The squares of a tile, in two lanes each.
struct TileSum {
    F2 mid{0}, big{0}, small{0};
    __device__ __forceinline__ void add(float a, float b) {
        const F2 x = f2(a, b), d = mul2(x, f2(kDown, kDown)), u = mul2(x, f2(kUp, kUp));
        mid = fma2(x, x, mid);
        big = fma2(d, d, big);
        small = fma2(u, u, small);
    }
};

// a + b, and what the addition lost.
__device__ __forceinline__ SumPair exact_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// What was lost is nothing once the sum is no number.
__device__ __forceinline__ SumPair plus(SumPair p, SumPair q) {
    const SumPair s = exact_sum(p.hi, q.hi);
    const float lo = __fadd_rn(s.lo, __fadd_rn(p.lo, q.lo)), hi = __fadd_rn(s.hi, lo);
    return isfinite(s.hi) ? SumPair{hi, __fsub_rn(lo, __fsub_rn(hi, s.hi))} : SumPair{s.hi, 0.0f};
}
__device__ __forceinline__ SumPair plus(SumPair p, F2 lanes) {
    float a, b;
    unpack(lanes, a, b);
    return plus(p, exact_sum(a, b));
}
__device__ __forceinline__ NormPart plus(const NormPart& a, const NormPart& b) {
    return {plus(a.mid, b.mid), plus(a.big, b.big), plus(a.small, b.small)};
}

// A tile of a tensor: the bytes [first, first + kTileBytes) of it, counted from
// its start rounded down to 16 bytes, of which [before, end) are its elements.
struct Tile {
    const char* base;
    uint64_t first, before, end;
    __device__ __forceinline__ Tile(const TensorList& L, int i, uint32_t tile) {
        before = (uintptr_t)L.in[i] % 16;
        base = static_cast<const char*>(L.in[i]) - before;
        first = (uint64_t)(tile - L.tile0[i]) * kTileBytes;
        end = before + (L.n[i] & ~kIsBf16) * (L.n[i] & kIsBf16 ? 2 : 4);
    }
    __device__ __forceinline__ bool whole() const { return first >= before && first + kTileBytes <= end; }
    // the thread's vector j, and whether it lies in the tensor as a whole
    __device__ __forceinline__ uint64_t at(uint32_t j) const { return first + (j * kThreads + threadIdx.x) * 16; }
    __device__ __forceinline__ bool has(uint64_t at) const { return at >= before && at + 16 <= end; }
    __device__ __forceinline__ void load(uint4 (&v)[kTileVectors]) const {
        if (whole()) {
#pragma unroll
            for (uint32_t j = 0; j < kTileVectors; ++j) v[j] = load16_once(base + at(j));
        } else {
#pragma unroll
            for (uint32_t j = 0; j < kTileVectors; ++j) {
                v[j] = make_uint4(0, 0, 0, 0);
                if (has(at(j))) v[j] = load16_once(base + at(j));
            }
        }
    }
};

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
__device__ __forceinline__ void sum_tile(const Tile& t, const uint4 (&v)[kTileVectors], TileSum& s) {
    using E = Element<DT>;
#pragma unroll
    for (uint32_t j = 0; j < kTileVectors; ++j) {
        float f[E::kLanes];
        E::unpack(v[j], f);
#pragma unroll
        for (int k = 0; k < E::kLanes; k += 2) s.add(f[k], f[k + 1]);
    }
    if (t.whole()) return;
    // vectors over the tensor's start or end: their elements one by one
    for (uint32_t j = 0; j < kTileVectors; ++j) {
        const uint64_t p = t.at(j);
        if (t.has(p)) continue;
        for (uint64_t e = max(p, t.before); e < min(p + 16, t.end); e += E::kBytes) s.add(E::get(t.base + e, 0), 0.0f);
    }
}

// The same on every thread of the CTA (kThreads threads).
__device__ __forceinline__ NormPart join(NormPart v) {
    __shared__ NormPart part[kThreads / 32];
#pragma unroll
    for (int d = 16; d; d /= 2) {
        NormPart o;
        o.mid = {__shfl_xor_sync(kAll, v.mid.hi, d), __shfl_xor_sync(kAll, v.mid.lo, d)};
        o.big = {__shfl_xor_sync(kAll, v.big.hi, d), __shfl_xor_sync(kAll, v.big.lo, d)};
        o.small = {__shfl_xor_sync(kAll, v.small.hi, d), __shfl_xor_sync(kAll, v.small.lo, d)};
        v = plus(v, o);
    }
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    NormPart t = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) t = plus(t, part[w]);
    return t;
}

// The tensor of a tile that is no earlier than tensor i's first.
__device__ __forceinline__ int tensor_from(const TensorList& L, int i, uint32_t tile) {
    while (L.tile0[i + 1] <= tile) ++i;
    return i;
}

__global__ void __launch_bounds__(kThreads, kNormCtas) norm_parts_kernel(const __grid_constant__ TensorList L, NormPart* parts) {
    const uint32_t tiles = L.tile0[L.count];
    NormPart sum{};
    int i = tensor_of(L, blockIdx.x);
    pdl_enter();
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        i = tensor_from(L, i, t);
        const Tile tile(L, i, t);
        uint4 v[kTileVectors];
        tile.load(v);
        TileSum s;
        if (L.n[i] & kIsBf16) sum_tile<MR_BF16>(tile, v, s);
        else sum_tile<MR_FP32>(tile, v, s);
        sum = {plus(sum.mid, s.mid), plus(sum.big, s.big), plus(sum.small, s.small)};
    }
    sum = join(sum);
    if (threadIdx.x == 0) parts[blockIdx.x] = sum;
}

// The norm as root * 2^power, with what the root is short of; power 0, 90 or -90.
struct Norm {
    float root, rest;
    int power;
    __device__ __forceinline__ float value() const {
        return power == 0 ? root : power > 0 ? __fmul_rn(root, 0x1p90f) : __fmul_rn(root, 0x1p-90f);
    }
    // max / norm where that is below 1, else 1; NaN where the norm is
    __device__ __forceinline__ float factor(float max) const {
        if (isnan(root)) return root;
        const float scaled = power == 0 ? max : power > 0 ? __fmul_rn(max, 0x1p-90f) : __fmul_rn(max, 0x1p90f);
        if (!(root > scaled || (root == scaled && rest > 0.0f))) return 1.0f;
        if (isinf(root)) return 0.0f;
        // scaled, but where 2^-90 would cost bits of max
        return power > 0 ? __fmul_rn(__fdiv_rn(max, root), 0x1p-90f) : __fdiv_rn(scaled, root);
    }
};
// On every thread.
__device__ __forceinline__ Norm norm_of(const NormOfParts& N) {
    NormPart v{};
    for (int i = threadIdx.x; i < N.count; i += kThreads) v = plus(v, N.parts[i]);
    v = join(v);
    Norm n;
    SumPair s = v.mid;
    n.power = 0;
    if (s.hi < 0x1p-60f) {
        s = v.small;
        n.power = -90;
    } else if (isinf(s.hi)) {
        s = v.big;
        n.power = 90;
    }
    n.root = __fsqrt_rn(s.hi);
    // a step of Newton's iteration for what it lacks
    n.rest = s.hi > 0.0f && isfinite(s.hi) ? __fdiv_rn(__fadd_rn(__fmaf_rn(-n.root, n.root, s.hi), s.lo), __fmul_rn(2.0f, n.root)) : 0.0f;
    return n;
}

__global__ void __launch_bounds__(kThreads) norm_join_kernel(const __grid_constant__ NormOfParts N) {
    pdl_enter();
    const Norm norm = norm_of(N);
    if (threadIdx.x == 0) *N.norm = norm.value();
}

// The tile's vectors, scaled; `to` is where its base goes.
template <int DT>
__device__ __forceinline__ void clip_tile(const Tile& t, const uint4 (&v)[kTileVectors], float coef, char* to) {
    using E = Element<DT>;
    const bool whole = t.whole(), vectors = (uintptr_t)to % 16 == 0;
#pragma unroll
    for (uint32_t j = 0; j < kTileVectors; ++j) {
        const uint64_t p = t.at(j);
        if (vectors && (whole || t.has(p))) {
            float f[E::kLanes];
            E::unpack(v[j], f);
#pragma unroll
            for (int k = 0; k < E::kLanes; ++k) f[k] = __fmul_rn(f[k], coef);
            store16_once(to + p, E::pack(f));
        } else {
            for (uint64_t e = max(p, t.before); e < min(p + 16, t.end); e += E::kBytes)
                E::put(to + e, 0, __fmul_rn(E::get(t.base + e, 0), coef));
        }
    }
}

// The tiles backwards: the last that the norm has read are still in L2.  A CTA's
// first tile is on its way while the norm is put together.
__global__ void __launch_bounds__(kThreads, kNormCtas) clip_kernel(const __grid_constant__ TensorList L, const __grid_constant__ NormOfParts N) {
    const uint32_t tiles = L.tile0[L.count];
    int i = tensor_of(L, tiles - 1 - blockIdx.x);
    float coef = 0.0f;
    bool first = true;
    pdl_enter();
    for (uint32_t k = blockIdx.x; k < tiles; k += gridDim.x) {
        const uint32_t t = tiles - 1 - k;
        while (L.tile0[i] > t) --i;
        const bool in_place = L.in[i] == L.out[i];
        if (!first && coef == 1.0f && in_place) continue;
        const Tile tile(L, i, t);
        uint4 v[kTileVectors];
        tile.load(v);
        if (first) {
            const Norm norm = norm_of(N);
            if (N.norm && blockIdx.x == 0 && threadIdx.x == 0) *N.norm = norm.value();
            coef = norm.factor(N.max_norm);
            first = false;
            if (coef == 1.0f && in_place) continue;
        }
        char* to = static_cast<char*>(L.out[i]) - tile.before;
        if (L.n[i] & kIsBf16) clip_tile<MR_BF16>(tile, v, coef, to);
        else clip_tile<MR_FP32>(tile, v, coef, to);
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
