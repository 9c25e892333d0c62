// grad_norm_kernel.cu -- the L2 norm of a list of tensors, and the tensors
// scaled to a largest norm.
//
//   norm = sqrt(sum x^2),   coef = norm > max ? max / norm : 1,   out = coef * x
//
// Squares of fp32 values leave fp32's range at both ends, so a thread's part of a
// tile is squared as it is where that sum lies from 2^-100 to 2^88, else scaled
// by 2^-90 or 2^90 first; each of the three kinds has a sum of its own, and the
// three are put together at the end.  Terms lose at most 2^-149 each to the
// range's lower end, less than 2^-42 of a part; 2^38 parts (a call's tiles) do
// not overflow: 2^126 as they are, 2^120 scaled down (2^44 elements below
// (2^128 2^-90)^2 each), 2^119 scaled up.  A thread tries the scale that its last
// part had: one pass over a part, but where the size of the elements changes.
//
// A sum is a pair of floats, the second what the first's additions lost.  Two
// squares are added to one another (off by 2 U = 2^-23 of themselves; bf16
// squares have 16 bits, and two of them are nearly always exact), and then to
// the pair without loss; threads, CTAs and launches are joined in pairs too,
// over a fixed split: the same bits on every run.  (Chains of 32 fp32
// multiply-adds left the norm of 1.5e9 normal bf16 values one step below the
// nearest: each addition rounds 16-bit squares to even, and the sum ends up
// 2.2e-8 low; chains of two are 6e-10 low.  In 64 bits the joins took longer
// than small lists' sums: this GPU does some two such operations a cycle and SM.)
#include "elements.cuh"
#include "grad_norm.h"
#include "packed.cuh"

namespace mr {
namespace {

constexpr float kDown = 0x1p-90f, kUp = 0x1p90f;
// What a thread multiplies by before it squares: 1, kDown or kUp.
enum Scale { kAsItIs, kScaledDown, kScaledUp };
constexpr unsigned kAll = 0xffffffffu;

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
// A thread's sum over its part of a tile, in two lanes.
struct LaneSums {
    F2 hi{0}, lo{0};
    __device__ __forceinline__ void add(F2 q) {
        const F2 s = add2(hi, q), t = sub2(s, hi);
        lo = add2(lo, add2(sub2(hi, sub2(s, t)), sub2(q, t)));
        hi = s;
    }
    __device__ __forceinline__ SumPair value() const {
        float a, b, c, d;
        unpack(hi, a, b);
        unpack(lo, c, d);
        return plus(SumPair{a, c}, SumPair{b, d});
    }
};
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

// The sum of (x scale)^2 over the thread's part of a tile, and whether any of it is not +0.
template <int DT>
__device__ __forceinline__ SumPair sum_tile(const Tile& t, const uint4 (&v)[kTileVectors], float scale, bool& any) {
    using E = Element<DT>;
    const F2 factor = f2(scale, scale);
    LaneSums s;
    uint32_t bits = 0;
#pragma unroll
    for (uint32_t j = 0; j < kTileVectors; ++j) {
        bits |= v[j].x | v[j].y | v[j].z | v[j].w;
        float f[E::kLanes];
        E::unpack(v[j], f);
#pragma unroll
        for (int k = 0; k < E::kLanes; k += 4) {
            const F2 a = mul2(f2(f[k], f[k + 1]), factor), b = mul2(f2(f[k + 2], f[k + 3]), factor);
            s.add(fma2(b, b, mul2(a, a)));
        }
    }
    if (!t.whole()) {
        // vectors over the tensor's start or end: their elements one by one
        for (uint32_t j = 0; j < kTileVectors; ++j) {
            const uint64_t p = t.at(j);
            if (t.has(p)) continue;
            for (uint64_t e = max(p, t.before); e < min(p + 16, t.end); e += E::kBytes) {
                const float x = E::get(t.base + e, 0), y = __fmul_rn(x, scale);
                bits |= __float_as_uint(x);
                s.add(f2(__fmul_rn(y, y), 0.0f));
            }
        }
    }
    any = bits != 0;
    return s.value();
}

// Adds the thread's part of a tile to the sum that it belongs to.
template <int DT>
__device__ __forceinline__ void add_tile(NormPart& sum, int& scale, const Tile& t) {
    SumPair s;
    // three at most: down, as it is and up, in this order or the other
#pragma unroll 1
    for (int tries = 0; tries < 3; ++tries) {
        uint4 v[kTileVectors];
        t.load(v);      // again where the scale changes: kept for that, the vectors would spill
        bool any;
        s = sum_tile<DT>(t, v, scale == kAsItIs ? 1.0f : scale == kScaledDown ? kDown : kUp, any);
        // a factor of 2 to spare on the way back, so that no sum is turned away by both
        int other = scale;
        if (scale == kAsItIs) other = !(s.hi < 0x1p88f) ? kScaledDown : s.hi < 0x1p-100f ? kScaledUp : kAsItIs;
        else if (scale == kScaledDown ? s.hi < 0x1p-93f : !(s.hi < 0x1p81f)) other = kAsItIs;
        if (other == scale || !any) break;      // zeros are right on any scale, and change none
        scale = other;
    }
    if (scale == kAsItIs) sum.mid = plus(sum.mid, s);
    else if (scale == kScaledDown) sum.big = plus(sum.big, s);
    else sum.small = plus(sum.small, s);
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
    int scale = kAsItIs, i = tensor_of(L, blockIdx.x);
    pdl_enter();
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        i = tensor_from(L, i, t);
        const Tile tile(L, i, t);
        if (L.n[i] & kIsBf16) add_tile<MR_BF16>(sum, scale, tile);
        else add_tile<MR_FP32>(sum, scale, tile);
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
__device__ __forceinline__ NormPart joined(const NormOfParts& N) {
    NormPart v{};
    for (int i = threadIdx.x; i < N.count; i += kThreads) v = plus(v, N.parts[i]);
    return join(v);
}
__device__ __forceinline__ Norm norm_of(const NormPart& v) {
    // the largest kind that there is, and 2^-180 of the next one, which may be something beside it
    const bool down = !(v.big.hi == 0.0f), plain = v.mid.hi > 0.0f;
    const SumPair first = down ? v.big : plain ? v.mid : v.small, next = down ? v.mid : plain ? v.small : SumPair{0.0f, 0.0f};
    const SumPair s = plus(first, SumPair{__fmul_rn(__fmul_rn(next.hi, kDown), kDown), __fmul_rn(__fmul_rn(next.lo, kDown), kDown)});
    Norm n;
    n.power = down ? 90 : plain ? 0 : -90;
    n.root = __fsqrt_rn(s.hi);
    n.rest = 0.0f;
    if (s.hi > 0.0f && isfinite(s.hi)) {
        // a step of Newton's iteration for what it lacks, which may be a step of the root's
        const float lacks = __fdiv_rn(__fadd_rn(__fmaf_rn(-n.root, n.root, s.hi), s.lo), __fmul_rn(2.0f, n.root)), root = __fadd_rn(n.root, lacks);
        n.rest = __fsub_rn(lacks, __fsub_rn(root, n.root));
        n.root = root;
    }
    return n;
}

__global__ void __launch_bounds__(kThreads) norm_join_kernel(const __grid_constant__ NormOfParts N) {
    pdl_enter();
    const NormPart all = joined(N);
    const Norm norm = norm_of(all);
    if (threadIdx.x > 0) return;
    if (N.norm) *N.norm = norm.value();
    if (N.all) *N.all = all;        // may be one of the parts: they have been read
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
            const Norm norm = norm_of(joined(N));
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
