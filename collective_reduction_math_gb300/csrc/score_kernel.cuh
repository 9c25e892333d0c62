// score_kernel.cuh -- what the token-score kernels share: the walk over a row
// of scores that W simulated ranks hold in shards, and the running softmax
// statistics.
//
// Rank r holds columns [floor(r*V/W), floor((r+1)*V/W)) of every row, so a
// row is W runs of memory that may start at any element.  The kernels walk a
// row in superblocks: 32 lanes x 4 vectors of 16 bytes, so 2 KiB of one
// shard, counted from the shard row's start rounded down to 16 bytes.  A
// column c of a shard is at place p = c + (elements from that boundary to the
// row's start); superblock i of the shard holds places [i*kSb, (i+1)*kSb), and
// vector j of lane l in it the places j*32*VE + l*VE ...: whole-warp loads of
// 512 consecutive bytes.  A superblock that reaches over either end of the
// shard row takes the element-wise loads, which read nothing outside it.
//
// Scores are y = scale * x.  A thread keeps the largest score x_m it has seen
// and, with c = scale * log2(e), the sums
//     s = sum 2^(c (x - x_m)),   u = sum 2^(c (x - x_m)) * c (x - x_m)
// in fp32 (the exponential by the 2^x instruction, relative error 2^-22); a
// new maximum rescales both.  Threads join as  X = max x_m,
// s = sum s_i 2^(c (x_i - X)).  One fused multiply-add makes an exponent,
// c x - R with R = c x_m rounded: what R lost, r = c x_m - R, is the same for
// every term, so 2^-r goes onto a superblock's sum and not onto its terms.
// Where |c x_m| reaches 2^31 (masks of the type's lowest value) two different
// scores are over 2^8 apart in the exponent and the smaller one's term is 0:
// any c that keeps them 2^7 apart gives the same sums, and the power of two
// that does so neither rounds nor overflows.
// NaN and +inf live in x_m (the maximum passes NaN on, a new one keeps an old NaN), and x_m = -inf stands
// for "nothing but -inf so far", where the sums stay 0.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mr_internal.h"
#include "packed.cuh"

namespace mr {

// Exponents are taken no lower where they are a factor: 2^d is 0 long before,
// and 0 * -inf (a mask) or an overflowing product (a mask of the type's lowest
// value) would be NaN.
constexpr float kFarBelow = -1e4f;
constexpr int kSbVectors = kSbRuns;         // 16-byte vectors per lane and superblock
constexpr int kScoreWarps = kThreads / 32;     // the warps that stream

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The largest of a warp's values, NaN above all.
__device__ __forceinline__ float redux_max_nan(float v) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// e^x to some 2^-22 relative: what the product lost is put back, its rounding
// and that of log2 e, up to |x| 2^-24 each.
__device__ __forceinline__ float exp_near(float x) {
    constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = 1.925963e-8f;
    float h = __fmul_rn(x, kLog2e);
    if (h < kFarBelow) h = kFarBelow;       // NaN stays
    const float lost = __fmaf_rn(x, kLog2eRest, __fmaf_rn(x, kLog2e, -h)), e = ex2(h);
    return e == 0.0f ? 0.0f : __fmaf_rn(e, __fmul_rn(lost, 0.69314718f), e);
}
// 1 / x for x of the size of a sum of exponentials: an estimate and a Newton step.
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return __fmaf_rn(__fmaf_rn(-x, r, 1.0f), r, r);
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// ---- a superblock's raw words, as pairs of scores ----
template <int DT>
struct Score;
template <>
struct Score<MR_FP32> {
    static constexpr int kBytes = 4, VE = 4, kPairs = 8, kLogSb = 9, kLogVe = 2;
    static constexpr uint32_t kFill = 0xff800000u;      // -inf
    static __device__ __forceinline__ void pair(const uint32_t (&w)[16], int i, float& a, float& b) {
        a = __uint_as_float(w[2 * i]);
        b = __uint_as_float(w[2 * i + 1]);
    }
    static __device__ __forceinline__ void set_pair(uint32_t (&w)[16], int i, float a, float b) {
        w[2 * i] = __float_as_uint(a);
        w[2 * i + 1] = __float_as_uint(b);
    }
    template <int N>
    static __device__ __forceinline__ float max_words(const uint32_t* w) {
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = __uint_as_float(w[i]);
#pragma unroll
        for (int i = 4; i < N; ++i) m[i % 4] = max_nan(m[i % 4], __uint_as_float(w[i]));
        return max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
    }
    // The least score that still counts, and a pair of scores no lower than it.
    static __device__ __forceinline__ uint32_t floor_word(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ void floored_pair(const uint32_t (&w)[16], int i, uint32_t least, float& a, float& b) {
        a = fmaxf(__uint_as_float(w[2 * i]), __uint_as_float(least));
        b = fmaxf(__uint_as_float(w[2 * i + 1]), __uint_as_float(least));
    }
    static __device__ __forceinline__ float load_one(const char* a) { return *reinterpret_cast<const volatile float*>(a); }
    static __device__ __forceinline__ void store_one(char* a, float v) { *reinterpret_cast<volatile float*>(a) = v; }
    // element e of vector j
    template <int N>
    static __device__ __forceinline__ void put(uint32_t (&w)[N], int j, int e, uint32_t bits) { w[4 * j + e] = bits; }
    template <int N>
    static __device__ __forceinline__ uint32_t get(const uint32_t (&w)[N], int j, int e) { return w[4 * j + e]; }
    static __device__ __forceinline__ uint32_t load_bits(const char* a) { return *reinterpret_cast<const volatile uint32_t*>(a); }
    static __device__ __forceinline__ void store_bits(char* a, uint32_t v) { *reinterpret_cast<volatile uint32_t*>(a) = v; }
    static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits); }
    static __device__ __forceinline__ void mask_one(char* a) { *reinterpret_cast<volatile uint32_t*>(a) = 0xff800000u; }
};
template <>
struct Score<MR_BF16> {
    static constexpr int kBytes = 2, VE = 8, kPairs = 16, kLogSb = 10, kLogVe = 3;
    static constexpr uint32_t kFill = 0xff80ff80u;
    static __device__ __forceinline__ void pair(const uint32_t (&w)[16], int i, float& a, float& b) {
        a = __uint_as_float(w[i] << 16);
        b = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ void set_pair(uint32_t (&w)[16], int i, float a, float b) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
    }
    template <int N>
    static __device__ __forceinline__ float max_words(const uint32_t* w) {
        uint32_t m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = w[i];
#pragma unroll
        for (int i = 4; i < N; ++i) m[i % 4] = max_nan_bf16x2(m[i % 4], w[i]);
        const uint32_t k = max_nan_bf16x2(max_nan_bf16x2(m[0], m[1]), max_nan_bf16x2(m[2], m[3]));
        return max_nan(__uint_as_float(k << 16), __uint_as_float(k & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t floor_word(float x) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(w) : "f"(x));
        return w;
    }
    static __device__ __forceinline__ void floored_pair(const uint32_t (&w)[16], int i, uint32_t least, float& a, float& b) {
        uint32_t m;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w[i]), "r"(least));
        a = __uint_as_float(m << 16);
        b = __uint_as_float(m & 0xffff0000u);
    }
    static __device__ __forceinline__ float load_one(const char* a) {
        return __uint_as_float((uint32_t)*reinterpret_cast<const volatile uint16_t*>(a) << 16);
    }
    static __device__ __forceinline__ void store_one(char* a, float v) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v), "f"(v));
        *reinterpret_cast<volatile uint16_t*>(a) = (uint16_t)w;
    }
    template <int N>
    static __device__ __forceinline__ void put(uint32_t (&w)[N], int j, int e, uint32_t bits) {
        const int i = 4 * j + e / 2;
        w[i] = (e & 1) ? (w[i] & 0xffffu) | (bits << 16) : (w[i] & 0xffff0000u) | bits;
    }
    template <int N>
    static __device__ __forceinline__ uint32_t get(const uint32_t (&w)[N], int j, int e) {
        return (e & 1) ? w[4 * j + e / 2] >> 16 : w[4 * j + e / 2] & 0xffffu;
    }
    static __device__ __forceinline__ uint32_t load_bits(const char* a) { return *reinterpret_cast<const volatile uint16_t*>(a); }
    static __device__ __forceinline__ void store_bits(char* a, uint32_t v) { *reinterpret_cast<volatile uint16_t*>(a) = (uint16_t)v; }
    static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits << 16); }
    static __device__ __forceinline__ void mask_one(char* a) { *reinterpret_cast<volatile uint16_t*>(a) = 0xff80u; }
};

// ---- where a row's shard lies ----
struct ShardRow {
    char* base;             // the row's start, rounded down to 16 bytes
    uint32_t lo, hi;        // its places [lo, hi)
};
template <int DT>
__device__ __forceinline__ ShardRow shard_row(const void* x, uint64_t ld, uint64_t row, uint32_t width) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x) + row * ld * Score<DT>::kBytes;
    ShardRow s;
    s.base = reinterpret_cast<char*>(a & ~(uintptr_t)15);
    s.lo = (uint32_t)(a & 15) / Score<DT>::kBytes;
    s.hi = s.lo + width;
    return s;
}

// 16 bytes; kept in program order with the stores around it (a call may be in place).
__device__ __forceinline__ void load16(uint32_t* w, const char* a) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(a));
}
__device__ __forceinline__ void store16(char* a, const uint32_t* w) {
    asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};"
                 :: "l"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

// The vector at places [p, p + VE) as vector j of the words; -inf outside the row.
template <int DT, int N>
__device__ __forceinline__ void load_vector(uint32_t (&w)[N], int j, const ShardRow& sr, uint32_t p) {
    using S = Score<DT>;
    if (p >= sr.lo && p + S::VE <= sr.hi) {
        load16(&w[4 * j], sr.base + (uint64_t)p * S::kBytes);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * j + i] = S::kFill;
#pragma unroll
        for (int e = 0; e < S::VE; ++e)
            if (p + e >= sr.lo && p + e < sr.hi) S::put(w, j, e, S::load_bits(sr.base + (uint64_t)(p + e) * S::kBytes));
    }
}

// ---- the walk over a row's superblocks (ordinals count through the shards) ----
// Few registers: what only the ends of a shard row need is worked out there.
template <int DT>
struct Walk {
    int r = -1;                     // current shard,
    uint32_t sb_hi = 0;             // the end of its superblocks,
    uint32_t in_lo = 0, in_n = 0;   // and those that lie in its row from end to end
    const char* at = nullptr;       // superblock sb's vector of this lane is at at + sb * kSuperblockBytes
    __device__ __forceinline__ ShardRow shard(const ScoreParams& P, uint64_t row) const {
        return shard_row<DT>(P.x[r], P.ld[r], row, P.col0[r + 1] - P.col0[r]);
    }
    // Moves to the shard of superblock sb (ascending within a row).
    __device__ __forceinline__ bool seek(const ScoreParams& P, uint64_t row, uint32_t sb, int lane) {
        if (sb < sb_hi) return false;
        do {
            ++r;
            sb_hi = P.sb0[r + 1];
        } while (sb >= sb_hi);
        const uint32_t sb_lo = P.sb0[r];
        const ShardRow sr = shard(P, row);
        in_lo = sb_lo + (sr.lo != 0);
        const uint32_t whole = sr.hi >> Score<DT>::kLogSb;      // from the shard's first on
        in_n = whole > (sr.lo != 0) ? whole - (sr.lo != 0) : 0;
        at = sr.base + lane * 16 - (int64_t)sb_lo * kSuperblockBytes;
        return true;
    }
    __device__ __forceinline__ uint32_t place(const ScoreParams& P, uint32_t sb) const { return (sb - P.sb0[r]) << Score<DT>::kLogSb; }
    __device__ __forceinline__ bool inside(uint32_t sb) const { return sb - in_lo < in_n; }
    __device__ __forceinline__ const char* address(uint32_t sb) const { return at + (uint64_t)sb * kSuperblockBytes; }
    // How many of the superblock's runs hold a place of the row.
    __device__ __forceinline__ uint32_t runs(const ScoreParams& P, uint64_t row, uint32_t sb) const {
        using S = Score<DT>;
        if (inside(sb)) return kSbRuns;
        const uint32_t p0 = place(P, sb), hi = shard(P, row).hi;
        return p0 >= hi ? 0 : min((hi - p0 + 32 * S::VE - 1) / (32 * S::VE), (uint32_t)kSbRuns);
    }
};

// The superblock the walk stands at; -inf outside the row.
template <int DT>
__device__ __forceinline__ void load_superblock(uint32_t (&w)[16], const ScoreParams& P, uint64_t row, const Walk<DT>& walk, uint32_t sb,
                                                int lane) {
    using S = Score<DT>;
    if (walk.inside(sb)) {
        const char* a = walk.address(sb);
#pragma unroll
        for (int j = 0; j < kSbVectors; ++j) load16(&w[4 * j], a + j * 512);
    } else {
        const ShardRow sr = walk.shard(P, row);
#pragma unroll
        for (int j = 0; j < kSbVectors; ++j) load_vector<DT>(w, j, sr, walk.place(P, sb) + (uint32_t)(j * 32 + lane) * S::VE);
    }
}

// The gradients' buffer of the shard the walk stands at.
template <int DT>
struct Output {
    char* at = nullptr;         // as the walk's, where both rows start at the same distance from a 16-byte boundary
    bool alike = false;
    __device__ __forceinline__ static ShardRow shard(const ScoreParams& P, uint64_t row, int r) {
        return shard_row<DT>(P.g[r], P.ldg[r], row, P.col0[r + 1] - P.col0[r]);
    }
    __device__ __forceinline__ void follow(const ScoreParams& P, uint64_t row, const Walk<DT>& walk, int lane) {
        const ShardRow sr = shard(P, row, walk.r);
        alike = sr.lo == walk.shard(P, row).lo;
        at = sr.base + lane * 16 - (int64_t)P.sb0[walk.r] * kSuperblockBytes;
    }
    // the element at a place of the walk's shard row
    __device__ __forceinline__ static char* element(const ScoreParams& P, uint64_t row, int r, uint32_t place) {
        const uint32_t lo = shard_row<DT>(P.x[r], P.ld[r], row, 0).lo;
        return static_cast<char*>(P.g[r]) + (row * P.ldg[r] + (place - lo)) * Score<DT>::kBytes;
    }
    // the element at byte `off` of the superblock the walk stands at
    __device__ __forceinline__ char* in_superblock(const ScoreParams& P, uint64_t row, const Walk<DT>& walk, uint32_t sb, uint32_t off,
                                                   int lane) const {
        if (alike) return at + (uint64_t)sb * kSuperblockBytes - lane * 16 + off;
        return element(P, row, walk.r, walk.place(P, sb) + off / Score<DT>::kBytes);
    }
    // Stores a superblock's words; element by element at the row's ends, and
    // everywhere where the two rows are not alike.
    __device__ __forceinline__ void store(const uint32_t (&w)[16], const ScoreParams& P, uint64_t row, const Walk<DT>& walk, uint32_t sb,
                                          int lane) const {
        using S = Score<DT>;
        if (alike && walk.inside(sb)) {
            char* a = at + (uint64_t)sb * kSuperblockBytes;
#pragma unroll
            for (int j = 0; j < kSbVectors; ++j) store16(a + j * 512, &w[4 * j]);
        } else {
            const ShardRow in = walk.shard(P, row), out = shard(P, row, walk.r);
            char* const place0 = out.base + ((int64_t)out.lo - in.lo) * S::kBytes;
#pragma unroll
            for (int j = 0; j < kSbVectors; ++j) {
                const uint32_t p = walk.place(P, sb) + (uint32_t)(j * 32 + lane) * S::VE;
                if (alike && p >= in.lo && p + S::VE <= in.hi) {
                    store16(place0 + (uint64_t)p * S::kBytes, &w[4 * j]);
                } else {
#pragma unroll
                    for (int e = 0; e < S::VE; ++e)
                        if (p + e >= in.lo && p + e < in.hi) S::store_bits(place0 + (uint64_t)(p + e) * S::kBytes, S::get(w, j, e));
                }
            }
        }
    }
};

// Which superblocks of its CTA's part [sb_lo, sb_hi) a warp takes of the
// CTA's count-th row: every 8th, from a start that moves on by one a row, so
// that the odd ones do not always fall to the same warps.
__device__ __forceinline__ uint32_t first_superblock(uint32_t sb_lo, int warp, uint32_t count) {
    return sb_lo + ((warp + count) & (kScoreWarps - 1));
}

// A warp's loads over all its rows, one superblock ahead of what it works on
// and through the ends of rows.  (Three ahead, through shared memory, was
// slower: 8192 x 131072 bf16 361 us against 352, and 189 against 169 for the
// distillation loss of half of it: the kernels are bound by their
// instructions as much as by memory.)
template <int DT>
struct Feed {
    uint32_t sb_lo, sb_hi;
    uint64_t row0, stride;      // the CTA's rows
    uint32_t count, rows;       // of the next superblock to load, and how many there are
    uint32_t sb;
    Walk<DT> walk;

    __device__ __forceinline__ uint64_t row() const { return row0 + count * stride; }
    __device__ __forceinline__ void next_row(int warp) {
        do {
            ++count;
            sb = first_superblock(sb_lo, warp, count);
        } while (count < rows && sb >= sb_hi);
        walk = Walk<DT>{};
    }
    // Loads the next superblock.  RUNS: returns how many of its runs hold a place of the row.
    template <bool RUNS>
    __device__ __forceinline__ uint32_t load(uint32_t (&w)[16], const ScoreParams& P, int warp, int lane) {
        if (count >= rows) return 0;
        walk.seek(P, row(), sb, lane);
        load_superblock<DT>(w, P, row(), walk, sb, lane);
        const uint32_t runs = RUNS ? walk.runs(P, row(), sb) : 0;
        sb += kScoreWarps;
        if (sb >= sb_hi) next_row(warp);
        return runs;
    }
    template <bool RUNS>
    __device__ __forceinline__ uint32_t start(uint32_t (&w)[16], const ScoreParams& P, uint32_t lo, uint32_t hi, uint64_t first_row,
                                              uint64_t row_stride, int warp, int lane) {
        sb_lo = lo;
        sb_hi = hi;
        row0 = first_row;
        stride = row_stride;
        rows = first_row < P.rows ? (uint32_t)((P.rows - first_row + row_stride - 1) / row_stride) : 0;
        count = 0;
        sb = first_superblock(lo, warp, 0);
        if (sb >= sb_hi && rows) next_row(warp);
        return load<RUNS>(w, P, warp, lane);
    }
    // Drops the count-th row, which is left out and whose first superblock (if it has one) is in w.
    template <bool RUNS>
    __device__ __forceinline__ uint32_t drop(uint32_t (&w)[16], uint32_t runs, const ScoreParams& P, uint32_t of, int warp, int lane) {
        if (count == of) next_row(warp);
        return first_superblock(sb_lo, warp, of) < sb_hi ? load<RUNS>(w, P, warp, lane) : runs;
    }
    // Gives work(w, sb, runs) a row's superblocks; on entry and on return w
    // holds the next one.  Two in turn, so that none is moved between registers;
    // with RUNS (the top-k kernels, whose stream has no registers to spare) one,
    // the next loaded when it has been worked on: top 64 of 2048 x 160000 bf16
    // 218 us against 240.
    template <bool RUNS, class Work>
    __device__ __forceinline__ uint32_t each(uint32_t (&w)[16], uint32_t runs, const ScoreParams& P, uint32_t first, int warp, int lane,
                                             Work work) {
        for (uint32_t s = first; RUNS && s < sb_hi; s += kScoreWarps) {
            work(w, s, runs);
            runs = load<RUNS>(w, P, warp, lane);
        }
        for (uint32_t s = first; !RUNS && s < sb_hi; s += 2 * kScoreWarps) {
            uint32_t x[16];
            const uint32_t more = load<RUNS>(x, P, warp, lane);
            work(w, s, runs);
            if (s + kScoreWarps < sb_hi) {
                runs = load<RUNS>(w, P, warp, lane);
                work(x, s + kScoreWarps, more);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = x[i];
                runs = more;
            }
        }
        return runs;
    }
};

// ---- superblocks in shared memory ----
// A warp's superblock takes 2 KiB, in the order of its places: vector j of
// lane l at 16-byte slot 32 j + l.  Each lane copies and reads back its own
// slots, so no barrier is needed; another lane's slot may be touched between
// two __syncwarp once its copy is there.
__device__ __forceinline__ void copy16(uint32_t to, const char* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// Begins to copy the superblock the walk stands at: whole vectors
// asynchronously, the row's ends element by element, -inf outside the row.
template <int DT>
__device__ __forceinline__ void begin_copy(uint4* block, const ScoreParams& P, uint64_t row, const Walk<DT>& walk, uint32_t sb, int lane) {
    using S = Score<DT>;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(block + lane);
    const char* from = walk.address(sb);
    if (walk.inside(sb)) {
#pragma unroll
        for (int j = 0; j < kSbVectors; ++j) copy16(to + j * 512, from + j * 512);
    } else {
        const ShardRow sr = walk.shard(P, row);
#pragma unroll
        for (int j = 0; j < kSbVectors; ++j) {
            const uint32_t p = walk.place(P, sb) + (uint32_t)(j * 32 + lane) * S::VE;
            if (p >= sr.lo && p + S::VE <= sr.hi) {
                copy16(to + j * 512, from + j * 512);
            } else {
                uint32_t v[4];
                load_vector<DT>(v, 0, sr, p);
                block[j * 32 + lane] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    }
}
__device__ __forceinline__ void read_block(uint32_t (&w)[16], const uint4* block, int lane) {
#pragma unroll
    for (int j = 0; j < kSbVectors; ++j) {
        const uint4 v = block[j * 32 + lane];
        w[4 * j] = v.x;
        w[4 * j + 1] = v.y;
        w[4 * j + 2] = v.z;
        w[4 * j + 3] = v.w;
    }
}

// The shard that holds column c (an fp32 estimate and a short walk).
__device__ __forceinline__ int shard_of(const ScoreParams& P, uint32_t c) {
    if (P.W == 1) return 0;
    int r = (int)((float)c * P.shards_per_col);
    r = r < 0 ? 0 : r >= P.W ? P.W - 1 : r;
    while (c < P.col0[r]) --r;
    while (c >= P.col0[r + 1]) ++r;
    return r;
}
template <int DT>
__device__ __forceinline__ const char* score_at(const ScoreParams& P, uint64_t row, uint32_t c) {
    const int r = shard_of(P, c);
    return static_cast<const char*>(P.x[r]) + (row * P.ld[r] + (c - P.col0[r])) * Score<DT>::kBytes;
}

// ---- thread-block clusters ----
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_address(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void peer_store(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" :: "r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
// For a thread that has nothing to show its peers: the other form waits until
// all its stores, a row's gradients among them, have been performed.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Eight bytes into a peer's shared memory, counted by a barrier of the peer's
// (mbarrier): what arrives there is complete without a fence here.  A fence
// at cluster scope would wait for every global store before it, and the loss-
// and-gradient kernel has a row's gradients on their way at that point.
__device__ __forceinline__ void counted_init(uint64_t* bar) {
    const uint32_t b = (uint32_t)__cvta_generic_to_shared(bar);
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(b) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void counted_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"((uint32_t)__cvta_generic_to_shared(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void counted_store(void* slot, uint64_t* bar, uint32_t rank, float a, float b) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
                 :: "r"(peer_address(slot, rank)), "f"(a), "f"(b), "r"(peer_address(bar, rank)) : "memory");
}
// Waits for a phase of the barrier; false after some seconds (the peers of a
// cluster run together and each sends before it waits, so this never is).
__device__ __forceinline__ bool counted_wait(uint64_t* bar, uint32_t parity) {
    const uint32_t b = (uint32_t)__cvta_generic_to_shared(bar);
    for (int i = 0; i < (1 << 24); ++i) {
        uint32_t done;
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done) : "r"(b), "r"(parity) : "memory");
        if (done) return true;
    }
    return false;
}

// ---- running softmax statistics ----
struct Stat {
    float x, s, u;
};
constexpr float kLn2 = 0.69314718055994531f;

constexpr float kFlatRef = 2147483648.0f;

// The reference that exponents are made against: c x - ref, off by r for every x.
struct Ref {
    float c, ref, r;
};
__device__ __forceinline__ Ref reference(float x, float c) {
    Ref f{c, __fmul_rn(x, c), 0.0f};
    if (x == neg_inf()) {
        f.ref = 0.0f;
        return f;
    }
    if (!(fabsf(f.ref) < kFlatRef)) {
        const uint32_t e = (__float_as_uint(x) >> 23) & 255;      // 2^(30 - exponent of x)
        f.c = __uint_as_float(min(284u - e, 254u) << 23);
        f.ref = __fmul_rn(x, f.c);
    }
    f.r = __fmaf_rn(x, f.c, -f.ref);
    return f;
}
__device__ __forceinline__ float undo(const Ref& f) { return ex2(-f.r); }

// A statistic against another maximum X >= x.
template <bool ENT>
__device__ __forceinline__ void rebase(Stat& a, float X, float c) {
    if (a.x == neg_inf()) {
        a.s = a.u = 0.0f;
    } else {
        const float d = fmaxf(__fmul_rn(__fadd_rn(a.x, -X), c), kFarBelow);
        const float f = ex2(d);
        if (ENT) a.u = __fmul_rn(__fmaf_rn(a.s, d, a.u), f);
        a.s = __fmul_rn(a.s, f);
    }
    a.x = X;
}

// A thread's running state.  For the entropy, scores are taken no lower than
// `least`, some 1000 below the maximum in the exponent: their terms are 0 all
// the same, and 0 * -inf (a mask) would be NaN.  One instruction a pair of
// bf16 scores; on the exponents it takes two.  `flat`: the reference is so
// large that every term is 1 or 0 and u gets nothing.
struct Running {
    Stat a;
    Ref f;
    uint32_t least;
    bool flat;
};
__device__ __forceinline__ Running start_running(float c) { return {{neg_inf(), 0.0f, 0.0f}, {c, 0.0f, 0.0f}, 0xff7fff7fu, true}; }

// One superblock, whose largest score (of this lane's) is `top`, into a thread's state.
template <int DT, bool ENT>
__device__ __forceinline__ void accumulate(Running& t, const uint32_t (&w)[16], float top, float c) {
    using S = Score<DT>;
    if (!(top <= t.a.x)) {      // a new maximum, or NaN: in this superblock or, which stays, in one before
        const float most = max_nan(t.a.x, top);
        rebase<ENT>(t.a, most, c);
        t.f = reference(most, c);
        if (ENT) {
            t.flat = !(fabsf(__fmul_rn(most, c)) < kFlatRef);
            // 1000 in the exponent or, for the rounding to the type, 1/64 of the maximum
            t.least = S::floor_word(__fadd_rn(most, -fmaxf(__fdiv_rn(1000.0f, c), fabsf(most) * 0.015625f)));
        }
    }
    const F2 cc = f2(t.f.c, t.f.c), off = f2(-t.f.ref, -t.f.ref);
    F2 s = f2(0.0f, 0.0f), u = s;
#pragma unroll
    for (int i = 0; i < S::kPairs; ++i) {
        float x0, x1, t0, t1;
        if (ENT) S::floored_pair(w, i, t.least, x0, x1);
        else S::pair(w, i, x0, x1);
        const F2 x = fma2(f2(x0, x1), cc, off);
        unpack(x, t0, t1);
        const F2 e = f2(ex2(t0), ex2(t1));
        s = add2(s, e);
        if (ENT) u = fma2(e, x, u);
    }
    float p, q;
    unpack(s, p, q);
    const float sum = __fadd_rn(p, q), k = undo(t.f);
    t.a.s = __fmaf_rn(sum, k, t.a.s);
    if (ENT) {
        unpack(u, p, q);
        const float more = __fmul_rn(__fmaf_rn(-t.f.r, sum, __fadd_rn(p, q)), k);
        if (!t.flat) t.a.u = __fadd_rn(t.a.u, more);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(~0u, v, o));
    return v;
}
// Joins the statistics of a warp's lanes; every lane gets the result.
template <bool ENT>
__device__ __forceinline__ Stat warp_join(Stat a, float c) {
    rebase<ENT>(a, redux_max_nan(a.x), c);
    a.s = warp_sum(a.s);
    if (ENT) a.u = warp_sum(a.u);
    return a;
}
// Joins the n statistics of a row's warps or CTAs (one warp; every lane gets the result).
static_assert(kScoreWarps <= 32 && kMaxScoreCluster <= 32, "a lane each");
template <bool ENT>
__device__ __forceinline__ Stat join_parts(const Stat* part, int n, int lane, float c) {
    return warp_join<ENT>(lane < n ? part[lane] : Stat{neg_inf(), 0.0f, 0.0f}, c);
}
// In the forward-only kernels the stream's threads leave their statistics of a
// row here for the row warp, which has time while the stream is in the next
// row: a join in every warp first kept the stream at its shuffles (distillation
// loss of 4096 x 131072 172 against 163 us).  Where the stream waits for the
// result (loss and gradient in one) the warps join first: 774 against 793 us.
struct LaneStats {
    float x[kThreads], s[kThreads], u[kThreads];
    template <bool ENT>
    __device__ __forceinline__ void put(const Stat& a) {
        x[threadIdx.x] = a.x;
        s[threadIdx.x] = a.s;
        if (ENT) u[threadIdx.x] = a.u;
    }
    template <bool ENT>
    __device__ __forceinline__ Stat join(int lane, float c) const {
        Stat o[kScoreWarps], b{neg_inf(), 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kScoreWarps; ++i) {
            o[i] = {x[32 * i + lane], s[32 * i + lane], ENT ? u[32 * i + lane] : 0.0f};
            b.x = max_nan(b.x, o[i].x);
        }
        b.x = redux_max_nan(b.x);
#pragma unroll
        for (int i = 0; i < kScoreWarps; ++i) {
            rebase<ENT>(o[i], b.x, c);
            b.s = __fadd_rn(b.s, o[i].s);
            if (ENT) b.u = __fadd_rn(b.u, o[i].u);
        }
        b.s = warp_sum(b.s);
        if (ENT) b.u = warp_sum(b.u);
        return b;
    }
};
// A warp's statistic of a row, into the cluster CTA `to_rank`'s array.
template <bool ENT>
__device__ __forceinline__ void push_stat(Stat* slot, int to_rank, const Stat& a) {
    const uint32_t to = peer_address(slot, to_rank);
    peer_store(to, __float_as_uint(a.x));
    peer_store(to + 4, __float_as_uint(a.s));
    if (ENT) peer_store(to + 8, __float_as_uint(a.u));
}

// What m = scale * x lost in its rounding; 0 where a whole unit and more is
// lost (a score of the type's lowest value): y is an fp32 number there.
__device__ __forceinline__ float rounding_of(float x, float scale, float m) {
    const float rho = __fmaf_rn(x, scale, -m);
    return fabsf(rho) < 1.0f ? rho : m == m ? 0.0f : m;
}

// A row's final values: the largest scaled score m, the log of the sum of
// exponentials relative to it (what the caller sees), and log s (relative to
// the unrounded scale * x); (-inf, 0, 0) for a row of nothing but -inf, NaN
// where a NaN or +inf was seen.
struct Final {
    float m, logs, log_s;
};
__device__ __forceinline__ Final finish(const Stat& a, float scale) {
    Final f;
    f.m = __fmul_rn(a.x, scale);
    if (f.m == neg_inf()) {
        f.logs = f.log_s = 0.0f;
    } else if (!(f.m < __int_as_float(0x7f800000))) {
        f.m = f.logs = f.log_s = quiet_nan();
    } else {
        f.log_s = logf(a.s);
        f.logs = __fadd_rn(f.log_s, rounding_of(a.x, scale, f.m));
    }
    return f;
}
// log p of a score: -inf for a masked one, NaN in a row that has NaN and for a
// column past the vocabulary, whose score is given as NaN.
__device__ __forceinline__ float log_prob(float x, const Stat& a, const Final& f, float scale) {
    if (f.m != f.m || x != x) return quiet_nan();
    if (x == neg_inf() || f.m == neg_inf()) return neg_inf();
    return __fmaf_rn(__fadd_rn(x, -a.x), scale, -f.log_s);
}

// The reference of saved statistics: the largest score x_m again from
// m = scale * x_m rounded, so that y - m = scale (x - x_m) + rho.  For bf16
// scores the quotient rounds to x_m itself.  For fp32 it may be off by a step,
// which rho makes good but for scores so large that a step is whole units:
// there the farther of the scores that round to m is taken, which finds a
// mask of the type's lowest value.
struct SavedRef {
    Ref f;
    float x, rho;
};
template <int DT>
__device__ __forceinline__ SavedRef saved_reference(float m, float scale, float c) {
    SavedRef k;
    k.x = m;
    k.rho = 0.0f;
    if (m != neg_inf()) {
        k.x = __fdiv_rn(m, scale);
        if (DT == MR_BF16) {
            uint32_t w;
            asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(w) : "f"(k.x));
            k.x = __uint_as_float(w << 16);
        } else if (fabsf(m) > 1e30f) {
            const float lowest = __int_as_float(0xff7fffff);
            k.x = fmaxf(k.x, lowest);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float next = __uint_as_float(__float_as_uint(k.x) + 1);
                if (k.x != lowest && __fmul_rn(next, scale) == m) k.x = next;
            }
        }
        k.rho = rounding_of(k.x, scale, m);
    }
    k.f = reference(k.x, c);
    return k;
}

// ---- barriers inside a CTA ----
// The forward kernels' CTAs: 8 warps that stream a row's scores and one warp
// that does everything else of it.  That warp fetches the next rows' ids and
// lists ahead of the stream, and joins the statistics of a row while the
// stream is in the next one, so the stream never waits for a chain of small
// loads.  They meet at named barriers; what passes through shared memory is
// double-buffered by the row's parity:
//   kRowReady + parity   the row warp has set a row up; the stream waits before
//                        it starts the row (loss and gradient in one: before the
//                        last row's gradients).  The log probabilities' row warp
//                        sets up the first two rows before it begins and row
//                        i+2 when it has joined row i; the distillation's the
//                        first one, and row i+1 before it joins row i
//   kRowDone + parity    the stream's warps have left their results of row i;
//                        the row warp waits before it joins them
//   kRowStep             loss and gradient in one: what row i's gradients need is
//                        there
//   kRowHelp             the runs that hold the row's best scores are picked; the
//   kRowHelped           stream's warps of the first CTA have read their share.
//                        In the loss and gradient: the last row is stored
// So the stream is at most one row ahead and no buffer of row i is still in
// use when row i+2 is set up.
enum { kRowReady = 1, kRowDone = 3, kRowStep = 5, kRowHelp = 6, kRowHelped = 7 };     // 0 is __syncthreads
__device__ __forceinline__ void bar_sync(int id) { asm volatile("barrier.cta.sync %0, %1;" :: "r"(id), "n"(kScoreThreads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("barrier.cta.arrive %0, %1;" :: "r"(id), "n"(kScoreThreads) : "memory"); }

}  // namespace mr
