// distill_kernel.cu -- distillation from a teacher's top logits over rows of
// scores in shards: the loss, its gradient, and both in one call.
//
// The teacher gives a list L of up to 128 (column, value) pairs per row.  With
// q the teacher's mass (over the list: renormalised, or as given with the rest
// q_R = 1 - sum q as one more outcome), p = softmax(scale * x) and p_R the
// student's mass outside the list,
//     loss = sum_L q (log q - log p)  [+ q_R (log q_R - log p_R)].
// The stream sums the places OUTSIDE the list only, with a maximum of their
// own: p_R then has full relative precision where 1 - sum_L p would cancel.
// The listed scores are gathered one by one and joined at the end.
//
// Gradient: with Q = sum q + q_R,
//     listed:  scale * g * (p Q - q)
//     others:  scale * g * e^(y - m_R) / S_R * (p_R Q - q_R)
// (S_R the rest's sum relative to its maximum m_R): one exponential and one
// product per place, and no quotient of small masses.
//
// The forward kernel streams a row's scores with 8 warps while a ninth, the row
// warp, sets the next row up (its list as places, the teacher's masses, the listed
// scores) and joins the last one.  A score that is in the list becomes -inf
// before it is summed.  With the gradient in the same call (STEP) a cluster
// of CTAs keeps the row in shared memory: pass 1 sums it, the row warps exchange
// their CTAs' statistics, pass 2 turns it into gradients, and as a block of
// it is used up the next row's is copied there.  While the statistics are
// exchanged, the stream's last warp works out the next row's masses: on the row
// warp they kept the stream waiting (8192 x 131072 bf16 737 us against 701).
//
// What bounds them (GB300, bf16): the loss alone memory, 6.4 TB/s of 6.69 at
// 4096 x 131072 with 64 entries (163 us); its gradient 5.9 TB/s (351 us at 4096 x
// 128000, 100 entries), the units' own reading of the list; loss and gradient
// in one 6.1 TB/s (693 us at 8192 x 131072, one row in 32 left out): two passes over a row cost some 460
// instructions a 2 KiB superblock, and the stream waits at each row's join.
#include "score_kernel.cuh"

namespace mr {

namespace {

constexpr int kListRegs = MR_MAX_TEACHER / 32;
constexpr int kTeacherWarp = kScoreWarps - 1;       // no warp has fewer superblocks
// What up to 128 fp32 log probabilities may lack of 1, or have over it, by their
// rounding and that of the log sum they were taken from: 128 additions' u each,
// the exponentials' 2^-22 and the rounding of their arguments, 2^-22 a nat of
// entropy (at most 4.9 over 128 places): below 2^-18.
constexpr float kRoundingMass = 0x1p-18f;
constexpr uint32_t kNoPlace = ~0u;     // past every superblock: a row has fewer than 2^32 - 2^10 places

// A warp's copy of a row's list: entry k = lane + 32 i, in the first `regs` of
// the four registers.  Every instruction here is one of the warp that the
// stream waits for, or of a unit of the gradient's: what a list shorter than
// 97 entries does not need is skipped, and what two steps share is kept.
struct List {
    uint32_t place[kListRegs];      // in units of scores, counted through the row's superblocks; kNoPlace if absent
    bool some;                      // any entry at all
};
template <class F>
__device__ __forceinline__ void each_reg(int regs, F f) {
#pragma unroll
    for (int i = 0; i < kListRegs; ++i)
        if (i < regs) f(i);
}

// The list as it lies in memory.
struct RawList {
    long long id[kListRegs];
    float v[kListRegs];
};
__device__ __forceinline__ void load_raw(RawList& R, const ScoreParams& P, uint64_t row, int regs, int lane) {
    const long long* ids = P.t_ids + row * P.K + lane;
    const float* val = P.t_val + row * P.K + lane;
    each_reg(regs, [&](int i) {
        R.id[i] = -1;
        R.v[i] = neg_inf();
        if (lane + 32 * i < P.K) {
            R.id[i] = ids[32 * i];
            R.v[i] = val[32 * i];
        }
    });
}
// Places, into `values` the teacher's values (-inf for no entry, NaN for a column
// past the vocabulary), and by entry(i, score's address, rank, column of the
// rank) whatever else is to be had of an entry.
template <int DT, class Entry>
__device__ __forceinline__ void place_list(List& L, float* values, const RawList& R, const ScoreParams& P, uint64_t row, int regs, int lane,
                                           Entry entry) {
    using S = Score<DT>;
    bool some = false;
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) L.place[i] = kNoPlace;
    each_reg(regs, [&](int i) {
        float v = neg_inf();
        if (R.id[i] >= 0) {
            some = true;
            v = quiet_nan();
            if (R.id[i] < (long long)P.vocab) {
                const uint32_t id = (uint32_t)R.id[i];
                const int r = shard_of(P, id);
                const uint32_t column = id - P.col0[r];
                const uintptr_t start = reinterpret_cast<uintptr_t>(P.x[r]) + row * P.ld[r] * S::kBytes;
                v = R.v[i];
                L.place[i] = (P.sb0[r] << S::kLogSb) + column + (uint32_t)(start & 15) / S::kBytes;
                entry(i, reinterpret_cast<const char*>(start + (uint64_t)column * S::kBytes), r, column);
            }
        }
        values[lane + 32 * i] = v;
    });
    L.some = __any_sync(~0u, some);
}

// ---- the teacher's masses, beyond fp32 ----
// The mass outside the list is 1 - sum q: where the list holds nearly all of
// it, sums and exponentials of fp32 would leave the rounding of q in its place
// (a remainder of 1e-6 off by 4 to 13 %).  So an exponential is the sum of two
// floats, and the sum over the list is one of integers.
struct Pair {
    float h, l;
};
// 2^(j/32), the part of it in a float and the rest.  The forward kernels keep
// a copy in shared memory: a load of it from beyond took its turn behind the
// stream's, some 1000 cycles a row of the step.
__device__ const float2 kTwoToThe32nds[32] = {
    {1.0f, 0.0f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f},
    {0x1.306fep+0f, 0x1.4636e2p-25f}, {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c561p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp+0f, -0x1.f8b55p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f}, {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f77p+0f, -0x1.a09438p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f}, {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246ebp-26f},
};
// e^(h + l) (l is small beside h) to 2^-33 relative.  Table-driven (P. T. P. Tang, Table-driven
// implementation of the exponential function, 1989): h + l = k ln 2 / 32 + r,
// e^r - 1 by its series, as |r| < 0.011.  0 below e^-87, NaN for NaN.
__device__ __forceinline__ Pair exp_pair(float h, float l, const float2* two_to_the_32nds) {
    constexpr float kRound = 12582912.0f;       // 1.5 * 2^23: an fp32 sum with it is rounded to a whole number
    constexpr float kLn2 = 0x1.62e43p-6f, kLn2Rest = -0x1.05c61p-34f;       // ln 2 / 32
    const float x = h < -88.0f ? -88.0f : h > 89.0f ? 89.0f : h;
    const float shifted = __fmaf_rn(x, 46.166241f, kRound), k = __fadd_rn(shifted, -kRound);
    const int i = __float_as_int(shifted) - __float_as_int(kRound);
    const float2 t = two_to_the_32nds[i & 31];
    // x - k ln 2 / 32, what the product and the difference lost put back
    const float p = __fmul_rn(k, kLn2), p_low = __fmaf_rn(k, kLn2, -p), d = __fadd_rn(x, -p);
    const float r = __fadd_rn(d, -p_low), r_low = __fmaf_rn(-k, kLn2Rest, __fadd_rn(__fadd_rn(__fadd_rn(d, -r), -p_low), l));
    const float series = __fmaf_rn(__fmul_rn(r, r), __fmaf_rn(r, __fmaf_rn(r, 0.041666667f, 0.16666667f), 0.5f), __fmaf_rn(r_low, r, r_low));
    const float a = __fmul_rn(t.x, r), a_low = __fmaf_rn(t.x, r, -a), e = __fadd_rn(t.x, a);
    const float low = __fadd_rn(__fadd_rn(__fadd_rn(t.x, -e), a), __fadd_rn(a_low, __fmaf_rn(t.x, series, __fmaf_rn(t.y, r, t.y))));
    const float whole = __fadd_rn(e, low), rest = __fadd_rn(low, -__fadd_rn(whole, -e));
    const float scale = x < -87.0f ? 0.0f : __int_as_float(((i >> 5) + 127) << 23);
    return {__fmul_rn(whole, scale), __fmul_rn(rest, scale)};
}
// The sum of masses, in units of 2^-20 and of 2^-42 (at most 128 of them, none
// over 2).  A sum with 1.5 * 2^(n + 23) is rounded to whole units of 2^n, which
// its last bits then count: no conversion, whose unit the 2^x of the stream
// keeps busy.
struct MassSum {
    int high = 0, low = 0;
    __device__ __forceinline__ void add(Pair q) {
        constexpr float kHigh = 12.0f, kLow = 0x1.8p-19f;
        const float h = __fadd_rn(q.h, kHigh), l = __fadd_rn(__fadd_rn(__fadd_rn(q.h, -__fadd_rn(h, -kHigh)), q.l), kLow);
        high += __float_as_int(h) - __float_as_int(kHigh);
        low += __float_as_int(l) - __float_as_int(kLow);
    }
    __device__ __forceinline__ void over_warp() {
        high = __reduce_add_sync(~0u, high);
        low = __reduce_add_sync(~0u, low);
    }
};

// The teacher's side of a row: its masses, what they leave, and what log q is
// made of.  It lives in shared memory and is worked out by one warp, entry
// k = lane + 32 i after the other: unrolled, its registers crowd the stream's,
// and what spills to local memory takes its turn behind the stream's stores (a
// row of the step 4000 cycles longer).
struct Teacher {
    float v[MR_MAX_TEACHER], q[MR_MAX_TEACHER], low[MR_MAX_TEACHER];
    float2 rest;            // q_rest and Q,
    float2 log_terms;       // ref and log_total
};
// log q is the value (the tail mode) or teacher_scale (value - ref) - log_total.
__device__ __forceinline__ float log_mass(float v, float2 terms, const ScoreParams& P) {
    return P.tail ? v : __fadd_rn(__fmul_rn(__fadd_rn(v, -terms.x), P.teacher_scale), -terms.y);
}
// From the values (of 32 regs entries) the rest.
__device__ __forceinline__ void teacher_mass(Teacher& T, const ScoreParams& P, int regs, const float2* powers, int lane) {
    MassSum sum;
    const int end = lane + 32 * regs;
    if (P.tail) {
        bool odd = false;       // no log probability: its mass is over 2, or NaN
#pragma unroll 1
        for (int k = lane; k < end; k += 32) {
            const Pair q = exp_pair(T.v[k], 0.0f, powers);
            T.q[k] = q.h;
            odd |= !(q.h <= 2.0f);
            sum.add(q);
        }
        sum.over_warp();
        float rest = __fmaf_rn((float)sum.low, -0x1p-42f, __fmul_rn((float)((1 << 20) - sum.high), 0x1p-20f));
        if (__any_sync(~0u, odd)) {
            float total = 0.0f;
#pragma unroll 1
            for (int k = lane; k < end; k += 32) total = __fadd_rn(total, T.q[k]);
            rest = __fadd_rn(1.0f, -warp_sum(total));
        }
        if (lane == 0) {
            T.rest = make_float2(rest < 0.0f ? 0.0f : rest, rest < 0.0f ? __fadd_rn(1.0f, -rest) : rest == rest ? 1.0f : rest);
            T.log_terms = make_float2(0.0f, 0.0f);
        }
    } else {
        float m = neg_inf();
#pragma unroll 1
        for (int k = lane; k < end; k += 32) m = max_nan(m, T.v[k]);
        m = redux_max_nan(m);
        const float ref = m == neg_inf() ? 0.0f : m;
#pragma unroll 1
        for (int k = lane; k < end; k += 32) {
            // teacher_scale (v - m), what the difference and the product lost put back
            const float v = T.v[k], d = __fadd_rn(v, -ref), from_v = __fadd_rn(d, -v);
            const float d_low = __fadd_rn(__fadd_rn(v, -__fadd_rn(d, -from_v)), -__fadd_rn(ref, from_v));
            const float y = __fmul_rn(d, P.teacher_scale);
            // no low part where there is no mass: -inf, or out of range
            const float low = y < -88.0f ? 0.0f : __fmaf_rn(d_low, P.teacher_scale, __fmaf_rn(d, P.teacher_scale, -y));
            const Pair q = exp_pair(y, low, powers);
            T.q[k] = q.h;
            T.low[k] = q.l;
            sum.add(q);
        }
        sum.over_warp();
        const bool none = m == neg_inf();
        const float high = __fmul_rn((float)sum.high, 0x1p-20f), total = __fmaf_rn((float)sum.low, 0x1p-42f, high);
        const float total_low = __fmaf_rn((float)sum.low, 0x1p-42f, __fadd_rn(high, -total));
        const float inv = none ? 0.0f : m == m ? __fdiv_rn(1.0f, total) : m;
#pragma unroll 1
        for (int k = lane; k < end; k += 32) {
            // the quotient of the two sums, rounded once
            const float h = T.q[k], x = __fmul_rn(h, inv);
            T.q[k] = __fmaf_rn(inv, __fadd_rn(__fmaf_rn(-x, total, h), __fmaf_rn(-x, total_low, T.low[k])), x);
        }
        if (lane == 0) {
            T.rest = make_float2(0.0f, none ? 0.0f : m == m ? 1.0f : m);
            T.log_terms = make_float2(ref, none ? 0.0f : logf(total));
        }
    }
    __syncwarp();
}

// The rounds (every `step`-th superblock from `first`, up to `end`) in which an
// entry of the list lies, as bits round mod 32.
template <int DT>
__device__ __forceinline__ uint32_t rounds_with_entries(const List& L, uint32_t first, uint32_t end, uint32_t step) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) {
        const uint32_t sb = L.place[i] >> Score<DT>::kLogSb, d = sb - first;
        if (sb >= first && sb < end && d % step == 0) bits |= 1u << ((d / step) & 31);
    }
    return __reduce_or_sync(~0u, bits);
}
// Takes the listed places of superblock sb out of its block in shared memory,
// whose copies are there.
template <int DT>
__device__ __forceinline__ void mask_listed(uint4* block, const List& L, uint32_t sb) {
    using S = Score<DT>;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kListRegs; ++i)
        if ((L.place[i] >> S::kLogSb) == sb)
            S::mask_one(reinterpret_cast<char*>(block) + (size_t)(L.place[i] & ((1u << S::kLogSb) - 1)) * S::kBytes);
    __syncwarp();
}
// The same for words in registers, through a block of the warp's: picking
// them out in registers, 32 tests a lane, costs as much as the sum.
template <int DT>
__device__ __forceinline__ void mask_listed(uint32_t (&w)[16], const List& L, uint32_t sb, uint4* block, int lane) {
#pragma unroll
    for (int j = 0; j < kSbVectors; ++j) block[j * 32 + lane] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    mask_listed<DT>(block, L, sb);
    read_block(w, block, lane);
}

// And in registers alone, for the superblocks of a row that is too long for
// its cache, which leaves no shared memory.
template <int DT>
__device__ __forceinline__ void mask_listed_in_registers(uint32_t (&w)[16], const List& L, uint32_t sb, int lane) {
    using S = Score<DT>;
    uint32_t mine = 0;      // this lane's listed places, bit VE * vector + element
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) {
        uint32_t hit = __ballot_sync(~0u, (L.place[i] >> S::kLogSb) == sb);
        while (hit) {
            const uint32_t p = __shfl_sync(~0u, L.place[i], __ffs(hit) - 1) & ((1u << S::kLogSb) - 1);
            hit &= hit - 1;
            if ((int)((p >> S::kLogVe) & 31) == lane) mine |= 1u << ((p >> (S::kLogVe + 5)) * S::VE + (p & (S::VE - 1)));
        }
    }
#pragma unroll
    for (int j = 0; j < kSbVectors; ++j)
#pragma unroll
        for (int e = 0; e < S::VE; ++e)
            if ((mine >> (j * S::VE + e)) & 1) S::put(w, j, e, S::kBytes == 2 ? S::kFill & 0xffffu : S::kFill);
}

// What the gradient outside the list needs: coef * 2^(c x - ref); c = 0 for a
// row whose teacher has no mass, which gets zeros whatever its scores are.
struct Coef {
    float c, ref, coef;
};

// The places of a superblock turned into gradients.
template <int DT>
__device__ __forceinline__ void rest_gradient(uint32_t (&w)[16], const Coef& k) {
    using S = Score<DT>;
    const F2 cc = f2(k.c, k.c), off = f2(-k.ref, -k.ref), f = f2(k.coef, k.coef);
#pragma unroll
    for (int i = 0; i < S::kPairs; ++i) {
        float x0, x1, t0, t1;
        S::pair(w, i, x0, x1);
        unpack(fma2(f2(x0, x1), cc, off), t0, t1);
        unpack(mul2(f2(ex2(t0), ex2(t1)), f), x0, x1);
        S::set_pair(w, i, x0, x1);
    }
}

template <int DT, bool STEP>
__global__ void __launch_bounds__(kScoreThreads, 3) distill_kernel(const __grid_constant__ ScoreParams P) {
    using S = Score<DT>;
    extern __shared__ uint4 smem[];         // STEP: this CTA's part of a row, [round][warp] blocks
    __shared__ uint4 bounce[STEP ? 1 : kScoreWarps][STEP ? 1 : kSbVectors * 32];      // a block of each warp
    __shared__ Stat part[2][kMaxScoreCluster];      // the CTAs' statistics
    __shared__ LaneStats stats[STEP ? 1 : 2];       // from these threads',
    __shared__ Stat warp_part[2][kScoreWarps];      // or for STEP from these warps'
    __shared__ float2 step_part[2][kMaxScoreCluster];       // STEP: the CTAs', as x and s,
    __shared__ uint64_t step_bar[2];                        // and the barriers that count them
    __shared__ uint32_t s_place[2][MR_MAX_TEACHER];
    __shared__ int row_out[2];              // the row is left out
    __shared__ uint32_t s_mask[2][STEP ? MR_MAX_TEACHER : 1];       // STEP: where the entries lie in the cache,
    // and in the gradients of this CTA's part: the last row's are stored when the
    // stream's vector stores of that row are done, while the next but one is set up
    __shared__ char* s_out[3][STEP ? MR_MAX_TEACHER : 1];
    __shared__ float s_listed[STEP ? MR_MAX_TEACHER : 1];
    __shared__ Coef s_coef;
    __shared__ Teacher s_teacher[2];
    __shared__ float2 powers[32];           // kTwoToThe32nds, the row warp's copy

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = P.csize, crank = C > 1 ? (int)cluster_rank() : 0;
    const uint32_t nsb = P.sb0[P.W];
    const uint32_t sb_lo = (uint32_t)((uint64_t)nsb * crank / C), sb_hi = (uint32_t)((uint64_t)nsb * (crank + 1) / C);
    const uint64_t stride = gridDim.x / C;
    uint64_t row = blockIdx.x / C;
    const int regs = (P.K + 31) / 32;
    if (STEP && C > 1 && threadIdx.x == 0) {
        counted_init(&step_bar[0]);
        counted_init(&step_bar[1]);
    }
    if (C > 1) cluster_arrive();        // every CTA of the cluster has started: waited for before the first store to a peer
    if (warp == kScoreWarps) powers[lane] = kTwoToThe32nds[lane];
    pdl_enter();

    if (warp < kScoreWarps) {
        // ================= the stream =================
        constexpr int kBlock = kSbVectors * 32;
        uint32_t w[16];
        Feed<DT> feed;          // without STEP
        uint32_t ahead_runs = 0;
        Walk<DT> walk;          // STEP: this row, and the next one's copies
        auto block_of = [&](uint32_t round) { return smem + (round * kScoreWarps + warp) * kBlock; };
        auto rounds_of = [&](uint32_t first) { return first < sb_hi ? (sb_hi - first + kScoreWarps - 1) / kScoreWarps : 0; };
        if constexpr (STEP) {
            const uint32_t first = sb_lo + warp;
            if (row < P.rows)
                for (uint32_t i = 0; i < min(rounds_of(first), P.cache_rounds); ++i) {
                    walk.seek(P, row, first + i * kScoreWarps, lane);
                    begin_copy<DT>(block_of(i), P, row, walk, first + i * kScoreWarps, lane);
                }
            copies_commit();
        } else {
            ahead_runs = feed.template start<false>(w, P, sb_lo, sb_hi, row, stride, warp, lane);
        }
        bool waited = C == 1;
        int parity = 0;
        if (STEP && row < P.rows) bar_sync(kRowReady);
        for (uint32_t count = 0; row < P.rows; row += stride, parity ^= 1, ++count) {
            if (!STEP) bar_sync(kRowReady + parity);
            const bool out = row_out[parity];
            const uint32_t first = STEP ? sb_lo + warp : first_superblock(sb_lo, warp, count);
            List L;
            auto take_list = [&] {
#pragma unroll
                for (int i = 0; i < kListRegs; ++i) L.place[i] = i < regs ? s_place[parity][lane + 32 * i] : kNoPlace;
            };
            const uint32_t rounds = rounds_of(first), cached = STEP ? min(rounds, P.cache_rounds) : 0;
            Running run = start_running(P.c);
            if constexpr (!STEP) {
                if (out) {
                    ahead_runs = feed.template drop<false>(w, ahead_runs, P, count, warp, lane);
                } else {
                    take_list();
                    const uint32_t entries = rounds_with_entries<DT>(L, first, sb_hi, kScoreWarps);
                    ahead_runs = feed.template each<false>(w, ahead_runs, P, first, warp, lane, [&](uint32_t (&x)[16], uint32_t sb, uint32_t) {
                        if ((entries >> (((sb - first) / kScoreWarps) & 31)) & 1) mask_listed<DT>(x, L, sb, bounce[warp], lane);
                        accumulate<DT, false>(run, x, S::template max_words<16>(x), P.c);
                    });
                }
            } else {
                copies_wait();          // this row's copies are there
                if (!out) {
                    // the listed places in this warp's blocks leave the sums
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kListRegs; ++i)
                        if (i < regs) {
                            const uint32_t at = s_mask[parity][lane + 32 * i];
                            if (at >> 28 == (uint32_t)warp) S::mask_one(reinterpret_cast<char*>(smem) + (at & 0xfffffffu));
                        }
                    __syncwarp();
                    for (uint32_t i = 0; i < cached; ++i) {
                        read_block(w, block_of(i), lane);
                        accumulate<DT, false>(run, w, S::template max_words<16>(w), P.c);
                    }
                    if (cached < rounds) {      // a row longer than the cache
                        take_list();
                        const uint32_t entries = rounds_with_entries<DT>(L, first, sb_hi, kScoreWarps);
                        walk = Walk<DT>{};
                        for (uint32_t i = cached; i < rounds; ++i) {
                            const uint32_t sb = first + i * kScoreWarps;
                            walk.seek(P, row, sb, lane);
                            load_superblock<DT>(w, P, row, walk, sb, lane);
                            if ((entries >> (i & 31)) & 1) mask_listed_in_registers<DT>(w, L, sb, lane);
                            accumulate<DT, false>(run, w, S::template max_words<16>(w), P.c);
                        }
                    }
                }
            }
            if (!out) {
                if constexpr (STEP) {
                    const Stat a = warp_join<false>(run.a, P.c);
                    if (lane == 0) warp_part[parity][warp] = a;
                } else {
                    stats[parity].template put<false>(run.a);
                }
            }
            bar_arrive(kRowDone + parity);
            if (!STEP && C > 1) {
                if (!waited) cluster_wait();
                cluster_arrive_relaxed();
                waited = false;     // for this row's phase: before the next one, or the end
            }
            if constexpr (STEP) {
                Coef coef{P.c, 0.0f, 0.0f};
                const uint64_t next_row = row + stride;
                const bool more = next_row < P.rows;
                if (more) {
                    bar_sync(kRowReady + (parity ^ 1));
                    if (warp == kTeacherWarp) teacher_mass(s_teacher[parity ^ 1], P, regs, powers, lane);
                }
                bar_sync(kRowStep);
                if (!out) coef = s_coef;
                const bool zero = out || coef.c == 0.0f;
                // The next row's copies go into the blocks as they empty; a row that
                // is left out has none.
                const bool copy = more && !row_out[parity ^ 1];
                Walk<DT> ahead;
                walk = Walk<DT>{};
                Output<DT> to;
                uint32_t sb = first;
                for (uint32_t i = 0; i < rounds; ++i, sb += kScoreWarps) {
                    if (walk.seek(P, row, sb, lane)) to.follow(P, row, walk, lane);
                    if (zero) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = 0;
                    } else {
                        if (i < cached) read_block(w, block_of(i), lane);
                        else load_superblock<DT>(w, P, row, walk, sb, lane);
                        rest_gradient<DT>(w, coef);
                    }
                    if (copy && i < cached) {
                        ahead.seek(P, next_row, sb, lane);
                        begin_copy<DT>(block_of(i), P, next_row, ahead, sb, lane);
                    }
                    to.store(w, P, row, walk, sb, lane);
                }
                copies_commit();
            }
        }
        if (STEP) bar_arrive(kRowHelped);       // the last row's vector stores are done
        if (!waited) cluster_wait();
        if (STEP && C > 1) {        // no CTA leaves while a peer may send to it
            cluster_arrive_relaxed();
            cluster_wait();
        }
        return;
    }

    // ================= the row warp =================
    const bool joins = STEP || crank == 0;
    RawList raw;        // the list after the one in `cur` / `next`
    List cur{}, next{};
    float x[kListRegs], x_next[kListRegs];
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) x_next[i] = neg_inf();
    auto store_listed = [&](int slot) {
        each_reg(regs, [&](int i) {
            char* const to = s_out[slot][lane + 32 * i];
            if (to) S::store_one(to, s_listed[lane + 32 * i]);
        });
    };
    // Sets a row up: places for the stream, and the listed scores.
    auto set_up = [&](uint64_t r, int par, int slot) {
        each_reg(regs, [&](int i) {
            x_next[i] = neg_inf();
            if (STEP) s_out[slot][lane + 32 * i] = nullptr;
        });
        place_list<DT>(next, s_teacher[par].v, raw, P, r, regs, lane, [&](int i, const char* score, int rank, uint32_t column) {
            if (joins) x_next[i] = S::load_one(score);
            if (STEP) {
                const uint32_t sb = next.place[i] >> S::kLogSb;
                if (sb >= sb_lo && sb < sb_hi)
                    s_out[slot][lane + 32 * i] = static_cast<char*>(P.g[rank]) + (r * P.ldg[rank] + column) * S::kBytes;
            }
        });
        each_reg(regs, [&](int i) {
            if (STEP) {
                const uint32_t sb = next.place[i] >> S::kLogSb, d = sb - sb_lo;
                s_mask[par][lane + 32 * i] = sb >= sb_lo && sb < sb_hi && d / kScoreWarps < P.cache_rounds
                    ? (d % kScoreWarps) << 28 | (d * kSuperblockBytes + (next.place[i] & ((1u << S::kLogSb) - 1)) * S::kBytes) : ~0u;
            }
            if (!STEP || P.cache_rounds * kScoreWarps < sb_hi - sb_lo) s_place[par][lane + 32 * i] = next.place[i];
        });
        if (lane == 0) row_out[par] = !next.some;
        bar_arrive(kRowReady + par);
        if (r + stride < P.rows) load_raw(raw, P, r + stride, regs, lane);
    };
    __syncwarp();       // of the lanes' entries of powers
    if (row < P.rows) {
        load_raw(raw, P, row, regs, lane);
        set_up(row, 0, 0);
        if (STEP) teacher_mass(s_teacher[0], P, regs, powers, lane);       // the stream has no wait yet
    }
    if (C > 1) cluster_wait();
    int parity = 0;
    uint32_t turn = 0;      // of the two counted barriers
    int slot = 0, last = -1;        // of s_out: this row's and the last one's
    for (; row < P.rows; row += stride, parity ^= 1) {
        const int after = slot == 2 ? 0 : slot + 1;
        cur = next;
#pragma unroll
        for (int i = 0; i < kListRegs; ++i) x[i] = x_next[i];
        if (row + stride < P.rows) set_up(row + stride, parity ^ 1, after);
        const bool out = !cur.some;
        const Teacher& t = s_teacher[parity];
        Stat l{neg_inf(), 0.0f, 0.0f};      // the listed scores, as one more statistic
        float g = 0.0f;
        if (joins && !out) {
            if (STEP) g = __fmul_rn(P.scale, P.g_row[row]);
            else teacher_mass(s_teacher[parity], P, regs, powers, lane);
            each_reg(regs, [&](int i) { l.x = max_nan(l.x, x[i]); });
            l.x = redux_max_nan(l.x);
            if (l.x != neg_inf()) {
                each_reg(regs, [&](int i) { l.s = __fadd_rn(l.s, expf(__fmul_rn(__fadd_rn(x[i], -l.x), P.scale))); });
                l.s = warp_sum(l.s);
            }
        }
        bar_sync(kRowDone + parity);
        Stat b{neg_inf(), 0.0f, 0.0f};
        if (!out) {
            if constexpr (STEP) b = join_parts<false>(warp_part[parity], kScoreWarps, lane, P.c);
            else b = stats[parity].template join<false>(lane, P.c);
        }
        if (STEP && C > 1 && !out) {
            // in turn by the rows that take part: a peer sends the row after next
            // only when it has this CTA's of the next, sent after this one is read
            const int slot = turn & 1;
            if (lane == 0) counted_expect(&step_bar[slot], (uint32_t)C * 8);
            __syncwarp();
            if (lane < C) counted_store(&step_part[slot][crank], &step_bar[slot], lane, b.x, b.s);
            const bool came = counted_wait(&step_bar[slot], turn >> 1 & 1);
            ++turn;
            Stat o{neg_inf(), 0.0f, 0.0f};
            if (lane < C) o = {step_part[slot][lane].x, step_part[slot][lane].y, 0.0f};
            if (!came) o.x = quiet_nan();
            b = warp_join<false>(o, P.c);
        } else if (!STEP && C > 1) {
            if (!out && lane == 0) push_stat<false>(&part[parity][crank], 0, b);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            if (joins && !out) b = join_parts<false>(part[parity], C, lane, P.c);
        }
        if (!joins) continue;
        if (out) {
            if (lane == 0 && crank == 0) {
                if (P.loss) P.loss[row] = 0.0f;
                if (P.stats) {
                    P.stats[4 * row] = P.stats[4 * row + 2] = neg_inf();
                    P.stats[4 * row + 1] = P.stats[4 * row + 3] = 0.0f;
                }
            }
            if (STEP) {
                bar_arrive(kRowStep);
                if (last >= 0) store_listed(last);
                last = slot;
                slot = after;
            }
            continue;
        }
        const float q_rest = t.rest.x, Q = t.rest.y;
        Stat all{max_nan(b.x, l.x), 0.0f, 0.0f}, r = b;
        rebase<false>(r, all.x, P.c);
        rebase<false>(l, all.x, P.c);
        all.s = __fadd_rn(r.s, l.s);
        if (STEP) {
            // The stream waits for this: no logarithm in it.  p_R = r.s / all.s
            // An empty row (its y all -inf) gets zeros, one with NaN or +inf NaN.
            const float y = __fmul_rn(all.x, P.scale);
            const float inv = fabsf(y) < __int_as_float(0x7f800000) ? reciprocal(all.s) : y == neg_inf() ? 0.0f : quiet_nan();
            const bool spoilt = inv != inv || Q != Q;       // every gradient is NaN
            if (lane == 0) {
                const Ref k = reference(b.x, P.c);
                const float mass = __fmul_rn(g, __fmaf_rn(__fmul_rn(r.s, inv), Q, -q_rest));
                const float none_left = spoilt ? quiet_nan() : 0.0f;        // every place there is masked
                s_coef = {Q == 0.0f ? 0.0f : k.c, k.ref,
                          __fmul_rn(b.x, P.scale) == neg_inf() ? none_left : __fmul_rn(__fmul_rn(mass, reciprocal(b.s)), undo(k))};
            }
            bar_arrive(kRowStep);
            // the row before: its vector stores were done when the stream came to this one
            if (last >= 0) store_listed(last);
            last = slot;
            slot = after;
            each_reg(regs, [&](int i) {
                const float p = __fmul_rn(exp_near(__fmul_rn(__fadd_rn(x[i], -all.x), P.scale)), inv);     // as the gradient's own call
                const bool no_part = Q == 0.0f || (__fmul_rn(x[i], P.scale) == neg_inf() && !spoilt);
                s_listed[lane + 32 * i] = no_part ? 0.0f : __fmul_rn(g, __fmaf_rn(p, Q, -t.q[lane + 32 * i]));
            });
        }
        if (crank != 0) continue;
        const Final f = finish(all, P.scale), rest = finish(b, P.scale);
        const float logp_rest = rest.m == neg_inf() ? neg_inf()
                              : __fmaf_rn(__fadd_rn(b.x, -all.x), P.scale, __fadd_rn(rest.log_s, -f.log_s));
        float loss = 0.0f;
        each_reg(regs, [&](int i) {
            const float q = t.q[lane + 32 * i], logq = log_mass(t.v[lane + 32 * i], t.log_terms, P);
            if (!(q == 0.0f)) loss = __fadd_rn(loss, __fmul_rn(q, __fadd_rn(logq, -log_prob(x[i], all, f, P.scale))));
        });
        loss = warp_sum(loss);
        // Against a student with no place outside the list, what the rounding of the
        // given log probabilities leaves of 1 is no mass: the loss would be +inf or
        // not by their last bits.
        if (!(q_rest <= (rest.m == neg_inf() ? kRoundingMass : 0.0f))) loss = __fadd_rn(loss, __fmul_rn(q_rest, __fadd_rn(logf(q_rest), -logp_rest)));
        if (lane == 0) {
            if (P.loss) P.loss[row] = loss;
            if (P.stats) {
                P.stats[4 * row] = f.m;
                P.stats[4 * row + 1] = f.logs;
                P.stats[4 * row + 2] = rest.m;
                P.stats[4 * row + 3] = rest.logs;
            }
        }
    }
    if (STEP) {
        bar_sync(kRowHelped);
        if (last >= 0) store_listed(last);
        if (C > 1) {
            cluster_arrive_relaxed();
            cluster_wait();
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 3) distill_grad_kernel(const __grid_constant__ ScoreParams P) {
    using S = Score<DT>;
    __shared__ Teacher teachers[kScoreWarps];
    const int lane = threadIdx.x & 31;
    const uint32_t nsb = P.sb0[P.W];
    const uint64_t units = P.rows * (uint64_t)P.parts;
    const int regs = (P.K + 31) / 32;
    Teacher& t = teachers[threadIdx.x >> 5];
    pdl_enter();
    for (uint64_t unit = (uint64_t)blockIdx.x * kScoreWarps + (threadIdx.x >> 5); unit < units;
         unit += (uint64_t)gridDim.x * kScoreWarps) {
        const uint64_t row = unit / (uint32_t)P.parts;
        const uint32_t part = (uint32_t)(unit - row * (uint32_t)P.parts);
        const uint32_t sb_lo = part * P.part_sb, sb_hi = min(nsb, sb_lo + P.part_sb);
        RawList raw;
        load_raw(raw, P, row, regs, lane);
        List L{};
        uint32_t bits = 0;
        __syncwarp();
        place_list<DT>(L, t.v, raw, P, row, regs, lane, [&](int i, const char*, int, uint32_t) {
            const uint32_t sb = L.place[i] >> S::kLogSb;
            if (sb >= sb_lo && sb < sb_hi) bits |= 1u << (sb - sb_lo);
        });
        const uint32_t entries = __reduce_or_sync(~0u, bits);      // superblocks of the unit that hold some
        Coef coef{P.c, 0.0f, 0.0f};
        float m = 0.0f, logs = 0.0f, g = 0.0f;
        if (L.some) {
            teacher_mass(t, P, regs, kTwoToThe32nds, lane);
            m = P.stats_in[4 * row];
            logs = P.stats_in[4 * row + 1];
            const float m_rest = P.stats_in[4 * row + 2], logs_rest = P.stats_in[4 * row + 3];
            g = __fmul_rn(P.scale, P.g_row[row]);
            if (m_rest != neg_inf()) {
                const SavedRef k = saved_reference<DT>(m_rest, P.scale, P.c);
                const float p_rest = expf(__fadd_rn(__fadd_rn(m_rest, -m), __fadd_rn(logs_rest, -logs)));
                coef = {k.f.c, k.f.ref, __fmul_rn(__fmul_rn(g, __fmaf_rn(p_rest, t.rest.y, -t.rest.x)),
                                                  __fmul_rn(expf(__fadd_rn(k.rho, -logs_rest)), undo(k.f)))};
            } else if (m != m || t.rest.y != t.rest.y) {
                coef.coef = quiet_nan();
            }
        }
        const bool zero = !L.some || t.rest.y == 0.0f;      // left out, or the teacher has no mass
        Walk<DT> walk;
        Output<DT> out;
        for (uint32_t sb = sb_lo; sb < sb_hi; ++sb) {
            if (walk.seek(P, row, sb, lane)) out.follow(P, row, walk, lane);
            uint32_t w[16];
            if (zero) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0;
                out.store(w, P, row, walk, sb, lane);
                continue;
            }
            load_superblock<DT>(w, P, row, walk, sb, lane);
            // the listed places' gradients, from their scores before an in-place store takes them
            const bool any = (entries >> (sb - sb_lo)) & 1;
            auto offset = [](uint32_t place) { return (place & ((1u << S::kLogSb) - 1)) * S::kBytes; };
            float listed[kListRegs];
            if (any) {
                each_reg(regs, [&](int i) {
                    listed[i] = 0.0f;
                    if ((L.place[i] >> S::kLogSb) == sb) {
                        const float x = S::load_one(walk.address(sb) - lane * 16 + offset(L.place[i]));
                        const float p = exp_near(__fadd_rn(__fmaf_rn(x, P.scale, -m), -logs));
                        if (__fmul_rn(x, P.scale) != neg_inf() || m != m || t.rest.y != t.rest.y) listed[i] = __fmul_rn(g, __fmaf_rn(p, t.rest.y, -t.q[lane + 32 * i]));
                    }
                });
                __syncwarp();
            }
            rest_gradient<DT>(w, coef);
            out.store(w, P, row, walk, sb, lane);
            if (any) {
                __syncwarp();
                each_reg(regs, [&](int i) {
                    if ((L.place[i] >> S::kLogSb) == sb)
                        S::store_one(out.in_superblock(P, row, walk, sb, offset(L.place[i]), lane), listed[i]);
                });
            }
        }
    }
}

}  // namespace

ScoreKernel distill_forward(int dtype, bool step) {
    if (dtype == MR_BF16) return step ? distill_kernel<MR_BF16, true> : distill_kernel<MR_BF16, false>;
    return step ? distill_kernel<MR_FP32, true> : distill_kernel<MR_FP32, false>;
}

cudaError_t launch_distill_grad(const ScoreParams& P, int dtype, dim3 grid, cudaStream_t s) {
    return dtype == MR_BF16 ? launch_kernel(distill_grad_kernel<MR_BF16>, grid, 0, s, 0, P)
                            : launch_kernel(distill_grad_kernel<MR_FP32>, grid, 0, s, 0, P);
}

}  // namespace mr
