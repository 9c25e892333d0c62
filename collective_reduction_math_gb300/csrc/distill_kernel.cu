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
// A warp keeps the list in registers, entry lane + 32 i, as places in the
// row's superblocks, and asks of each superblock with one vote whether an
// entry lies in it.
#include "score_kernel.cuh"

namespace mr {

namespace {

constexpr int kListRegs = MR_MAX_TEACHER / 32;
constexpr uint32_t kNoPlace = ~0u;     // past every superblock: a row has fewer than 2^32 - 2^10 places

// A warp's copy of a row's list: entry k = lane + 32 i.
struct List {
    uint32_t place[kListRegs];      // in units of scores, counted through the row's superblocks; kNoPlace if absent
    float v[kListRegs];             // the teacher's value; -inf if absent, NaN for a column past the vocabulary
    bool some;                      // any entry at all
};

// The list as it lies in memory.
struct RawList {
    long long id[kListRegs];
    float v[kListRegs];
};
__device__ __forceinline__ void load_raw(RawList& R, const ScoreParams& P, uint64_t row, int lane) {
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) {
        const int k = lane + 32 * i;
        R.id[i] = -1;
        R.v[i] = neg_inf();
        if (k < P.K) {
            R.id[i] = P.t_ids[row * P.K + k];
            R.v[i] = P.t_val[row * P.K + k];
        }
    }
}
template <int DT>
__device__ __forceinline__ void place_list(List& L, const RawList& R, const ScoreParams& P, uint64_t row, int regs) {
    using S = Score<DT>;
    bool some = false;
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) {
        L.place[i] = kNoPlace;
        L.v[i] = neg_inf();
        const long long id = i < regs ? R.id[i] : -1;
        if (id >= 0) {
            some = true;
            L.v[i] = id < (long long)P.vocab ? R.v[i] : quiet_nan();
            if (id < (long long)P.vocab) {
                const int r = shard_of(P, (uint32_t)id);
                const ShardRow sr = shard_row<DT>(P.x[r], P.ld[r], row, 0);
                L.place[i] = (P.sb0[r] << S::kLogSb) + ((uint32_t)id - P.col0[r] + sr.lo);
            }
        }
    }
    L.some = __any_sync(~0u, some);
}

// The score at a place.
template <int DT>
__device__ __forceinline__ float listed_score(const ScoreParams& P, uint64_t row, uint32_t place) {
    using S = Score<DT>;
    int r = 0;
    const uint32_t sb = place >> S::kLogSb;
    while (sb >= P.sb0[r + 1]) ++r;
    const ShardRow sr = shard_row<DT>(P.x[r], P.ld[r], row, 0);
    return S::load_one(sr.base + (uint64_t)(place - (P.sb0[r] << S::kLogSb)) * S::kBytes);
}

// The teacher's side of a row.
struct Teacher {
    float q[kListRegs], logq[kListRegs];
    float q_rest, Q;
};
__device__ __forceinline__ void teacher_mass(Teacher& t, const List& L, const ScoreParams& P) {
    float total = 0.0f;
    if (P.tail) {
#pragma unroll
        for (int i = 0; i < kListRegs; ++i) {
            t.logq[i] = L.v[i];
            t.q[i] = expf(L.v[i]);
            total = __fadd_rn(total, t.q[i]);
        }
        const float rest = __fadd_rn(1.0f, -warp_sum(total));
        t.q_rest = rest < 0.0f ? 0.0f : rest;
        t.Q = rest < 0.0f ? __fadd_rn(1.0f, -rest) : rest == rest ? 1.0f : rest;
    } else {
        float m = neg_inf();
#pragma unroll
        for (int i = 0; i < kListRegs; ++i) {
            t.logq[i] = __fmul_rn(L.v[i], P.teacher_scale);
            m = max_nan(m, t.logq[i]);
        }
        m = warp_max_nan(m);
        const float ref = m == neg_inf() ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < kListRegs; ++i) {
            t.logq[i] = __fadd_rn(t.logq[i], -ref);
            t.q[i] = expf(t.logq[i]);
            total = __fadd_rn(total, t.q[i]);
        }
        total = warp_sum(total);
        const float log_total = m == neg_inf() ? 0.0f : logf(total);
#pragma unroll
        for (int i = 0; i < kListRegs; ++i) {
            t.logq[i] = __fadd_rn(t.logq[i], -log_total);
            t.q[i] = m == neg_inf() ? 0.0f : __fdiv_rn(t.q[i], total);
        }
        t.q_rest = 0.0f;
        t.Q = m == neg_inf() ? 0.0f : m == m ? 1.0f : m;
    }
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

// What the gradient outside the list needs: coef * 2^(c x - ref).
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
    __shared__ LaneStats stats[2];
    __shared__ Stat part[2][kMaxScoreCluster];
    __shared__ uint32_t s_place[2][MR_MAX_TEACHER];
    __shared__ int row_out[2];              // the row is left out
    __shared__ float s_grad[MR_MAX_TEACHER];        // STEP: the listed places' gradients
    __shared__ Coef s_coef;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = P.csize, crank = C > 1 ? (int)cluster_rank() : 0;
    const uint32_t nsb = P.sb0[P.W];
    const uint32_t sb_lo = (uint32_t)((uint64_t)nsb * crank / C), sb_hi = (uint32_t)((uint64_t)nsb * (crank + 1) / C);
    const uint64_t stride = gridDim.x / C;
    uint64_t row = blockIdx.x / C;
    const int regs = (P.K + 31) / 32;
    if (C > 1) cluster_arrive();        // every CTA of the cluster has started: waited for before the first store to a peer
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
            const uint32_t first = first_superblock(sb_lo, warp, 0);
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
        for (uint32_t count = 0; row < P.rows; row += stride, parity ^= 1, ++count) {
            bar_sync(kRowReady + parity);
            const bool out = row_out[parity];
            const uint32_t first = first_superblock(sb_lo, warp, count);
            List L;
#pragma unroll
            for (int i = 0; i < kListRegs; ++i) L.place[i] = i < regs ? s_place[parity][lane + 32 * i] : kNoPlace;
            const uint32_t entries = out ? 0 : rounds_with_entries<DT>(L, first, sb_hi, kScoreWarps);
            const uint32_t rounds = rounds_of(first), cached = STEP ? min(rounds, P.cache_rounds) : 0;
            Running run = start_running(P.c);
            if constexpr (!STEP) {
                if (out) {
                    ahead_runs = feed.template drop<false>(w, ahead_runs, P, count, warp, lane);
                } else {
                    ahead_runs = feed.template each<false>(w, ahead_runs, P, first, warp, lane, [&](uint32_t (&x)[16], uint32_t sb, uint32_t) {
                        if ((entries >> (((sb - first) / kScoreWarps) & 31)) & 1) mask_listed<DT>(x, L, sb, bounce[warp], lane);
                        accumulate<DT, false>(run, x, S::template max_words<16>(x), P.c);
                    });
                }
            } else {
                copies_wait();          // this row's copies are there
                if (!out) {
                    for (uint32_t i = 0; i < cached; ++i) {
                        if ((entries >> (i & 31)) & 1) mask_listed<DT>(block_of(i), L, first + i * kScoreWarps);
                        read_block(w, block_of(i), lane);
                        accumulate<DT, false>(run, w, S::template max_words<16>(w), P.c);
                    }
                    walk = Walk<DT>{};
                    for (uint32_t i = cached; i < rounds; ++i) {        // a row longer than the cache
                        const uint32_t sb = first + i * kScoreWarps;
                        walk.seek(P, row, sb, lane);
                        load_superblock<DT>(w, P, row, walk, sb, lane);
                        if ((entries >> (i & 31)) & 1) mask_listed_in_registers<DT>(w, L, sb, lane);
                        accumulate<DT, false>(run, w, S::template max_words<16>(w), P.c);
                    }
                }
            }
            if (!out) stats[parity].template put<false>(run.a);
            bar_arrive(kRowDone + parity);
            if (C > 1) {
                if (!waited) cluster_wait();
                cluster_arrive();
                waited = false;     // for this row's phase: before the next one, or the end
            }
            if constexpr (STEP) {
                Coef coef{P.c, 0.0f, 0.0f};
                bar_sync(kRowStep);
                if (!out) coef = s_coef;
                Walk<DT> ahead;
                walk = Walk<DT>{};
                Output<DT> to;
                // the next row's copies go into the blocks as they empty
                const uint64_t next_row = row + stride;
                const uint32_t next_first = first_superblock(sb_lo, warp, count + 1);
                const uint32_t next_cached = next_row < P.rows ? min(rounds_of(next_first), P.cache_rounds) : 0;
                for (uint32_t i = 0; i < max(rounds, next_cached); ++i) {
                    const uint32_t sb = first + i * kScoreWarps;
                    if (i < rounds) {
                        if (walk.seek(P, row, sb, lane)) to.follow(P, row, walk, lane);
                        if (out) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = 0;
                        } else {
                            if (i < cached) read_block(w, block_of(i), lane);
                            else load_superblock<DT>(w, P, row, walk, sb, lane);
                            rest_gradient<DT>(w, coef);
                        }
                    }
                    if (i < next_cached) {
                        const uint32_t next_sb = next_first + i * kScoreWarps;
                        ahead.seek(P, next_row, next_sb, lane);
                        begin_copy<DT>(block_of(i), P, next_row, ahead, next_sb, lane);
                    }
                    if (i < rounds) {
                        to.store(w, P, row, walk, sb, lane);
                        if ((entries >> (i & 31)) & 1) {        // after the vector stores of every lane
                            __syncwarp();
#pragma unroll
                            for (int e = 0; e < kListRegs; ++e)
                                if ((L.place[e] >> S::kLogSb) == sb)
                                    S::store_one(Output<DT>::element(P, row, walk.r, L.place[e] - (P.sb0[walk.r] << S::kLogSb)), s_grad[lane + 32 * e]);
                        }
                    }
                }
                copies_commit();
            }
        }
        if (!waited) cluster_wait();
        return;
    }

    // ================= the row warp =================
    const bool joins = STEP || crank == 0;
    RawList raw;        // the list after the one in `cur` / `next`
    List cur, next;
    float x[kListRegs], x_next[kListRegs];
    // Sets a row up: places for the stream, then the listed scores.
    auto set_up = [&](uint64_t r, int par) {
        place_list<DT>(next, raw, P, r, regs);
#pragma unroll
        for (int i = 0; i < kListRegs; ++i)
            if (i < regs) s_place[par][lane + 32 * i] = next.place[i];
        if (lane == 0) row_out[par] = !next.some;
        bar_arrive(kRowReady + par);
        if (r + stride < P.rows) load_raw(raw, P, r + stride, lane);
        if (joins) {
#pragma unroll
            for (int i = 0; i < kListRegs; ++i) {
                x_next[i] = neg_inf();
                if (next.place[i] != kNoPlace) x_next[i] = listed_score<DT>(P, r, next.place[i]);
            }
        }
    };
    if (row < P.rows) {
        load_raw(raw, P, row, lane);
        set_up(row, 0);
    }
    if (C > 1) cluster_wait();
    int parity = 0;
    for (; row < P.rows; row += stride, parity ^= 1) {
        cur = next;
#pragma unroll
        for (int i = 0; i < kListRegs; ++i) x[i] = x_next[i];
        if (row + stride < P.rows) set_up(row + stride, parity ^ 1);
        const bool out = !cur.some;
        Teacher t;
        Stat l{neg_inf(), 0.0f, 0.0f};      // the listed scores, as one more statistic
        float g = 0.0f;
        if (joins && !out) {
            if (STEP) g = __fmul_rn(P.scale, P.g_row[row]);
            teacher_mass(t, cur, P);
#pragma unroll
            for (int i = 0; i < kListRegs; ++i) l.x = max_nan(l.x, x[i]);
            l.x = warp_max_nan(l.x);
            if (l.x != neg_inf()) {
#pragma unroll
                for (int i = 0; i < kListRegs; ++i) l.s = __fadd_rn(l.s, ex2(__fmul_rn(__fadd_rn(x[i], -l.x), P.c)));
                l.s = warp_sum(l.s);
            }
        }
        bar_sync(kRowDone + parity);
        Stat b{neg_inf(), 0.0f, 0.0f};
        if (!out) b = stats[parity].template join<false>(lane, P.c);
        if (C > 1) {
            if (!out && lane < (STEP ? C : 1)) push_stat<false>(part[parity], crank, lane, b);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            if (joins && !out) b = join_cluster<false>(part[parity], C, lane, P.c);
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
            if (STEP) bar_arrive(kRowStep);
            continue;
        }
        Stat all{max_nan(b.x, l.x), 0.0f, 0.0f};
        {
            Stat r = b;
            rebase<false>(r, all.x, P.c);
            rebase<false>(l, all.x, P.c);
            all.s = __fadd_rn(r.s, l.s);
        }
        const Final f = finish(all, P.scale), rest = finish(b, P.scale);
        const float logp_rest = rest.m == neg_inf() ? neg_inf()
                              : __fmaf_rn(__fadd_rn(b.x, -all.x), P.scale, __fadd_rn(rest.log_s, -f.log_s));
        float logp[kListRegs];
#pragma unroll
        for (int i = 0; i < kListRegs; ++i) {
            logp[i] = log_prob(x[i], all, f, P.scale);
            if (STEP && lane + 32 * i < P.K)
                s_grad[lane + 32 * i] = x[i] == neg_inf() ? 0.0f : __fmul_rn(g, __fmaf_rn(expf(logp[i]), t.Q, -t.q[i]));
        }
        if (STEP) {
            if (lane == 0) {
                const Ref k = reference(b.x, P.c);
                const float mass = __fmul_rn(g, __fmaf_rn(expf(logp_rest), t.Q, -t.q_rest));
                s_coef = {k.c, k.ref, rest.m == neg_inf() ? 0.0f : __fmul_rn(__fdiv_rn(mass, b.s), undo(k))};
            }
            bar_arrive(kRowStep);
        }
        if (crank != 0) continue;
        float loss = 0.0f;
#pragma unroll
        for (int i = 0; i < kListRegs; ++i)
            if (!(t.q[i] == 0.0f)) loss = __fadd_rn(loss, __fmul_rn(t.q[i], __fadd_rn(t.logq[i], -logp[i])));
        loss = warp_sum(loss);
        if (!(t.q_rest == 0.0f)) loss = __fadd_rn(loss, __fmul_rn(t.q_rest, __fadd_rn(logf(t.q_rest), -logp_rest)));
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
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 3) distill_grad_kernel(const __grid_constant__ ScoreParams P) {
    using S = Score<DT>;
    const int lane = threadIdx.x & 31;
    const uint32_t nsb = P.sb0[P.W];
    const uint64_t units = P.rows * (uint64_t)P.parts;
    const int regs = (P.K + 31) / 32;
    pdl_enter();
    for (uint64_t unit = (uint64_t)blockIdx.x * kScoreWarps + (threadIdx.x >> 5); unit < units;
         unit += (uint64_t)gridDim.x * kScoreWarps) {
        const uint64_t row = unit / (uint32_t)P.parts;
        const uint32_t part = (uint32_t)(unit - row * (uint32_t)P.parts);
        const uint32_t sb_lo = part * P.part_sb, sb_hi = min(nsb, sb_lo + P.part_sb);
        RawList raw;
        load_raw(raw, P, row, lane);
        List L;
        place_list<DT>(L, raw, P, row, regs);
        Coef coef{P.c, 0.0f, 0.0f};
        float m = 0.0f, logs = 0.0f, g = 0.0f;
        Teacher t;
        if (L.some) {
            teacher_mass(t, L, P);
            m = P.stats_in[4 * row];
            logs = P.stats_in[4 * row + 1];
            const float m_rest = P.stats_in[4 * row + 2], logs_rest = P.stats_in[4 * row + 3];
            g = __fmul_rn(P.scale, P.g_row[row]);
            if (m_rest != neg_inf()) {
                const SavedRef k = saved_reference<DT>(m_rest, P.scale, P.c);
                const float p_rest = expf(__fadd_rn(__fadd_rn(m_rest, -m), __fadd_rn(logs_rest, -logs)));
                coef = {k.f.c, k.f.ref, __fmul_rn(__fmul_rn(g, __fmaf_rn(p_rest, t.Q, -t.q_rest)),
                                                  __fmul_rn(expf(__fadd_rn(k.rho, -logs_rest)), undo(k.f)))};
            }
        }
        const uint32_t entries = rounds_with_entries<DT>(L, sb_lo, sb_hi, 1);
        Walk<DT> walk;
        Output<DT> out;
        for (uint32_t sb = sb_lo; sb < sb_hi; ++sb) {
            if (walk.seek(P, row, sb, lane)) out.follow(P, row, walk, lane);
            uint32_t w[16];
            if (!L.some) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0;
                out.store(w, P, row, walk, sb, lane);
                continue;
            }
            load_superblock<DT>(w, P, row, walk, sb, lane);
            // the listed places' gradients, from their scores before an in-place store takes them
            const bool any = (entries >> ((sb - sb_lo) & 31)) & 1;
            float listed[kListRegs];
            if (any) {
#pragma unroll
                for (int i = 0; i < kListRegs; ++i) {
                    listed[i] = 0.0f;
                    if ((L.place[i] >> S::kLogSb) == sb) {
                        const float x = S::load_one(walk.shard(P, row).base + (uint64_t)(L.place[i] - (P.sb0[walk.r] << S::kLogSb)) * S::kBytes);
                        const float logp = __fadd_rn(__fmaf_rn(x, P.scale, -m), -logs);
                        if (x != neg_inf()) listed[i] = __fmul_rn(g, __fmaf_rn(expf(logp), t.Q, -t.q[i]));
                    }
                }
                __syncwarp();
            }
            rest_gradient<DT>(w, coef);
            out.store(w, P, row, walk, sb, lane);
            if (any) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kListRegs; ++i)
                    if ((L.place[i] >> S::kLogSb) == sb)
                        S::store_one(Output<DT>::element(P, row, walk.r, L.place[i] - (P.sb0[walk.r] << S::kLogSb)), listed[i]);
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
