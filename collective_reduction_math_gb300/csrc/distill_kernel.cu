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
    float v[kListRegs];             // the teacher's value; NaN for a column past the vocabulary
    bool some;                      // any entry at all
};

template <int DT>
__device__ __forceinline__ void load_list(List& L, const ScoreParams& P, uint64_t row, int lane) {
    using S = Score<DT>;
    bool some = false;
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) {
        L.place[i] = kNoPlace;
        L.v[i] = neg_inf();
        const int k = lane + 32 * i;
        if (k < P.K) {
            const long long id = P.t_ids[row * P.K + k];
            if (id >= 0) {
                some = true;
                L.v[i] = P.t_val[row * P.K + k];
                if (id >= (long long)P.vocab) {
                    L.v[i] = quiet_nan();
                } else {
                    const int r = shard_of(P, (uint32_t)id);
                    const ShardRow sr = shard_row<DT>(P.x[r], P.ld[r], row, 0);
                    L.place[i] = (P.sb0[r] << S::kLogSb) + ((uint32_t)id - P.col0[r] + sr.lo);
                }
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

// Takes the listed places of superblock sb out of its words.
template <int DT>
__device__ __forceinline__ void mask_listed(uint32_t (&w)[16], const List& L, uint32_t sb, int lane, int regs) {
    using S = Score<DT>;
    uint32_t mine = 0;      // this lane's listed places, bit VE * vector + element
#pragma unroll
    for (int i = 0; i < kListRegs; ++i) {
        if (i >= regs) break;
        uint32_t hit = __ballot_sync(~0u, (L.place[i] >> S::kLogSb) == sb);
        while (hit) {
            const uint32_t p = __shfl_sync(~0u, L.place[i], __ffs(hit) - 1) & ((1u << S::kLogSb) - 1);
            hit &= hit - 1;
            if ((int)((p >> S::kLogVe) & 31) == lane) mine |= 1u << ((p >> (S::kLogVe + 5)) * S::VE + (p & (S::VE - 1)));
        }
    }
    if (mine) {
#pragma unroll
        for (int j = 0; j < kSbVectors; ++j)
#pragma unroll
            for (int e = 0; e < S::VE; ++e)
                if ((mine >> (j * S::VE + e)) & 1) S::put(w, j, e, S::kBytes == 2 ? S::kFill & 0xffffu : S::kFill);
    }
}

// What the gradient of a row needs.
struct Coef {
    float m_rest, c_rest;       // others: c_rest * e^(y - m_rest)
};

// The places of a superblock turned into gradients.
template <int DT>
__device__ __forceinline__ void rest_gradient(uint32_t (&w)[16], const Coef& c, float scale) {
    using S = Score<DT>;
    const F2 sc = f2(scale, scale), off = f2(-c.m_rest, -c.m_rest), l2 = f2(kLog2e, kLog2e), f = f2(c.c_rest, c.c_rest);
#pragma unroll
    for (int i = 0; i < S::kPairs; ++i) {
        float x0, x1, e0, e1;
        S::pair(w, i, x0, x1);
        unpack(mul2(fma2(f2(x0, x1), sc, off), l2), e0, e1);
        unpack(mul2(f2(ex2(e0), ex2(e1)), f), x0, x1);
        S::set_pair(w, i, x0, x1);
    }
}

template <int DT, bool STEP>
__global__ void __launch_bounds__(kThreads, 3) distill_kernel(const __grid_constant__ ScoreParams P) {
    using S = Score<DT>;
    extern __shared__ uint4 cache[];        // STEP: this CTA's part of the row, [round][vector][thread]
    __shared__ Stat part[2][kMaxScoreCluster * kScoreWarps];
    __shared__ float s_grad[MR_MAX_TEACHER];        // STEP: the listed places' gradients
    __shared__ Coef s_coef;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = P.csize, crank = C > 1 ? (int)cluster_rank() : 0;
    const uint32_t nsb = P.sb0[P.W];
    const uint32_t sb_lo = (uint32_t)((uint64_t)nsb * crank / C), sb_hi = (uint32_t)((uint64_t)nsb * (crank + 1) / C);
    const int regs = (P.K + 31) / 32;
    pdl_enter();

    int parity = 0;
    for (uint64_t row = blockIdx.x / C; row < P.rows; row += gridDim.x / C) {
        List L;
        load_list<DT>(L, P, row, lane);
        if (!L.some) {      // left out
            if (crank == 0 && threadIdx.x == 0) {
                if (P.loss) P.loss[row] = 0.0f;
                if (P.stats) {
                    P.stats[4 * row] = P.stats[4 * row + 2] = neg_inf();
                    P.stats[4 * row + 1] = P.stats[4 * row + 3] = 0.0f;
                }
            }
            if (STEP) {
                Walk<DT> walk;
                ShardRow out{};
                uint32_t w[16] = {};
                for (uint32_t sb = sb_lo + warp; sb < sb_hi; sb += kScoreWarps) {
                    if (walk.seek(P, row, sb))
                        out = shard_row<DT>(P.g[walk.r], P.ldg[walk.r], row, P.col0[walk.r + 1] - P.col0[walk.r]);
                    store_superblock<DT>(w, walk.sr, out, walk.place(sb), lane);
                }
            }
            continue;
        }
        const bool lister = warp == 0 && (STEP || crank == 0);      // the warp that joins
        float x[kListRegs];
        if (lister) {
#pragma unroll
            for (int i = 0; i < kListRegs; ++i) {
                x[i] = neg_inf();
                if (L.place[i] != kNoPlace) x[i] = listed_score<DT>(P, row, L.place[i]);
            }
        }

        // ---- the stream over the places outside the list ----
        Stat a{neg_inf(), 0.0f, 0.0f};
        {
            Walk<DT> walk;
            uint32_t w[16], nx[16];
            uint32_t sb = sb_lo + warp, round = 0;
            if (sb < sb_hi) {
                walk.seek(P, row, sb);
                load_superblock<DT>(w, walk.sr, walk.place(sb), lane);
            }
            while (sb < sb_hi) {
                const uint32_t next = sb + kScoreWarps;
                if (next < sb_hi) {
                    walk.seek(P, row, next);
                    load_superblock<DT>(nx, walk.sr, walk.place(next), lane);
                }
                if (STEP && round < P.cache_rounds) {
#pragma unroll
                    for (int j = 0; j < kSbVectors; ++j)
                        cache[(round * kSbVectors + j) * kThreads + threadIdx.x] =
                            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                }
                mask_listed<DT>(w, L, sb, lane, regs);
                accumulate<DT, false>(a, w, P.scale);
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = nx[i];
                sb = next;
                ++round;
            }
        }
        a = warp_join<false>(a);

        // ---- join ----
        if (lane == 0 && C == 1) part[parity][warp] = a;
        if (C > 1 && lane < (STEP ? C : 1)) {
            const uint32_t to = peer_address(&part[parity][crank * kScoreWarps + warp], lane);
            peer_store(to, __float_as_uint(a.m));
            peer_store(to + 4, __float_as_uint(a.s));
        }
        Teacher t;
        if (lister) teacher_mass(t, L, P);
        if (C == 1) __syncthreads();
        else cluster_barrier();
        if (lister) {
            Stat b{neg_inf(), 0.0f, 0.0f};
            for (int i = lane; i < C * kScoreWarps; i += 32) {
                Stat o{part[parity][i].m, part[parity][i].s, 0.0f};
                const float M = max_nan(b.m, o.m);
                rebase<false>(b, M);
                rebase<false>(o, M);
                b.s = __fadd_rn(b.s, o.s);
            }
            b = warp_join<false>(b);
            // the listed scores, as one more statistic
            float y[kListRegs];
            Stat l{neg_inf(), 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kListRegs; ++i) {
                y[i] = __fmul_rn(x[i], P.scale);
                l.m = max_nan(l.m, y[i]);
            }
            l.m = warp_max_nan(l.m);
            if (l.m != neg_inf()) {
#pragma unroll
                for (int i = 0; i < kListRegs; ++i) l.s = __fadd_rn(l.s, expf(__fmaf_rn(x[i], P.scale, -l.m)));
                l.s = warp_sum(l.s);
            }
            Stat all{max_nan(b.m, l.m), 0.0f, 0.0f};
            {
                Stat r = b;
                rebase<false>(r, all.m);
                rebase<false>(l, all.m);
                all.s = __fadd_rn(r.s, l.s);
            }
            float m, logs, m_rest, logs_rest;
            finish(all, m, logs);
            finish(b, m_rest, logs_rest);
            const float logp_rest = m_rest == neg_inf() ? neg_inf() : __fadd_rn(__fadd_rn(m_rest, -m), __fadd_rn(logs_rest, -logs));
            const float p_rest = expf(logp_rest);
            const float g = STEP ? __fmul_rn(P.scale, P.g_row ? P.g_row[row] : 1.0f) : 0.0f;
            float loss = 0.0f;
#pragma unroll
            for (int i = 0; i < kListRegs; ++i) {
                const float logp = x[i] == neg_inf() && m == m ? neg_inf() : __fadd_rn(__fmaf_rn(x[i], P.scale, -m), -logs);
                if (!(t.q[i] == 0.0f)) loss = __fadd_rn(loss, __fmul_rn(t.q[i], __fadd_rn(t.logq[i], -logp)));
                if (STEP && lane + 32 * i < P.K)
                    s_grad[lane + 32 * i] = x[i] == neg_inf() ? 0.0f : __fmul_rn(g, __fmaf_rn(expf(logp), t.Q, -t.q[i]));
            }
            loss = warp_sum(loss);
            if (!(t.q_rest == 0.0f)) loss = __fadd_rn(loss, __fmul_rn(t.q_rest, __fadd_rn(logf(t.q_rest), -logp_rest)));
            if (lane == 0) {
                if (crank == 0) {
                    if (P.loss) P.loss[row] = loss;
                    if (P.stats) {
                        P.stats[4 * row] = m;
                        P.stats[4 * row + 1] = logs;
                        P.stats[4 * row + 2] = m_rest;
                        P.stats[4 * row + 3] = logs_rest;
                    }
                }
                if (STEP) {
                    const bool none = m_rest == neg_inf();
                    s_coef.m_rest = none ? 0.0f : m_rest;
                    s_coef.c_rest = none ? 0.0f : __fdiv_rn(__fmul_rn(g, __fmaf_rn(p_rest, t.Q, -t.q_rest)), b.s);
                }
            }
        }
        if (STEP) {
            __syncthreads();
            const Coef c = s_coef;
            Walk<DT> walk;
            ShardRow out{};
            uint32_t round = 0;
            for (uint32_t sb = sb_lo + warp; sb < sb_hi; sb += kScoreWarps, ++round) {
                if (walk.seek(P, row, sb))
                    out = shard_row<DT>(P.g[walk.r], P.ldg[walk.r], row, P.col0[walk.r + 1] - P.col0[walk.r]);
                const uint32_t p0 = walk.place(sb);
                uint32_t w[16];
                if (round < P.cache_rounds) {
#pragma unroll
                    for (int j = 0; j < kSbVectors; ++j) {
                        const uint4 v = cache[(round * kSbVectors + j) * kThreads + threadIdx.x];
                        w[4 * j] = v.x;
                        w[4 * j + 1] = v.y;
                        w[4 * j + 2] = v.z;
                        w[4 * j + 3] = v.w;
                    }
                } else {
                    load_superblock<DT>(w, walk.sr, p0, lane);
                }
                rest_gradient<DT>(w, c, P.scale);
                store_superblock<DT>(w, walk.sr, out, p0, lane);
#pragma unroll
                for (int i = 0; i < kListRegs; ++i) {
                    if (i >= regs) break;
                    const bool mine = (L.place[i] >> S::kLogSb) == sb;
                    if (__any_sync(~0u, mine)) {        // after the vector stores of every lane
                        __syncwarp();
                        if (mine)
                            S::store_one(out.base + (uint64_t)(L.place[i] - (walk.sb_lo << S::kLogSb) - walk.sr.lo + out.lo) * S::kBytes,
                                         s_grad[lane + 32 * i]);
                    }
                }
            }
            __syncthreads();        // before the next row takes s_grad and s_coef
        }
        parity ^= 1;
    }
    if (C > 1) cluster_barrier();       // no CTA leaves while a peer may still write to it
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
        List L;
        load_list<DT>(L, P, row, lane);
        Coef c{0.0f, 0.0f};
        float m = 0.0f, logs = 0.0f, g = 0.0f;
        Teacher t;
        if (L.some) {
            teacher_mass(t, L, P);
            m = P.stats_in[4 * row];
            logs = P.stats_in[4 * row + 1];
            const float m_rest = P.stats_in[4 * row + 2], logs_rest = P.stats_in[4 * row + 3];
            g = __fmul_rn(P.scale, P.g_row ? P.g_row[row] : 1.0f);
            if (m_rest != neg_inf()) {
                const float p_rest = expf(__fadd_rn(__fadd_rn(m_rest, -m), __fadd_rn(logs_rest, -logs)));
                c.m_rest = m_rest;
                c.c_rest = __fmul_rn(__fmul_rn(g, __fmaf_rn(p_rest, t.Q, -t.q_rest)), expf(-logs_rest));
            }
        }
        Walk<DT> walk;
        ShardRow out{};
        for (uint32_t sb = sb_lo; sb < sb_hi; ++sb) {
            if (walk.seek(P, row, sb)) out = shard_row<DT>(P.g[walk.r], P.ldg[walk.r], row, P.col0[walk.r + 1] - P.col0[walk.r]);
            const uint32_t p0 = walk.place(sb);
            uint32_t w[16];
            if (!L.some) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0;
                store_superblock<DT>(w, walk.sr, out, p0, lane);
                continue;
            }
            load_superblock<DT>(w, walk.sr, p0, lane);
            // the listed places' gradients, from their scores before an in-place store takes them
            float listed[kListRegs];
            bool any = false;
#pragma unroll
            for (int i = 0; i < kListRegs; ++i) {
                if (i >= regs) break;
                const bool mine = (L.place[i] >> S::kLogSb) == sb;
                any |= mine;
                if (mine) {
                    const float x = S::load_one(walk.sr.base + (uint64_t)(L.place[i] - (walk.sb_lo << S::kLogSb)) * S::kBytes);
                    const float logp = __fadd_rn(__fmaf_rn(x, P.scale, -m), -logs);
                    listed[i] = x == neg_inf() ? 0.0f : __fmul_rn(g, __fmaf_rn(expf(logp), t.Q, -t.q[i]));
                }
            }
            any = __any_sync(~0u, any);
            if (any) __syncwarp();
            rest_gradient<DT>(w, c, P.scale);
            store_superblock<DT>(w, walk.sr, out, p0, lane);
            if (any) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kListRegs; ++i) {
                    if (i >= regs) break;
                    if ((L.place[i] >> S::kLogSb) == sb)
                        S::store_one(out.base + (uint64_t)(L.place[i] - (walk.sb_lo << S::kLogSb) - walk.sr.lo + out.lo) * S::kBytes,
                                     listed[i]);
                }
            }
        }
    }
}

template <int DT, bool STEP>
cudaError_t launch(const ScoreParams& P, dim3 grid, size_t smem, cudaStream_t s) {
    auto* kernel = distill_kernel<DT, STEP>;
    cudaError_t e = cudaSuccess;
    // 48 KB without the opt-in, static shared memory included (up to 20 KB)
    if (smem > 28 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && P.csize > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, grid, smem, s, P.csize > 1 ? P.csize : 0, P);
}

}  // namespace

cudaError_t launch_distill(const ScoreParams& P, int dtype, bool step, dim3 grid, size_t smem, cudaStream_t s) {
    if (dtype == MR_BF16) return step ? launch<MR_BF16, true>(P, grid, smem, s) : launch<MR_BF16, false>(P, grid, smem, s);
    return step ? launch<MR_FP32, true>(P, grid, smem, s) : launch<MR_FP32, false>(P, grid, smem, s);
}

cudaError_t launch_distill_grad(const ScoreParams& P, int dtype, dim3 grid, cudaStream_t s) {
    return dtype == MR_BF16 ? launch_kernel(distill_grad_kernel<MR_BF16>, grid, 0, s, 0, P)
                            : launch_kernel(distill_grad_kernel<MR_FP32>, grid, 0, s, 0, P);
}

}  // namespace mr
