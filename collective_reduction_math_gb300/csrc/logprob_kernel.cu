// logprob_kernel.cu -- log probabilities of given tokens with the entropy and
// the top alternatives of each row of scores, and their gradient.
//
// Forward: a cluster of C CTAs takes a row at a time, CTA c the c-th run of
// its superblocks, warp w of it every 8th one.  Every score is read once; the
// threads' running statistics join through shuffles, then through shared
// memory of the cluster's first CTA, which writes the row's results.
//
// The top k come out of the same pass.  The stream keeps one key per run of
// 512 bytes, the run's largest score (order-preserving bits).  Order the runs
// by (largest score, first run first): an element of a run outside the first
// k of them comes after k others, the largest of each of those k runs (equal
// scores: the lower column first, and runs are in column order).  So the k
// best elements lie in the k best runs, whatever the data: these are read
// again, and of the run at place j only its first k - j elements at or above
// the k-th run's largest can count.  The few that remain are ranked by
// counting.
//
// Gradient: with t = y - m, p = e^t / e^logs and a, b of the row alone,
//     dx = scale * (-g_lp p - g_H p (log p + H)) = e^t (a + b t),
// plus scale * g_lp at the given token.  Elementwise, so every warp takes a
// run of a row's superblocks by itself and there is no barrier.
#include "score_kernel.cuh"

namespace mr {

namespace {

// Order-preserving bits of a score: NaN above all, -0 as +0, 0 for "no score".
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return k == 0xffffffffu ? quiet_nan() : __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) { return __reduce_max_sync(~0u, v); }
__device__ __forceinline__ uint32_t warp_min_u32(uint32_t v) { return __reduce_min_sync(~0u, v); }

// (key, column) a before b
__device__ __forceinline__ bool before(uint2 a, uint2 b) { return a.x > b.x || (a.x == b.x && a.y < b.y); }

template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(kThreads, 3) logprob_kernel(const __grid_constant__ ScoreParams P) {
    using S = Score<DT>;
    constexpr int kRuns = kSbRuns;
    extern __shared__ uint32_t top_smem[];
    // every warp's statistics, by row parity; the cluster's first CTA joins them
    __shared__ Stat part[2][kMaxScoreCluster * kScoreWarps];
    __shared__ uint2 peer_top[2][TOP ? kMaxScoreCluster * MR_MAX_TOP : 1];
    __shared__ int peer_count[2][kMaxScoreCluster];
    __shared__ int n_cand, n_sel;
    __shared__ float row_m, row_logs;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = P.csize, crank = C > 1 ? (int)cluster_rank() : 0;
    const uint32_t nsb = P.sb0[P.W];
    const uint32_t sb_lo = (uint32_t)((uint64_t)nsb * crank / C), sb_hi = (uint32_t)((uint64_t)nsb * (crank + 1) / C);
    const int k = P.top_k;
    const uint32_t runs = (sb_hi - sb_lo) * kRuns;
    uint32_t* keys = top_smem;
    uint32_t* sel = keys + (((nsb + C - 1) / C) * kRuns);
    uint2* cand = reinterpret_cast<uint2*>(sel + ((k + 2) & ~1));
    pdl_enter();

    int parity = 0;
    for (uint64_t row = blockIdx.x / C; row < P.rows; row += gridDim.x / C) {
        const long long id = P.ids ? P.ids[row] : 0;
        if (id < 0) {       // left out: nothing of it is read
            if (crank == 0) {
                if (threadIdx.x == 0) {
                    if (P.logprob) P.logprob[row] = 0.0f;
                    if (ENT) P.entropy[row] = 0.0f;
                    if (P.stats) {
                        P.stats[2 * row] = neg_inf();
                        P.stats[2 * row + 1] = 0.0f;
                    }
                }
                if (TOP)
                    for (int i = threadIdx.x; i < k; i += kThreads) {
                        if (P.top_ids) P.top_ids[row * k + i] = -1;
                        if (P.top_logprob) P.top_logprob[row * k + i] = neg_inf();
                    }
            }
            continue;
        }
        float x_id = quiet_nan();
        if (crank == 0 && P.ids && id < (long long)P.vocab) x_id = S::load_one(score_at<DT>(P, row, (uint32_t)id));

        // ---- the stream ----
        Stat a{neg_inf(), 0.0f, 0.0f};
        Walk<DT> walk;
        uint32_t sb = sb_lo + warp;
        uint32_t w[16], nx[16];
        uint32_t p0 = 0;
        ShardRow sr{};
        if (sb < sb_hi) {
            walk.seek(P, row, sb);
            sr = walk.sr;
            p0 = walk.place(sb);
            load_superblock<DT>(w, sr, p0, lane);
        }
        while (sb < sb_hi) {
            const uint32_t next = sb + kScoreWarps;
            const ShardRow now = sr;
            const uint32_t now_p0 = p0;
            if (next < sb_hi) {
                walk.seek(P, row, next);
                sr = walk.sr;
                p0 = walk.place(next);
                load_superblock<DT>(nx, sr, p0, lane);
            }
            accumulate<DT, ENT>(a, w, P.scale);
            if (TOP) {
#pragma unroll
                for (int j = 0; j < kRuns; ++j) {
                    uint32_t key = warp_max_u32(order_key(S::max_words(&w[4 * j], 4)));
                    // a run with no place of the row in it has no score
                    const uint32_t rp = now_p0 + j * 32 * S::VE;
                    if (rp + 32 * S::VE <= now.lo || rp >= now.hi) key = 0;
                    if (lane == 0) keys[(sb - sb_lo) * kRuns + j] = key;
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = nx[i];
            sb = next;
        }
        a = warp_join<ENT>(a);

        // ---- the top k of this CTA's part ----
        if (TOP) {
            if (threadIdx.x == 0) n_cand = 0;
            __syncthreads();
            if (warp == 0) {
                uint32_t best = 0, at = 0;      // this lane's best run left
                auto rescan = [&] {
                    best = 0;
                    for (uint32_t i = lane; i < runs; i += 32)
                        if (keys[i] > best) {
                            best = keys[i];
                            at = i;
                        }
                };
                rescan();
                int n = 0;
                for (; n < k; ++n) {
                    const uint32_t top = warp_max_u32(best);
                    if (top == 0) break;
                    const uint32_t first = warp_min_u32(best == top ? at : ~0u);
                    if (best == top && at == first) {
                        sel[n] = first;
                        keys[first] = 0;
                        rescan();
                    }
                    if (lane == 0 && n == k - 1) sel[k] = top;     // the k-th run's largest
                }
                if (lane == 0) {
                    n_sel = n;
                    if (n < k) sel[k] = 1;      // fewer runs than k: every score counts
                }
            }
            __syncthreads();
            const int n = n_sel;
            const uint32_t floor_key = sel[k];
            for (int j = warp; j < n; j += kScoreWarps) {
                const uint32_t run = sel[j], s = sb_lo + run / kRuns;
                Walk<DT> at;
                at.seek(P, row, s);
                const uint32_t p = at.place(s) + ((run % kRuns) * 32 + lane) * S::VE;
                const uint32_t col = P.col0[at.r] + p - at.sr.lo;
                uint32_t v[4], key[S::VE];
                load_vector<DT>(v, 0, at.sr, p);
#pragma unroll
                for (int e = 0; e < S::VE; ++e) {
                    key[e] = order_key(S::value(S::get(v, 0, e)));
                    if (p + e < at.sr.lo || p + e >= at.sr.hi || key[e] < floor_key) key[e] = 0;
                }
                for (int left = k - j; left > 0; --left) {
                    uint32_t best = key[0];
                    int e_best = 0;
#pragma unroll
                    for (int e = 1; e < S::VE; ++e)
                        if (key[e] > best) {
                            best = key[e];
                            e_best = e;
                        }
                    const uint32_t top = warp_max_u32(best);
                    if (top == 0) break;
                    const uint32_t who = __ballot_sync(~0u, best == top);
                    if (lane == __ffs(who) - 1) {
                        cand[atomicAdd(&n_cand, 1)] = make_uint2(top, col + e_best);
#pragma unroll
                        for (int e = 0; e < S::VE; ++e)
                            if (e == e_best) key[e] = 0;
                    }
                }
            }
        }

        // ---- join ----
        if (lane == 0) {
            if (C == 1) {
                part[parity][warp] = a;
            } else {
                const uint32_t to = peer_address(&part[parity][crank * kScoreWarps + warp], 0);
                peer_store(to, __float_as_uint(a.m));
                peer_store(to + 4, __float_as_uint(a.s));
                peer_store(to + 8, __float_as_uint(a.u));
            }
        }
        if (TOP && C > 1) {
            __syncthreads();
            const int n = n_cand;
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const uint2 mine = cand[i];
                int rank = 0;
                for (int o = 0; o < n; ++o) rank += before(cand[o], mine);
                if (rank < k) {
                    const uint32_t to = peer_address(&peer_top[parity][crank * MR_MAX_TOP + rank], 0);
                    peer_store(to, mine.x);
                    peer_store(to + 4, mine.y);
                }
            }
            if (threadIdx.x == 0) peer_store(peer_address(&peer_count[parity][crank], 0), (uint32_t)min(n, k));
        }
        if (C == 1) __syncthreads();
        else cluster_barrier();
        if (crank == 0) {
            if (warp == 0) {
                Stat b{neg_inf(), 0.0f, 0.0f};
                for (int i = lane; i < C * kScoreWarps; i += 32) {
                    Stat o = part[parity][i];
                    const float M = max_nan(b.m, o.m);
                    rebase<ENT>(b, M);
                    rebase<ENT>(o, M);
                    b.s = __fadd_rn(b.s, o.s);
                    if (ENT) b.u = __fadd_rn(b.u, o.u);
                }
                b = warp_join<ENT>(b);
                if (lane == 0) {
                    float m, logs;
                    finish(b, m, logs);
                    if (P.stats) {
                        P.stats[2 * row] = m;
                        P.stats[2 * row + 1] = logs;
                    }
                    if (P.logprob)
                        P.logprob[row] = x_id == neg_inf() && m == m ? neg_inf()
                                                                     : __fadd_rn(__fmaf_rn(x_id, P.scale, -m), -logs);
                    if (ENT) P.entropy[row] = m == neg_inf() ? 0.0f : __fadd_rn(logs, -__fdiv_rn(b.u, b.s));
                    if (TOP) {
                        row_m = m;
                        row_logs = logs;
                    }
                }
            }
            if (TOP) {
                __syncthreads();
                const uint2* list = C == 1 ? cand : peer_top[parity];
                const int slots = C == 1 ? n_cand : C * MR_MAX_TOP;
                const float m = row_m, logs = row_logs;
                for (int i = threadIdx.x; i < slots; i += kThreads) {
                    if (C > 1 && i % MR_MAX_TOP >= peer_count[parity][i / MR_MAX_TOP]) continue;
                    const uint2 mine = list[i];
                    int rank = 0;
                    if (C == 1) {
                        for (int o = 0; o < slots; ++o) rank += before(list[o], mine);
                    } else {
                        for (int c = 0; c < C; ++c)
                            for (int o = 0; o < peer_count[parity][c]; ++o) rank += before(list[c * MR_MAX_TOP + o], mine);
                    }
                    if (rank < k) {
                        const float x = key_value(mine.x);
                        if (P.top_ids) P.top_ids[row * k + rank] = mine.y;
                        if (P.top_logprob)
                            P.top_logprob[row * k + rank] = x == neg_inf() && m == m ? neg_inf()
                                                          : __fadd_rn(__fmaf_rn(x, P.scale, -m), -logs);
                    }
                }
                __syncthreads();        // before the next row takes the lists
            }
        }
        parity ^= 1;
    }
    if (C > 1) cluster_barrier();       // no CTA leaves while a peer may still write to it
}

template <int DT, bool ENT>
__global__ void __launch_bounds__(kThreads, 3) logprob_grad_kernel(const __grid_constant__ ScoreParams P) {
    using S = Score<DT>;
    const int lane = threadIdx.x & 31;
    const uint32_t nsb = P.sb0[P.W];
    const uint64_t units = P.rows * (uint64_t)P.parts;
    pdl_enter();
    for (uint64_t unit = (uint64_t)blockIdx.x * kScoreWarps + (threadIdx.x >> 5); unit < units;
         unit += (uint64_t)gridDim.x * kScoreWarps) {
        const uint64_t row = unit / (uint32_t)P.parts;
        const uint32_t part = (uint32_t)(unit - row * (uint32_t)P.parts);
        const uint32_t sb_lo = part * P.part_sb, sb_hi = min(nsb, sb_lo + P.part_sb);
        const long long id = P.ids ? P.ids[row] : 0;
        float A = 0.0f, B = 0.0f, m = 0.0f, g_lp = 0.0f;
        uint32_t id_sb = ~0u, id_place = 0;
        int id_r = 0;
        if (id >= 0) {
            m = P.stats_in[2 * row];
            const float logs = P.stats_in[2 * row + 1];
            g_lp = P.g_row ? P.g_row[row] : 0.0f;
            const float g_h = ENT ? P.g_entropy[row] : 0.0f, h = ENT ? P.entropy_in[row] : 0.0f;
            if (m == neg_inf()) {
                m = 0.0f;       // nothing but -inf: every gradient is 0
            } else {
                const float f = __fmul_rn(P.scale, expf(-logs));
                A = -__fmul_rn(f, __fmaf_rn(g_h, __fadd_rn(h, -logs), g_lp));
                B = -__fmul_rn(f, g_h);
            }
            if (P.ids) {
                if (id >= (long long)P.vocab) {
                    A = quiet_nan();
                } else {
                    id_r = shard_of(P, (uint32_t)id);
                    const ShardRow sr = shard_row<DT>(P.x[id_r], P.ld[id_r], row, 0);
                    id_place = (uint32_t)id - P.col0[id_r] + sr.lo;
                    id_sb = P.sb0[id_r] + (id_place >> S::kLogSb);
                }
            }
        }
        Walk<DT> walk;
        ShardRow out{};
        const F2 sc = f2(P.scale, P.scale), off = f2(-m, -m), l2 = f2(kLog2e, kLog2e), a2 = f2(A, A), b2 = f2(B, B);
        for (uint32_t sb = sb_lo; sb < sb_hi; ++sb) {
            if (walk.seek(P, row, sb)) out = shard_row<DT>(P.g[walk.r], P.ldg[walk.r], row, P.col0[walk.r + 1] - P.col0[walk.r]);
            const uint32_t p0 = walk.place(sb);
            uint32_t w[16];
            if (id < 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0;
            } else {
                load_superblock<DT>(w, walk.sr, p0, lane);
            }
            float g_id = 0.0f;
            const bool has_id = sb == id_sb;
            if (has_id) {       // before an in-place store takes the score
                const float x = S::load_one(walk.sr.base + (uint64_t)id_place * S::kBytes);
                const float t = fmaxf(__fmaf_rn(x, P.scale, -m), kFarBelow);
                g_id = x == neg_inf() ? 0.0f
                                      : __fmaf_rn(ex2(__fmul_rn(t, kLog2e)), __fmaf_rn(B, t, A), __fmul_rn(P.scale, g_lp));
                __syncwarp();
            }
            if (id >= 0) {
#pragma unroll
                for (int i = 0; i < S::kPairs; ++i) {
                    float x0, x1, e0, e1;
                    S::pair(w, i, x0, x1);
                    F2 t = fma2(f2(x0, x1), sc, off);
                    unpack(mul2(t, l2), e0, e1);
                    F2 f = a2;
                    if (ENT) {
                        float t0, t1;
                        unpack(t, t0, t1);
                        f = fma2(b2, f2(fmaxf(t0, kFarBelow), fmaxf(t1, kFarBelow)), a2);
                    }
                    unpack(mul2(f2(ex2(e0), ex2(e1)), f), x0, x1);
                    S::set_pair(w, i, x0, x1);
                }
            }
            store_superblock<DT>(w, walk.sr, out, p0, lane);
            if (has_id) {
                __syncwarp();
                if (lane == 0) S::store_one(out.base + (uint64_t)(id_place - walk.sr.lo + out.lo) * S::kBytes, g_id);
            }
        }
    }
}

template <int DT, bool ENT, bool TOP>
cudaError_t launch(const ScoreParams& P, dim3 grid, size_t smem, cudaStream_t s) {
    auto* kernel = logprob_kernel<DT, ENT, TOP>;
    cudaError_t e = cudaSuccess;
    // 48 KB without the opt-in, static shared memory included (up to 20 KB)
    if (smem > 28 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && P.csize > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, grid, smem, s, P.csize > 1 ? P.csize : 0, P);
}

}  // namespace

cudaError_t launch_logprob(const ScoreParams& P, int dtype, dim3 grid, size_t smem, cudaStream_t s) {
    const bool ent = P.entropy != nullptr, top = P.top_k > 0;
    if (dtype == MR_BF16) {
        if (top) return ent ? launch<MR_BF16, true, true>(P, grid, smem, s) : launch<MR_BF16, false, true>(P, grid, smem, s);
        return ent ? launch<MR_BF16, true, false>(P, grid, smem, s) : launch<MR_BF16, false, false>(P, grid, smem, s);
    }
    if (top) return ent ? launch<MR_FP32, true, true>(P, grid, smem, s) : launch<MR_FP32, false, true>(P, grid, smem, s);
    return ent ? launch<MR_FP32, true, false>(P, grid, smem, s) : launch<MR_FP32, false, false>(P, grid, smem, s);
}

cudaError_t launch_logprob_grad(const ScoreParams& P, int dtype, dim3 grid, cudaStream_t s) {
    if (dtype == MR_BF16)
        return P.g_entropy ? launch_kernel(logprob_grad_kernel<MR_BF16, true>, grid, 0, s, 0, P)
                           : launch_kernel(logprob_grad_kernel<MR_BF16, false>, grid, 0, s, 0, P);
    return P.g_entropy ? launch_kernel(logprob_grad_kernel<MR_FP32, true>, grid, 0, s, 0, P)
                       : launch_kernel(logprob_grad_kernel<MR_FP32, false>, grid, 0, s, 0, P);
}

}  // namespace mr
