// logprob_kernel.cu -- log probabilities of given tokens with the entropy and
// the top alternatives of each row of scores, and their gradient.
//
// Forward: a cluster of C CTAs takes a row at a time, CTA c the c-th run of
// its superblocks, warp w of it every 8th one.  Every score is read once; the
// threads' running statistics join through shuffles, then through shared
// memory of the cluster's first CTA, whose row warp writes the results.
//
// The top k come out of the same pass.  The stream keeps one key per run of
// 512 bytes, the run's largest score (order-preserving bits).  The k-th
// largest of any of the keys is a bound L that at least k scores reach, so the
// best k are among the scores at or above L: all those above it, and of those
// equal to it the first k (equal scores: the lower column first).  L is taken
// from the largest keys of up to 128 groups of runs, found in registers and
// ranked by counting; runs that reach L (a little over k of them on scores
// without a pattern) are read again, 1/600 of the row a run, and the scores
// that count are ranked by counting.  Scores that crowd in a few runs can
// overflow the lists; then the runs are taken one by one: order them by
// (largest score, first run first), and an element of the run at place j has j
// others before it, so only its first k - j elements can count and
// k (k + 1) / 2 places hold them all.
//
// What bounds it (GB300): 8192 x 131072 bf16 in 337 us, 6.17 TB/s of the copy's
// 6.69; 67 % of the issue slots (8.7 instructions a score with the entropy) and
// memory bind together.  Three CTAs an SM, 72 registers.  Top 64 of 160000
// takes 3.4 TB/s (2048 rows in 188 us): its stream has no registers for a
// superblock ahead, and the row warp's picking and ranking are chains of votes
// and small loads.  One token of 131072 with 20 alternatives takes 10.6 us, 2.8 of them without the
// alternatives: the rest is that chain.
//
// Gradient: with t = y - m, p = e^t / e^logs and a, b of the row alone,
//     dx = scale * (-g_lp p - g_H p (log p + H)) = e^t (a + b t),
// plus scale * g_lp at the given token.  Elementwise, so every warp takes a
// run of a row's superblocks by itself and there is no barrier: 625 us at
// 8192 x 131072 bf16, the copy's rate.
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

// A bound that at least k of a warp's keys reach, and not many more (0 where
// fewer than k of them are not 0), bisected by votes.  A lane gives the largest
// of each of four groups of its keys.
__device__ __forceinline__ uint32_t kth_bound(const uint32_t (&top)[4], int k) {
    auto reach = [&](uint32_t bound) {
        int c = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) c += __popc(__ballot_sync(~0u, top[q] >= bound));
        return c;
    };
    // A bound to start from: with the lanes that have one, the least of their
    // largest keys is reached once by each, the least of their second ones twice.
    const uint32_t a = max(top[0], top[1]), b = max(top[2], top[3]), most = max(a, b);
    const uint32_t second = max(min(a, b), a > b ? min(top[0], top[1]) : min(top[2], top[3]));
    uint32_t lo = 1, hi = warp_max_u32(most);
    if (__popc(__ballot_sync(~0u, most != 0)) >= k) lo = __reduce_min_sync(~0u, most ? most : ~0u);
    else if (2 * __popc(__ballot_sync(~0u, second != 0)) >= k) lo = __reduce_min_sync(~0u, second ? second : ~0u);
    else if (reach(1) < k) return 0;
    // reach(lo) >= k > reach(hi + 1)
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        const int c = reach(mid);
        if (c >= k) {
            lo = mid;
            if (c <= k + k / 8) break;
        } else {
            hi = mid - 1;
        }
    }
    return lo;
}

// The best k of a CTA's runs, in order, into sel (one warp); returns how many
// there are, and in `floor_key` the last one's key (1 where there are fewer
// than k: then every score counts).  The runs are in groups of 32 q; lane g
// keeps the largest key of group g, so a round looks at one group.
__device__ __forceinline__ int select_runs(uint32_t* keys, uint32_t runs, int k, uint32_t* sel, uint32_t& floor_key, int lane) {
    const uint32_t q = (runs + 1023) / 1024, size = 32 * q;
    uint32_t mine = 0;
    for (uint32_t g = 0; g * size < runs; ++g) {
        uint32_t v = 0;
        for (uint32_t t = 0; t < q; ++t) {
            const uint32_t i = g * size + t * 32 + lane;
            if (i < runs) v = max(v, keys[i]);
        }
        v = warp_max_u32(v);
        if (lane == (int)g) mine = v;
    }
    floor_key = 1;
    int n = 0;
    while (n < k) {
        const uint32_t top = warp_max_u32(mine);
        if (top == 0) break;
        const uint32_t g = __ffs(__ballot_sync(~0u, mine == top)) - 1;
        uint32_t rest = 0;
        bool found = false;
        for (uint32_t t = 0; t < q; ++t) {
            const uint32_t i = g * size + t * 32 + lane;
            uint32_t key = i < runs ? keys[i] : 0;
            if (!found) {
                const uint32_t who = __ballot_sync(~0u, key == top);
                if (who) {
                    found = true;
                    if (lane == __ffs(who) - 1) {
                        sel[n] = i;
                        keys[i] = key = 0;      // this lane alone reads it again
                    }
                }
            }
            rest = max(rest, key);
        }
        rest = warp_max_u32(rest);
        if (lane == (int)g) mine = rest;
        if (++n == k) floor_key = top;
    }
    __syncwarp();
    return n;
}

// Where a run lies: the address of its first place, that place's column (it
// wraps below the row's start) and the places [lo, hi) that are in the row.
template <int DT>
__device__ __forceinline__ uint4 locate_run(const ScoreParams& P, uint64_t row, uint32_t run) {
    using S = Score<DT>;
    Walk<DT> at;
    at.seek(P, row, run / kSbRuns, 0);
    const ShardRow sr = at.shard(P, row);
    const uint32_t place = at.place(P, run / kSbRuns) + (run % kSbRuns) * 32 * S::VE;
    const uint64_t a = reinterpret_cast<uint64_t>(sr.base) + (uint64_t)place * S::kBytes;
    const uint32_t lo = place < sr.lo ? sr.lo - place : 0;
    const uint32_t hi = place < sr.hi ? min(sr.hi - place, 32u * S::VE) : 0;
    return make_uint4((uint32_t)a, (uint32_t)(a >> 32), P.col0[at.r] + place - sr.lo, lo | hi << 16);
}
// A lane's vector of a run; returns which of its places are in the row (-inf elsewhere).
template <int DT, int N>
__device__ __forceinline__ uint32_t load_run(uint32_t (&w)[N], int j, uint4 run, int lane) {
    using S = Score<DT>;
    const uint32_t lo = run.w & 0xffffu, hi = run.w >> 16, first = lane * S::VE;
    const char* a = reinterpret_cast<const char*>((uint64_t)run.y << 32 | run.x) + lane * 16;
    if (first >= lo && first + S::VE <= hi) {
        load16(&w[4 * j], a);
        return (1u << S::VE) - 1;
    }
    uint32_t in_row = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * j + i] = S::kFill;
#pragma unroll
    for (int e = 0; e < S::VE; ++e)
        if (first + e >= lo && first + e < hi) {
            S::put(w, j, e, S::load_bits(a + e * S::kBytes));
            in_row |= 1u << e;
        }
    return in_row;
}

// Vectors that reach the bound wait for a full warp of them in a ring of 64
// for each warp, as (run << 5 | lane).
constexpr int kWaiting = 64;

// Takes batches of the n runs of `at` (in column order; `next` counts what the
// CTA's warps have taken): appends every score above `bound` and, of those
// equal to it, the first k that this warp meets.  Counts past the list's end
// are not stored.  A run has a score or two that reach the bound: its lanes
// only note the vectors that do, and 32 of those are taken apart at a time, a
// lane each; once a warp has its k that equal the bound it passes such vectors
// by (a mask that leaves less than k places makes all the others equal to it).
template <int DT>
__device__ __forceinline__ void collect(const uint4* at, int n, int k, uint32_t bound, int* next, uint32_t* ring, uint2* cand,
                                        int* n_cand, int lane) {
    using S = Score<DT>;
    constexpr int kBatch = 2;       // runs in flight: they were prefetched, and more registers cost more than they hide
    const int cap = score_top_candidates(k);
    int ties = 0, head = 0, tail = 0;
    auto take_apart = [&](int count) {
        __syncwarp();
        uint32_t v[4], in_row = 0, col = 0;
        if (lane < count) {
            const uint32_t t = ring[(head + lane) % kWaiting];
            const uint4 run = at[t >> 5];
            in_row = load_run<DT>(v, 0, run, t & 31);
            col = run.z + (t & 31) * S::VE;
        }
        uint32_t more = 0, same = 0, key[S::VE];
#pragma unroll
        for (int e = 0; e < S::VE; ++e) {
            key[e] = (in_row >> e) & 1 ? order_key(S::value(S::get(v, 0, e))) : 0;
            more |= (uint32_t)(key[e] > bound) << e;
            same |= (uint32_t)(key[e] == bound && key[e] != 0) << e;
        }
        if (__any_sync(~0u, same != 0)) {       // keep the first k - ties of them
            int before = __popc(same);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(~0u, before, o);
                if (lane >= o) before += up;
            }
            const int total = __shfl_sync(~0u, before, 31);
            int keep = k - ties - (before - __popc(same));
#pragma unroll
            for (int e = 0; e < S::VE; ++e)
                if (((same >> e) & 1) && keep-- > 0) more |= 1u << e;
            ties += total;
        }
        if (more) {
            int to = atomicAdd(n_cand, __popc(more));
#pragma unroll
            for (int e = 0; e < S::VE; ++e)
                if ((more >> e) & 1) {
                    if (to < cap) cand[to] = make_uint2(key[e], col + e);
                    ++to;
                }
        }
        head += count;
        __syncwarp();
    };
    while (true) {
        int j0 = 0;
        if (lane == 0) j0 = atomicAdd(next, kBatch);
        j0 = __shfl_sync(~0u, j0, 0);
        if (j0 >= n) break;
        uint32_t v[4 * kBatch], in_row[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            in_row[b] = 0;
            if (j0 + b < n) in_row[b] = load_run<DT>(v, b, at[j0 + b], lane);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (j0 + b >= n) break;
            const uint32_t most = order_key(S::template max_words<4>(&v[4 * b]));
            const bool hit = in_row[b] != 0 && (most > bound || (most == bound && ties < k));
            const uint32_t who = __ballot_sync(~0u, hit);
            if (hit) ring[(tail + __popc(who & ((1u << lane) - 1))) % kWaiting] = (uint32_t)(j0 + b) << 5 | lane;
            tail += __popc(who);
            if (tail - head >= 32) take_apart(32);
        }
    }
    if (tail > head) take_apart(tail - head);
}

// Runs in the order of their largest scores: the best k - j elements of the
// run at place j (one warp).
template <int DT>
__device__ __forceinline__ void collect_in_order(const uint4* at, int n, int k, uint32_t floor_key, uint2* cand, int* n_cand, int lane) {
    using S = Score<DT>;
    int count = 0;
    for (int j = 0; j < n; ++j) {
        uint32_t v[4], key[S::VE];
        const uint32_t in_row = load_run<DT>(v, 0, at[j], lane), col = at[j].z + lane * S::VE;
#pragma unroll
        for (int e = 0; e < S::VE; ++e) {
            key[e] = (in_row >> e) & 1 ? order_key(S::value(S::get(v, 0, e))) : 0;
            if (key[e] < floor_key) key[e] = 0;
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
            if (lane == __ffs(__ballot_sync(~0u, best == top)) - 1) {
                cand[count] = make_uint2(top, col + e_best);
#pragma unroll
                for (int e = 0; e < S::VE; ++e)
                    if (e == e_best) key[e] = 0;
            }
            __syncwarp();
            count++;
            if (j == 0 && left == 1) floor_key = top;       // this run alone holds k: nothing below its k-th counts
        }
    }
    if (lane == 0) *n_cand = count;
    __syncwarp();
}

__device__ __forceinline__ uint64_t in_order(uint2 c) { return (uint64_t)c.x << 32 | ~c.y; }      // the lower column first

// Ranking by counting grows with the square of the list: of one longer than
// kRanked the best stay, at least k, at most kRanked of them (one warp; the
// entries differ).  Returns how many.
constexpr int kRanked = 128;
__device__ __noinline__ int shorten(uint2* list, int n, int k, int lane) {
    uint32_t least = ~0u, most = 0;
    for (int i = lane; i < n; i += 32) {
        least = min(least, list[i].x);
        most = max(most, list[i].x);
    }
    // at least k of the entries reach lo, fewer than k reach hi + 1
    uint64_t lo = (uint64_t)__reduce_min_sync(~0u, least) << 32, hi = (uint64_t)warp_max_u32(most) << 32 | ~0u;
    while (lo < hi) {
        const uint64_t mid = lo + (hi - lo) / 2 + 1;
        int c = 0;
#pragma unroll 4
        for (int i = lane; i < n; i += 32) c += in_order(list[i]) >= mid;
        c = __reduce_add_sync(~0u, c);
        if (c >= k) {
            lo = mid;
            if (c <= kRanked) break;
        } else {
            hi = mid - 1;
        }
    }
    int m = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const uint2 c = i0 + lane < n ? list[i0 + lane] : make_uint2(0, 0);
        const bool stays = i0 + lane < n && in_order(c) >= lo;
        const uint32_t who = __ballot_sync(~0u, stays);
        if (stays) list[m + __popc(who & ((1u << lane) - 1))] = c;      // before what is read next
        m += __popc(who);
    }
    __syncwarp();
    return m;
}

// The best k of a list of (key, column), in order (one warp; kEach entries of
// a lane at a time).
template <int kEach>
__device__ __forceinline__ void rank_list(const uint2* list, int n, int k, uint2* best, int lane) {
    for (int i = lane; i < n; i += 32 * kEach) {
        uint64_t mine[kEach];
        int rank[kEach];
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const uint2 c = i + 32 * q < n ? list[i + 32 * q] : make_uint2(0, 0);
            mine[q] = in_order(c);
            rank[q] = 0;
        }
#pragma unroll 4
        for (int o = 0; o < n; ++o) {
            const uint64_t other = in_order(list[o]);
#pragma unroll
            for (int q = 0; q < kEach; ++q) rank[q] += other > mine[q];
        }
#pragma unroll
        for (int q = 0; q < kEach; ++q)
            if (i + 32 * q < n && rank[q] < k) best[rank[q]] = make_uint2((uint32_t)(mine[q] >> 32), ~(uint32_t)mine[q]);
    }
    __syncwarp();
}

// The top k of a row from its runs' keys, by the row warp of the cluster's
// first CTA while the stream is in the next row: it picks the runs and begins
// to read them again; the stream's warps, when they are through with their
// row, take what is left (2048 rows of 160000 with 64: 188 us, against 207 with
// only those that found runs picked when they came by).
constexpr int kMaxPicked = 192;
struct TopShared {
    uint4 at[kMaxPicked];           // the picked runs
    uint32_t ring[kScoreWarps + 1][kWaiting];
    uint32_t picked[kMaxPicked];
    uint32_t bound;
    int n_picked, n_cand, next;
};
template <int DT>
__device__ __noinline__ void help(int k, TopShared& T, uint2* cand, int warp, int lane) {
    collect<DT>(T.at, T.n_picked, k, T.bound, &T.next, T.ring[warp], cand, &T.n_cand, lane);
}

// Calls of their own: inlined, their registers crowd the stream's.
template <int DT>
__device__ __forceinline__ void locate(const ScoreParams& P, uint64_t row, TopShared& T, int n, int lane) {
    // The row left the L2 when the others streamed through it: all its runs are
    // asked for at once, before they are read in batches.
    for (int i = lane; i < n; i += 32) {
        const uint4 run = locate_run<DT>(P, row, T.picked[i]);
        const uint32_t lo = run.w & 0xffffu, hi = run.w >> 16;
        const char* a = reinterpret_cast<const char*>((uint64_t)run.y << 32 | run.x);
        for (uint32_t e = lo; e < hi; e += 128 / Score<DT>::kBytes)
            asm volatile("prefetch.global.L2 [%0];" :: "l"(a + e * Score<DT>::kBytes));
        T.at[i] = run;
    }
    __syncwarp();
}
// Picks a row's runs for the CTA's warps; false, and none, where they overflow.
template <int DT>
__device__ __noinline__ bool pick_runs(const ScoreParams& P, uint64_t row, const uint32_t* keys, uint32_t runs, TopShared& T, int lane) {
    using S = Score<DT>;
    const int k = P.top_k;
    // Lane l has runs [l n, (l + 1) n): a lane's finds are in column order, and
    // one scan over the lanes places them.
    const uint32_t n = (runs + 127) / 128 * 4, lo = min(runs, lane * n), hi = min(runs, lo + n);
    uint32_t top[4] = {0, 0, 0, 0};
    for (uint32_t i = lo; i < hi; i += 16) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (i + 4 * q < hi) {
                const uint4 v = *reinterpret_cast<const uint4*>(keys + i + 4 * q);
                top[q] = max(top[q], max(max(v.x, v.y), max(v.z, v.w)));
            }
    }
    uint32_t bound = kth_bound(top, k);
    // the runs that reach it: all those above, the first k of those at it
    uint32_t found = 0;         // above in the low half, at it in the high one
    for (uint32_t i = lo; i < hi; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
        found += (v.x > bound) + (v.y > bound) + (v.z > bound) + (v.w > bound);
        if (bound) found += ((v.x == bound) + (v.y == bound) + (v.z == bound) + (v.w == bound)) << 16;
    }
    uint32_t upto = found;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += up;
    }
    const uint32_t all = __shfl_sync(~0u, upto, 31), before = upto - found;
    const int m = (int)(all & 0xffffu) + min((int)(all >> 16), k);
    if (m <= kMaxPicked && found) {
        int to = (int)(before & 0xffffu) + min((int)(before >> 16), k), keep = k - (int)(before >> 16);
        for (uint32_t i = lo; i < hi; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
            const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool tie = key[e] == bound && bound != 0 && keep > 0, take = key[e] > bound || tie;
                if (take) T.picked[to] = i + e;
                to += take;
                keep -= tie;
            }
        }
    }
    __syncwarp();
    const bool fits = m <= kMaxPicked;
    if (fits) locate<DT>(P, row, T, m, lane);
    if (bound == 0 && fits && m > k) {      // places without a score left too few groups: without them
        uint32_t most[4] = {0, 0, 0, 0};
        for (int i = lane; i < m; i += 128) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (i + 32 * q < m) most[q] = max(most[q], keys[T.picked[i + 32 * q]]);
        }
        bound = kth_bound(most, k);
    } else if (bound == 0 && fits) {
        // fewer runs than k: a bound from the lanes' largest scores in them
        uint32_t most[4] = {0, 0, 0, 0};
        for (int j0 = 0; j0 < m; j0 += 4) {
            uint32_t v[16], in_row[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (j0 + b < m) in_row[b] = load_run<DT>(v, b, T.at[j0 + b], lane);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (j0 + b < m && in_row[b]) most[b] = max(most[b], order_key(S::template max_words<4>(&v[4 * b])));
        }
        bound = kth_bound(most, k);
    }
    __syncwarp();
    if (lane == 0) {
        T.n_cand = T.next = 0;
        T.n_picked = fits ? m : 0;
        T.bound = bound;
    }
    __syncwarp();
    return fits;
}
// The candidates are complete: the runs one by one where they overflowed.
template <int DT>
__device__ __noinline__ void mend_candidates(const ScoreParams& P, uint64_t row, uint32_t* keys, uint32_t runs, uint2* cand, TopShared& T,
                                             int lane) {
    uint32_t floor_key;
    const int r = select_runs(keys, runs, P.top_k, T.picked, floor_key, lane);
    locate<DT>(P, row, T, r, lane);
    collect_in_order<DT>(T.at, r, P.top_k, floor_key, cand, &T.n_cand, lane);
}
__device__ __noinline__ void put_top(const ScoreParams& P, uint64_t row, uint2* cand, TopShared& T, const Stat& all, const Final& f,
                                     int lane) {
    const int k = P.top_k;
    uint2* const best = reinterpret_cast<uint2*>(T.ring);       // its readers are through
    static_assert(sizeof(T.ring) >= MR_MAX_TOP * sizeof(uint2), "the best k fit");
    int n = T.n_cand;
    if (n > kRanked) n = shorten(cand, n, k, lane);
    // A list of a warp's size spares the other entries' compares (one token with
    // 20 alternatives 10.6 us against 11.2); longer ones are read once for four
    // (2048 rows with 64: 207 us against 216 one at a time).
    if (n <= 32) rank_list<1>(cand, n, k, best, lane);
    else rank_list<4>(cand, n, k, best, lane);
#pragma unroll 1
    for (int i = lane; i < k; i += 32) {
        const uint2 c = best[i];
        if (P.top_ids) P.top_ids[row * k + i] = c.y;
        if (P.top_logprob) P.top_logprob[row * k + i] = log_prob(key_value(c.x), all, f, P.scale);
    }
    __syncwarp();
}

template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(kScoreThreads, 3) logprob_kernel(const __grid_constant__ ScoreParams P) {
    using S = Score<DT>;
    extern __shared__ __align__(16) uint32_t top_smem[];     // TOP: its fixed part, two rows' keys, the candidates
    __shared__ LaneStats stats[2];
    __shared__ Stat part[2][kMaxScoreCluster];      // the CTAs' statistics, in the cluster's first CTA
    __shared__ int row_out[2];      // the row is left out
    TopShared& top = *reinterpret_cast<TopShared*>(top_smem);
    static_assert(sizeof(TopShared) <= kTopSharedBytes, "score_top_smem counts them");

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int C = P.csize, crank = C > 1 ? (int)cluster_rank() : 0;
    const uint32_t nsb = P.sb0[P.W];
    const uint32_t sb_lo = (uint32_t)((uint64_t)nsb * crank / C), sb_hi = (uint32_t)((uint64_t)nsb * (crank + 1) / C);
    const uint64_t stride = gridDim.x / C;
    uint64_t row = blockIdx.x / C;
    const int k = P.top_k;
    const uint32_t runs = nsb * kSbRuns;
    uint32_t* const keys = top_smem + kTopSharedBytes / 4;
    uint2* const cand = reinterpret_cast<uint2*>(keys + 2 * runs);
    if (C > 1) cluster_arrive();        // every CTA of the cluster has started: waited for before the first store to a peer
    pdl_enter();

    if (warp < kScoreWarps) {
        // ================= the stream =================
        uint32_t w[16];
        Feed<DT> feed;
        uint32_t ahead = feed.template start<TOP>(w, P, sb_lo, sb_hi, row, stride, warp, lane);
        bool waited = C == 1, last_out = true;
        int parity = 0;
        uint32_t count = 0;     // this CTA's rows so far
        const uint32_t keys_at = TOP ? (C > 1 ? peer_address(keys, 0) : (uint32_t)__cvta_generic_to_shared(keys)) : 0;
        for (; row < P.rows; row += stride, parity ^= 1) {
            bar_sync(kRowReady + parity);
            const bool out = row_out[parity];
            if (TOP && !waited) {       // the keys of the row before last have been used
                cluster_wait();
                waited = true;
            }
            Running run = start_running(P.c);
            const uint32_t first = first_superblock(sb_lo, warp, count);
            if (out) {
                ahead = feed.template drop<TOP>(w, ahead, P, count, warp, lane);
            } else {
                ahead = feed.template each<TOP>(w, ahead, P, first, warp, lane, [&](const uint32_t (&x)[16], uint32_t sb, uint32_t with_scores) {
                    if constexpr (TOP) {
                        float top[kSbRuns], mine = quiet_nan();
#pragma unroll
                        for (int j = 0; j < kSbRuns; ++j) {
                            top[j] = S::template max_words<4>(&x[4 * j]);
                            const float most = redux_max_nan(top[j]);
                            if (lane == j) mine = most;
                        }
                        if (lane < kSbRuns)
                            peer_store(keys_at + (parity * runs + sb * kSbRuns + lane) * 4, lane < with_scores ? order_key(mine) : 0);
                        accumulate<DT, ENT>(run, x, max_nan(max_nan(top[0], top[1]), max_nan(top[2], top[3])), P.c);
                    } else {
                        accumulate<DT, ENT>(run, x, S::template max_words<16>(x), P.c);
                    }
                });
            }
            if (!out) stats[parity].template put<ENT>(run.a);
            bar_arrive(kRowDone + parity);
            if (C > 1) {
                if (!waited) cluster_wait();
                if (TOP) cluster_arrive();      // its runs' keys
                else cluster_arrive_relaxed();
                waited = false;         // for this row's phase: before the next one, or the end
            }
            if (TOP && crank == 0) {
                // the row before: its runs have to be read before the row after this one can start
                if (!last_out) {
                    bar_sync(kRowHelp);
                    help<DT>(k, top, cand, warp, lane);
                    bar_arrive(kRowHelped);
                }
                last_out = out;
            }
            ++count;
        }
        if (TOP && !last_out) {
            bar_sync(kRowHelp);
            help<DT>(k, top, cand, warp, lane);
            bar_arrive(kRowHelped);
        }
        if (!waited) cluster_wait();
        return;
    }

    // ================= the row warp =================
    auto id_of = [&](uint64_t r) -> long long { return P.ids && r < P.rows ? P.ids[r] : 0; };
    auto row_ready = [&](uint64_t r, long long id, int par) {
        if (r < P.rows) {
            if (lane == 0) row_out[par] = id < 0;
            bar_arrive(kRowReady + par);
        }
    };
    long long id = id_of(row), id_next = id_of(row + stride);
    row_ready(row, id, 0);
    row_ready(row + stride, id_next, 1);
    if (C > 1) cluster_wait();
    int parity = 0;
    for (; row < P.rows; row += stride, parity ^= 1) {
        const bool out = id < 0;
        const long long id_after = id_of(row + 2 * stride);
        float x_id = quiet_nan();
        if (crank == 0 && P.ids && !out && id < (long long)P.vocab) x_id = S::load_one(score_at<DT>(P, row, (uint32_t)id));
        bar_sync(kRowDone + parity);
        id = id_next;
        id_next = id_after;
        Stat all{neg_inf(), 0.0f, 0.0f};
        if (!out) all = stats[parity].template join<ENT>(lane, P.c);
        if (C > 1) {
            if (lane == 0 && !out) push_stat<ENT>(&part[parity][crank], 0, all);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            if (crank != 0) {
                row_ready(row + 2 * stride, id_after, parity);
                continue;
            }
            if (!out) all = join_parts<ENT>(part[parity], C, lane, P.c);
        }
        Final f{neg_inf(), 0.0f, 0.0f};
        bool fits = true;
        if (TOP && !out) {
            fits = pick_runs<DT>(P, row, keys + parity * runs, runs, top, lane);
            bar_arrive(kRowHelp);
        }
        if (!out) f = finish(all, P.scale);
        if (lane == 0) {
            if (P.stats) {
                P.stats[2 * row] = f.m;
                P.stats[2 * row + 1] = f.logs;
            }
            if (P.logprob) P.logprob[row] = out ? 0.0f : log_prob(x_id, all, f, P.scale);
            if (ENT) P.entropy[row] = f.m == neg_inf() ? 0.0f : __fmaf_rn(-kLn2, __fdiv_rn(all.u, all.s), f.log_s);
        }
        if (TOP && !out) {
            if (fits) help<DT>(k, top, cand, kScoreWarps, lane);
            bar_sync(kRowHelped);
            if (!fits || top.n_cand > score_top_candidates(k)) mend_candidates<DT>(P, row, keys + parity * runs, runs, cand, top, lane);
        }
        row_ready(row + 2 * stride, id_after, parity);
        if (TOP) {
            if (out) {
                for (int i = lane; i < k; i += 32) {
                    if (P.top_ids) P.top_ids[row * k + i] = -1;
                    if (P.top_logprob) P.top_logprob[row * k + i] = neg_inf();
                }
            } else {
                put_top(P, row, cand, top, all, f, lane);
            }
        }
    }
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
        // gradient: 2^(c x - ref) (A + B (c x - ref))
        float A = 0.0f, B = 0.0f, g_lp = 0.0f;
        Ref ref{P.c, 0.0f, 0.0f};
        uint32_t id_sb = ~0u, id_place = 0;
        int id_r = 0;
        if (id >= 0) {
            const float m = P.stats_in[2 * row], logs = P.stats_in[2 * row + 1];
            g_lp = P.g_row ? P.g_row[row] : 0.0f;
            const float g_h = ENT ? P.g_entropy[row] : 0.0f, h = ENT ? P.entropy_in[row] : 0.0f;
            if (m != neg_inf()) {       // else nothing but -inf: every gradient is 0
                const SavedRef k = saved_reference<DT>(m, P.scale, P.c);
                ref = k.f;
                // p = 2^(c x - ref) f; log p = ln 2 (c x - ref) + off
                const float f = __fmul_rn(P.scale, __fmul_rn(expf(__fadd_rn(k.rho, -logs)), undo(ref)));
                const float off = __fmaf_rn(-kLn2, ref.r, __fadd_rn(k.rho, -logs));
                A = -__fmul_rn(f, __fmaf_rn(g_h, __fadd_rn(h, off), g_lp));
                B = -__fmul_rn(f, __fmul_rn(g_h, kLn2));
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
        Output<DT> out;
        const F2 cc = f2(ref.c, ref.c), off = f2(-ref.ref, -ref.ref), a2 = f2(A, A), b2 = f2(B, B);
        for (uint32_t sb = sb_lo; sb < sb_hi; ++sb) {
            if (walk.seek(P, row, sb, lane)) out.follow(P, row, walk, lane);
            uint32_t w[16];
            if (id < 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0;
            } else {
                load_superblock<DT>(w, P, row, walk, sb, lane);
            }
            float g_id = 0.0f;
            const bool has_id = sb == id_sb;
            if (has_id) {       // before an in-place store takes the score
                const float x = S::load_one(score_at<DT>(P, row, (uint32_t)id));
                const float t = fmaxf(__fmaf_rn(x, ref.c, -ref.ref), kFarBelow);
                g_id = x == neg_inf() ? (A == A ? 0.0f : A) : __fmaf_rn(ex2(t), __fmaf_rn(B, t, A), __fmul_rn(P.scale, g_lp));
                __syncwarp();
            }
            if (id >= 0) {
#pragma unroll
                for (int i = 0; i < S::kPairs; ++i) {
                    float x0, x1, t0, t1;
                    S::pair(w, i, x0, x1);
                    unpack(fma2(f2(x0, x1), cc, off), t0, t1);
                    F2 f = a2;
                    if (ENT) f = fma2(b2, f2(fmaxf(t0, kFarBelow), fmaxf(t1, kFarBelow)), a2);
                    unpack(mul2(f2(ex2(t0), ex2(t1)), f), x0, x1);
                    S::set_pair(w, i, x0, x1);
                }
            }
            out.store(w, P, row, walk, sb, lane);
            if (has_id) {
                __syncwarp();
                if (lane == 0) S::store_one(Output<DT>::element(P, row, id_r, id_place), g_id);
            }
        }
    }
}

ScoreKernel variant(int dtype, bool ent, bool top) {
    if (dtype == MR_BF16)
        return top ? (ent ? logprob_kernel<MR_BF16, true, true> : logprob_kernel<MR_BF16, false, true>)
                   : (ent ? logprob_kernel<MR_BF16, true, false> : logprob_kernel<MR_BF16, false, false>);
    return top ? (ent ? logprob_kernel<MR_FP32, true, true> : logprob_kernel<MR_FP32, false, true>)
               : (ent ? logprob_kernel<MR_FP32, true, false> : logprob_kernel<MR_FP32, false, false>);
}

}  // namespace

ScoreKernel logprob_forward(const ScoreParams& P, int dtype) { return variant(dtype, P.entropy != nullptr, P.top_k > 0); }

cudaError_t launch_logprob_grad(const ScoreParams& P, int dtype, dim3 grid, cudaStream_t s) {
    if (dtype == MR_BF16)
        return P.g_entropy ? launch_kernel(logprob_grad_kernel<MR_BF16, true>, grid, 0, s, 0, P)
                           : launch_kernel(logprob_grad_kernel<MR_BF16, false>, grid, 0, s, 0, P);
    return P.g_entropy ? launch_kernel(logprob_grad_kernel<MR_FP32, true>, grid, 0, s, 0, P)
                       : launch_kernel(logprob_grad_kernel<MR_FP32, false>, grid, 0, s, 0, P);
}

}  // namespace mr
