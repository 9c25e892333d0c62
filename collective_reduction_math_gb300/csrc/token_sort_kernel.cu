// token_sort_kernel.cu -- the tokens of a batch sorted by their table row, and
// cut into units for the embedding's gradient.
//
// One cluster sorts them all, in its shared memory: a stable radix sort from
// the lowest digit, of as many passes as the vocabulary's bits need at
// kSortDigit bits a pass (2 up to a vocabulary of 2^20 - 1).  In a pass a warp
// ranks its tokens among themselves, round by round (votes on the digit's bits,
// a count a digit and warp); the counts are summed over the CTA's warps, the
// CTAs' totals are exchanged, and each token goes to its place in the CTA that
// has it, over distributed shared memory.  Tokens stay in registers between a
// pass's reads and its writes, so one buffer is enough.
//
// A token without a row (negative, or past the vocabulary) gets the key
// `vocab`, behind all others, and so does what fills the last CTA up.
//
// Then the runs of one row: each position finds its run's start (the last
// start among the lanes, warps and CTAs before it); a unit starts every kUnit
// positions of a run; units are numbered by a scan.
#include <atomic>

#include "elements.cuh"
#include "embedding.h"

namespace mr {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = kSortThreads / 32;
constexpr uint32_t kNone = 0xffffffffu;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t shared_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t remote(uint32_t at, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(cta));
    return r;
}
__device__ __forceinline__ uint32_t load_remote(const uint32_t* p, uint32_t cta) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(shared_at(p), cta)) : "memory");
    return v;
}
__device__ __forceinline__ void store_remote(uint2* p, uint32_t cta, uint2 v) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(remote(shared_at(p), cta)), "r"(v.x), "r"(v.y) : "memory");
}

// Exclusive sum over the CTA's threads (every thread calls it).
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t* sums) {
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t s = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t o = __shfl_up_sync(kAll, s, d);
        if (lane >= d) s += o;
    }
    __syncthreads();        // sums' last readers are done
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    if (warp == 0) {
        uint32_t t = sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t o = __shfl_up_sync(kAll, t, d);
            if (lane >= d) t += o;
        }
        sums[lane] = t;
    }
    __syncthreads();
    return s - v + (warp ? sums[warp - 1] : 0);
}

// While one cluster sorts, the others ask for the first rows of g from L2 and
// clear the first rows of the table (those of tokens are written again).
__device__ __forceinline__ void help(const EmbeddingGradParams& P, int g_bytes, int table_bytes, uint32_t cta, uint32_t ctas) {
    for (uint32_t t = threadIdx.x * ctas + cta; t < P.ahead; t += ctas * kSortThreads) {
        const uint64_t p = (uint64_t)P.g + (uint64_t)t * P.ld_g * g_bytes, from = (p + 15) / 16 * 16, upto = (p + P.hidden * g_bytes) / 16 * 16;
        if (from < upto) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(upto - from)) : "memory");
    }
    for (uint32_t v = threadIdx.x / 32 * ctas + cta; v < P.cleared; v += ctas * kWarps) {
        if (table_bytes == 2) clear_bytes<2>(row_of(P.grad, v, 2), P.hidden * 2, threadIdx.x % 32);
        else clear_bytes<4>(row_of(P.grad, v, 4), P.hidden * 4, threadIdx.x % 32);
    }
}

// x: the key, y: the token
template <int K>
__global__ void __launch_bounds__(kSortThreads, 1) token_sort_kernel(const __grid_constant__ EmbeddingGradParams P, int g_bytes, int table_bytes) {
    constexpr uint32_t E = kSortThreads * K;        // tokens a CTA
    extern __shared__ uint4 dynamic[];
    uint2* item = reinterpret_cast<uint2*>(dynamic);
    const uint32_t bins = 1u << P.digit;
    uint32_t* total = reinterpret_cast<uint32_t*>(item + E);        // of the CTA's tokens, by digit
    uint32_t* place = total + (1 << kSortDigit);                    // where the CTA's first token of a digit goes
    uint16_t* count = reinterpret_cast<uint16_t*>(place + (1 << kSortDigit));      // [warp][digit]
    __shared__ uint32_t sums[32], last_start[kWarps], cta_last, cta_units;
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, cta = cluster_rank(), ctas = cluster_ctas();
    const uint32_t before = (1u << lane) - 1;
    const uint32_t at0 = warp * 32 * K + lane;      // this thread's tokens: at0 + 32 j of the CTA's
    // no early launch of the next kernel: its CTAs, waiting, took the helpers' places
    // (777 rows of 1001 into 32003 x 1001 fp32: 30.9 us against 26.7)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x >= ctas) return help(P, g_bytes, table_bytes, blockIdx.x - ctas, gridDim.x - ctas);

    if (cta == 0 && threadIdx.x == 0) P.counts->longs = 0;
    if (!P.accumulate)
        for (uint32_t i = cta * kSortThreads + threadIdx.x; i < (P.grad.vocab + 31) / 32; i += ctas * kSortThreads) P.present[i] = 0;

    uint2 v[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const uint32_t t = cta * E + at0 + 32 * j;
        const long long id = t < P.rows ? P.ids[t] : -1;
        v[j] = make_uint2((uint64_t)id < P.grad.vocab ? (uint32_t)id : P.grad.vocab, t);
    }
    for (uint32_t pass = 0; pass < P.passes; ++pass) {
        const uint32_t shift = pass * P.digit;
        if (pass) {
#pragma unroll
            for (int j = 0; j < K; ++j) v[j] = item[at0 + 32 * j];
        }
        for (uint32_t i = threadIdx.x; i < kWarps * bins / 8; i += kSortThreads) reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint16_t* mine = count + warp * bins;
        uint32_t rank[K];
        // the lanes with a lane's digit, from a vote on each of its bits (the
        // instruction that matches whole values took longer: 38 against 33 us for
        // 65536 tokens), some rounds at a time
        constexpr int kRounds = K < 4 ? K : 4;
#pragma unroll
        for (int j0 = 0; j0 < K; j0 += kRounds) {
            uint32_t same[kRounds];
#pragma unroll
            for (int j = 0; j < kRounds; ++j) same[j] = kAll;
            for (uint32_t bit = shift; bit < shift + P.digit; ++bit) {
#pragma unroll
                for (int j = 0; j < kRounds; ++j) {
                    const uint32_t ones = __ballot_sync(kAll, v[j0 + j].x >> bit & 1);
                    same[j] &= v[j0 + j].x >> bit & 1 ? ones : ~ones;
                }
            }
#pragma unroll
            for (int j = 0; j < kRounds; ++j) {
                const uint32_t d = v[j0 + j].x >> shift & (bins - 1), seen = mine[d];
                __syncwarp();
                if (!(same[j] & before)) mine[d] = (uint16_t)(seen + __popc(same[j]));
                __syncwarp();
                rank[j0 + j] = seen + __popc(same[j] & before);
            }
        }
        __syncthreads();
        uint32_t n = 0;
        if (threadIdx.x < bins) {
#pragma unroll 8
            for (int w = 0; w < kWarps; ++w) {
                const uint32_t c = count[w * bins + threadIdx.x];
                count[w * bins + threadIdx.x] = (uint16_t)n;
                n += c;
            }
            total[threadIdx.x] = n;
        }
        cluster_sync();     // every CTA has its tokens in registers and its totals in place
        uint32_t earlier = 0, all = 0;
        if (threadIdx.x < bins) {
            for (uint32_t c = 0; c < ctas; ++c) {
                const uint32_t t = c == cta ? n : load_remote(total + threadIdx.x, c);
                if (c < cta) earlier += t;
                all += t;
            }
        }
        const uint32_t first = scan(all, sums);
        if (threadIdx.x < bins) place[threadIdx.x] = first + earlier;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const uint32_t d = v[j].x >> shift & (bins - 1);
            const uint32_t p = place[d] + mine[d] + rank[j];
            store_remote(item + p % E, p / E, v[j]);
        }
        cluster_sync();
    }

    // runs
    uint32_t starts[K];     // the warp's starts of each round, a bit a lane
    uint32_t last = kNone;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const uint32_t at = at0 + 32 * j, p = cta * E + at;
        v[j] = item[at];
        const bool there = v[j].x < P.grad.vocab;
        uint32_t prev = kNone;
        if (there && p > 0) prev = at ? item[at - 1].x : load_remote(&item[E - 1].x, cta - 1);
        starts[j] = __ballot_sync(kAll, there && prev != v[j].x);
        if (starts[j]) last = p - lane + 31 - __clz(starts[j]);
    }
    if (lane == 0) last_start[warp] = last;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t t = kNone;
        for (int w = 0; w < kWarps; ++w) t = last_start[w] != kNone ? last_start[w] : t;
        cta_last = t;
    }
    cluster_sync();
    uint32_t run = kNone;       // the last start before the warp's tokens
    for (uint32_t c = 0; c < cta; ++c) {
        const uint32_t t = load_remote(&cta_last, c);
        if (t != kNone) run = t;
    }
    for (uint32_t w = 0; w < warp; ++w)
        if (last_start[w] != kNone) run = last_start[w];

    // units
    uint32_t unit[K], begin[K], units = 0;      // the warp's units of each round, a bit a lane; this lane's run
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const uint32_t p = cta * E + at0 + 32 * j, upto = starts[j] & (before << 1 | 1);
        begin[j] = upto ? p - lane + 31 - __clz(upto) : run;
        if (starts[j]) run = p - lane + 31 - __clz(starts[j]);
        unit[j] = __ballot_sync(kAll, v[j].x < P.grad.vocab && (p - begin[j]) % kUnit == 0);
        units += __popc(unit[j]);
    }
    uint32_t number = scan(lane == 0 ? units : 0, sums);
    if (threadIdx.x == 0) cta_units = sums[31];
    cluster_sync();
    uint32_t earlier = 0, all = 0;
    for (uint32_t c = 0; c < ctas; ++c) {
        const uint32_t t = load_remote(&cta_units, c);
        if (c < cta) earlier += t;
        all += t;
    }
    number = __shfl_sync(kAll, number, 0) + earlier;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const uint32_t at = at0 + 32 * j, p = cta * E + at;
        const uint32_t row = v[j].x;
        const bool there = row < P.grad.vocab;
        if (there) {
            P.tokens[p] = v[j].y;
            if (unit[j] >> lane & 1) {
                uint32_t flags = 0;
                if (p != begin[j]) flags = kPart;
                else {
                    // a run longer than a unit has the same row kUnit places on
                    const uint32_t on = at + kUnit;
                    const uint32_t later = on < E ? item[on].x : cta + 1 < ctas ? load_remote(&item[on - E].x, cta + 1) : P.grad.vocab;
                    if (later == row) flags = kPart | kFirst;
                    if (!P.accumulate) atomicOr(P.present + row / 32, 1u << row % 32);
                }
                const uint32_t u = number + __popc(unit[j] & before);
                P.units[u] = {p | flags, row};
                if (flags & kFirst) P.longs[atomicAdd(&P.counts->longs, 1u)] = u;
            }
            // the last token of all: where the last unit ends
            const uint32_t next = at + 1 < E ? item[at + 1].x : cta + 1 < ctas ? load_remote(&item[0].x, cta + 1) : P.grad.vocab;
            if (next >= P.grad.vocab) P.units[all] = {p + 1, P.grad.vocab};
        }
        number += __popc(unit[j]);
    }
    if (cta == 0 && threadIdx.x == 0) P.counts->units = all;
    cluster_sync();     // no CTA leaves while another reads its memory
}

template <int K>
constexpr size_t sort_smem() {
    return kSortThreads * K * sizeof(uint2) + 2 * sizeof(uint32_t) * (1 << kSortDigit) + kWarps * sizeof(uint16_t) * (1 << kSortDigit);
}
static_assert(sort_smem<kMostSortItems>() <= kMostDynamicSmem, "the sort's shared memory");

template <int K>
cudaError_t allow(int cluster) {
    const cudaError_t e = allow_dynamic_smem(token_sort_kernel<K>, sort_smem<K>());
    return e == cudaSuccess && cluster > 8 ? cudaFuncSetAttribute(token_sort_kernel<K>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : e;
}

template <int K>
cudaError_t launch(const EmbeddingGradParams& P, int g_bytes, int table_bytes, const SortPlan& plan, cudaStream_t s) {
    const cudaError_t e = allow<K>(plan.cluster);
    if (e != cudaSuccess) return e;
    return launch_kernel_of(kSortThreads, token_sort_kernel<K>, dim3(plan.cluster * (1 + plan.helpers), 1, 1), sort_smem<K>(), s,
                            plan.cluster > 1 ? plan.cluster : 0, P, g_bytes, table_bytes);
}

}  // namespace

// Clusters of more than eight CTAs are not promised by every device: the
// driver is asked (some 10 us) once for each.
int most_sort_cluster() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) dev = 64;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMostSortCluster, 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    cfg.dynamicSmemBytes = sort_smem<kMostSortItems>();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMostSortCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = allow<kMostSortItems>(kMostSortCluster);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, token_sort_kernel<kMostSortItems>, &cfg);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return kMostSortCluster;        // not kept: the launch will say what is wrong
    }
    n = n > 0 ? kMostSortCluster : kMostSortCluster / 2;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_token_sort(const EmbeddingGradParams& P, int g_dtype, int table_dtype, const SortPlan& plan, cudaStream_t s) {
    const int g = g_dtype == MR_BF16 ? 2 : 4, t = table_dtype == MR_BF16 ? 2 : 4;
    switch (plan.items) {
        case 1: return launch<1>(P, g, t, plan, s);
        case 2: return launch<2>(P, g, t, plan, s);
        case 4: return launch<4>(P, g, t, plan, s);
        case 8: return launch<8>(P, g, t, plan, s);
        default: return launch<kMostSortItems>(P, g, t, plan, s);
    }
}

}  // namespace mr
