// sort_plan.h -- how the embedding's gradient sorts its tokens on a device of a
// given size.  Host only, and without CUDA: any device can be asked about.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace mr {

constexpr int kSortThreads = 1024;
constexpr int kMostSortItems = 16;      // tokens a thread of the sort holds
constexpr int kMostSortCluster = 16;

struct SortPlan {
    int cluster, items;         // CTAs that sort, and tokens that a thread of them holds; cluster 0: they hold fewer than there are
    int helpers;                // more clusters, which meanwhile
    uint32_t ahead, cleared;    // ask for the first rows of g from L2, and clear the first rows of the table
};
// sms: the device's; most_cluster: CTAs that a cluster of the sort may have there.
//
// Up to 32768 tokens eight CTAs sort as fast as sixteen, which have to be free in
// one group of SMs (the whole call, rows of 256: 16384 tokens 25.4 and 28.8 us,
// 32768 33.3 and 32.6); beyond they do not (65536 48.6 and 44.0, 131072 87 and 66).
//
// What the other SMs do meanwhile stops at two fixed sizes, whatever the sort
// takes.  Clearing 48 MiB of the table, also rows that are then written: 777
// rows of 1001 into 32003 x 1001 fp32 32.9 us without, 29.7, 26.7 and 27.7
// with 32, 48 and 64 MiB; 128 MiB of g asked for from L2, which holds no more:
// 16384 rows of 4096 bf16 83.3 us without, 81.7 and 80.1 with 64 and 128 MiB.
// A device without SMs beside the sort's has nobody for it: then nothing counts
// as cleared, and the sums' launch clears every row of no token.
inline SortPlan plan_sort(size_t rows, size_t vocab, size_t hidden, size_t g_bytes, size_t table_bytes, bool accumulate, int sms,
                          int most_cluster) {
    SortPlan p{1, 1, 0, 0, 0};
    const int most = std::min(most_cluster, rows > 32768 ? kMostSortCluster : kMostSortCluster / 2);
    while (2 * p.cluster <= std::min(most, sms) && (size_t)kSortThreads * p.cluster < rows) p.cluster *= 2;
    while (p.items < kMostSortItems && (size_t)kSortThreads * p.cluster * p.items < rows) p.items *= 2;
    if ((size_t)kSortThreads * p.cluster * p.items < rows) return {0, 0, 0, 0, 0};
    const int beside = std::max(0, sms / p.cluster - 1);
    if (beside == 0) return p;
    p.ahead = (uint32_t)std::min<size_t>(rows, ((size_t)128 << 20) / (hidden * g_bytes));
    p.cleared = accumulate ? 0 : (uint32_t)std::min<size_t>(vocab, ((size_t)48 << 20) / (hidden * table_bytes)) / 8 * 8;
    p.helpers = p.ahead || p.cleared ? beside : 0;
    return p;
}

}  // namespace mr
