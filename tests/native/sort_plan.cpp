// The plan of the embedding gradient's sort for any device, as C functions.
#include "sort_plan.h"

extern "C" void sort_plan(size_t rows, size_t vocab, size_t hidden, size_t g_bytes, size_t table_bytes, int accumulate, int sms,
                          int most_cluster, int* out) {
    const mr::SortPlan p = mr::plan_sort(rows, vocab, hidden, g_bytes, table_bytes, accumulate != 0, sms, most_cluster);
    out[0] = p.cluster;
    out[1] = p.items;
    out[2] = p.helpers;
    out[3] = (int)p.ahead;
    out[4] = (int)p.cleared;
}
