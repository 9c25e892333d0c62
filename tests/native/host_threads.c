/* Calls of the library from several host threads at once (no interpreter lock
 * between them): each thread repeats one call on a stream of its own and
 * counts the refusals. */
#include <pthread.h>
#include <stddef.h>

#include "mr.h"

enum { TOP_K, STEP, NORM, GATHER };

typedef struct {
    int kind, W, k, last;           /* last: status of the last refused call */
    size_t rows, n;                 /* n: vocabulary, row length or elements */
    const void* const* in;
    void* const* out;
    const void *a, *b, *c;          /* teacher columns, values and weights; NORM: a the weight */
    void *p, *q;                    /* results besides `out` */
    void* stream;
    long calls, refused;
} Job;

static mr_status_t once(const Job* j) {
    switch (j->kind) {
        case TOP_K:
            return mr_logprob(j->in, NULL, j->W, j->rows, j->n, MR_FP32, 1.0f, NULL, j->k, NULL, NULL, NULL, j->p, j->q, j->stream);
        case STEP:
            return mr_distill_topk_step(j->in, NULL, j->W, j->rows, j->n, MR_FP32, 1.0f, j->k, j->a, j->b, MR_DISTILL_RENORM, 1.0f, j->c,
                                        j->p, j->out, NULL, j->stream);
        case NORM:
            return mr_allreduce_rmsnorm(j->in, j->out, j->W, j->rows, j->n, NULL, NULL, j->a, 1e-6f, MR_FP32, MR_RING, j->stream);
        default:
            return mr_all_gather(j->in, j->out, j->W, j->n, MR_FP32, j->stream);
    }
}

static void* work(void* arg) {
    Job* j = arg;
    for (long i = 0; i < j->calls; ++i) {
        const mr_status_t st = once(j);
        if (st != MR_OK) {
            j->refused++;
            j->last = (int)st;
        }
    }
    return NULL;
}

/* 0, or -1 where a thread could not be started. */
int run_together(Job* jobs, int n) {
    pthread_t t[16];
    int started = 0;
    while (started < n && started < 16 && !pthread_create(&t[started], NULL, work, &jobs[started])) ++started;
    for (int i = 0; i < started; ++i) pthread_join(t[i], NULL);
    return started == n ? 0 : -1;
}
