/* Calls of iabn_block_norm_forward from several host threads at once: thread
 * k makes `calls` calls with the k-th descriptor, tensors and stream, and
 * counts those that were refused.  Built as a shared library by the tests,
 * which pass the entry point. */
#include <pthread.h>
#include <stddef.h>

#include "iabn_block.h"

typedef iabn_status (*forward_fn)(const iabn_block_desc*, const void*, const void*, void*, void*,
                                  const float*, const float*, const float*, const float*,
                                  const float*, float*, float*, float*, float*, void*);

typedef struct {
    iabn_block_desc desc;
    const void *u, *h;
    void *h_out, *n;
    const float* beta_pre;
    void* stream;
    long refused;
} concurrent_call;

typedef struct {
    forward_fn forward;
    concurrent_call* c;
    long calls;
    pthread_barrier_t* start;
} job;

static void* run(void* p) {
    job* j = p;
    concurrent_call* c = j->c;
    pthread_barrier_wait(j->start);
    for (long i = 0; i < j->calls; ++i)
        if (j->forward(&c->desc, c->u, c->h, c->h_out, c->n, NULL, NULL, NULL, NULL, c->beta_pre,
                       NULL, NULL, NULL, NULL, c->stream) != IABN_OK)
            ++c->refused;
    return NULL;
}

/* Returns 0 if all threads ran. */
int concurrent_forward(forward_fn forward, concurrent_call* calls, int threads, long count) {
    pthread_t id[16];
    job jobs[16];
    pthread_barrier_t start;
    if (threads < 1 || threads > 16) return 1;
    pthread_barrier_init(&start, NULL, (unsigned)threads);
    for (int k = 0; k < threads; ++k) {
        jobs[k] = (job){forward, &calls[k], count, &start};
        if (pthread_create(&id[k], NULL, run, &jobs[k]) != 0) return 2;
    }
    for (int k = 0; k < threads; ++k) pthread_join(id[k], NULL);
    pthread_barrier_destroy(&start);
    return 0;
}
