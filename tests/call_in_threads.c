/* Calls of one entry point from several host threads at once, each with its own arrays and sizes (test code). */
#include <pthread.h>
#include <stdint.h>

#include "ssd.h"

typedef ssd_status (*norm_fn)(const ssd_norm_dims *, ssd_dtype, ssd_dtype, int, const void *, const void *, const float *,
                              float, const void *, void *, void *, float *, void *, size_t, ssd_stream_t);
typedef ssd_status (*scan_fn)(const ssd_glr_dims *, ssd_dtype, const void *, const void *, const void *, const float *,
                              const float *, void *, float *, ssd_stream_t);

typedef struct {
  void *fn;
  int64_t scan, rows, dim;      /* scan: 0: gated norm gradient, 1: prefill of `rows` tokens */
  void *in, *weight, *out, *vec; /* in: x, y, gates and gradients; out: 2 x [rows, dim]; vec: [dim], the final state */
  void *workspace, *stream;
  int64_t workspace_bytes, calls, failed;
  pthread_t thread;
} job;

static void *work(void *p) {
  job *j = p;
  const ssd_norm_dims n = {j->rows, j->dim, 1, j->dim, j->dim};
  const ssd_glr_dims g = {1, j->rows, j->dim, j->dim, j->dim};
  for (int64_t k = 0; k < j->calls; ++k) {
    ssd_status s =
        j->scan ? ((scan_fn)j->fn)(&g, SSD_F32, j->in, j->in, j->in, j->weight, 0, j->out, j->vec, j->stream)
                : ((norm_fn)j->fn)(&n, SSD_F32, SSD_F32, 1, j->in, j->in, j->weight, 1e-5f, j->in, j->out,
                                   (float *)j->out + j->rows * j->dim, j->vec, j->workspace, j->workspace_bytes, j->stream);
    if (s != SSD_OK) ++j->failed;
  }
  return 0;
}

int call_in_threads(job *jobs, int n) {
  int started = 0;
  for (; started < n; ++started)
    if (pthread_create(&jobs[started].thread, 0, work, &jobs[started])) break;
  for (int i = 0; i < started; ++i) pthread_join(jobs[i].thread, 0);
  return started == n;
}
