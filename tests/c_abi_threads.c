/* Two host threads call the attention to the 8-bit cache side by side, one with trees of 5
 * tokens and one with trees of 1000 (fp32, one sequence, a head of 128): their launches
 * take shared memory of different sizes.  Exits 0 when every call succeeds. */
#include <pthread.h>
#include <stdint.h>
#include <stdio.h>

#include <cuda_runtime_api.h>

#include "specverify.h"

enum { kCalls = 20000, kD = 128, kPages = 64, kMost = 1000 };

static void *zeros(size_t bytes) {
  void *p = NULL;
  if (cudaMalloc(&p, bytes) != cudaSuccess || cudaMemset(p, 0, bytes) != cudaSuccess) return NULL;
  return p;
}

static int failures[2];

static void *worker(void *arg) {
  const int me = (int)(intptr_t)arg, T = me ? kMost : 5;
  int32_t parents[kMost], pages[kPages];
  for (int i = 0; i < T - 1; ++i) parents[i] = i - 1;
  for (int i = 0; i < kPages; ++i) pages[i] = i;
  cudaStream_t s;
  if (cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) != cudaSuccess) return (void *)1;
  float *q = zeros((size_t)T * kD * 4), *out = zeros((size_t)T * kD * 4);
  float *k = zeros(kPages * 16 * kD * 4), *v = zeros(kPages * 16 * kD * 4), *ks = zeros(16), *vs = zeros(16);
  int32_t *table = zeros(sizeof pages), *par = zeros(sizeof parents), *codes = zeros(16), *length = zeros(4), *stored = zeros(4);
  void *kc = zeros(4 * 16 * kD), *vc = zeros(4 * 16 * kD);
  if (!q || !out || !k || !v || !ks || !vs || !table || !par || !codes || !length || !stored || !kc || !vc) return (void *)1;
  cudaMemcpy(table, pages, sizeof pages, cudaMemcpyHostToDevice);
  cudaMemcpy(par, parents, (size_t)(T - 1) * 4, cudaMemcpyHostToDevice);
  if (cudaDeviceSynchronize() != cudaSuccess) return (void *)1;
  for (int i = 0; i < kCalls; ++i) {
    const int rc = spec_kv_attention_f32(q, kD, k, v, kPages, 16, table, kPages, length, NULL, par, kc, vc, ks, vs, 4, 16, codes, 4, stored,
                                         SPEC_KV_INT8, 1, T, 1, 1, kD, 0.1f, out, s);
    if (rc != SPEC_OK && failures[me]++ == 0) fprintf(stderr, "thread %d, call %d: %s\n", me, i, spec_status_string(rc));
    if (i % 50 == 0) cudaStreamSynchronize(s);
  }
  return cudaStreamSynchronize(s) == cudaSuccess ? NULL : (void *)1;
}

int main(void) {
  pthread_t t[2];
  int bad = 0;
  if (cudaFree(0) != cudaSuccess) return 2;
  for (intptr_t i = 0; i < 2; ++i)
    if (pthread_create(&t[i], NULL, worker, (void *)i)) return 2;
  for (int i = 0; i < 2; ++i) {
    void *r = NULL;
    pthread_join(t[i], &r);
    bad |= r != NULL;
  }
  uint32_t flags = 1;
  if (bad || spec_get_status(0, &flags) != SPEC_OK || flags) return 2;
  return failures[0] || failures[1] ? 1 : 0;
}
