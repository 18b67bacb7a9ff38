/* The microscaled entry points used from plain C: integer rows small enough
 * that every format holds them exactly go through quantisation and its
 * inverse unchanged, their product equals the integer product, and the norm's
 * in-place sum is exact; guard rows stay as they were; the argument errors are
 * returned.  Prints "ok" and exits 0 on success.  Test infrastructure: built
 * and run by tests/test_mx_from_c_gpu.py. */
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "attn_res.h"

#define M 5
#define N 37
#define K 96
#define XROW (K + 8)       /* bf16 row stride */
#define OROW 48            /* result row stride */
#define GUARD 0x7FA1u

#define CK(x)                                                         \
  do {                                                                \
    cudaError_t e_ = (x);                                             \
    if (e_ != cudaSuccess) {                                          \
      fprintf(stderr, "%s: %s\n", #x, cudaGetErrorString(e_));        \
      return 1;                                                       \
    }                                                                 \
  } while (0)
#define OK(x)                                                         \
  do {                                                                \
    attn_res_status_t s_ = (x);                                       \
    if (s_ != ATTN_RES_OK) {                                          \
      fprintf(stderr, "%s: %s\n", #x, attn_res_status_string(s_));    \
      return 1;                                                       \
    }                                                                 \
  } while (0)

static uint16_t bf16(float f) {
  uint32_t u;
  memcpy(&u, &f, 4);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}
static float value(uint16_t b) {
  uint32_t u = (uint32_t)b << 16;
  float f;
  memcpy(&f, &u, 4);
  return f;
}

/* every group of 16 holds a 6, so a scale of 1 (NVFP4: the tensor's 1 / 1)
 * stands and the integers below are elements */
static int entry(int r, int k, int salt) {
  static const int v[8] = {0, 1, -1, 2, -3, 4, -6, 3};
  return k % 16 == 5 ? 6 : v[(r * 7 + k * 5 + salt) % 8];
}

static int make(int format, int rows, attn_res_mx_t* q) {
  const int bytes = format == ATTN_RES_MXFP8 ? K : K / 2;
  memset(q, 0, sizeof *q);
  q->format = format;
  q->rows = rows;
  q->cols = K;
  q->row_bytes = (bytes + 15) / 16 * 16 + 16;
  CK(cudaMalloc(&q->data, (size_t)rows * q->row_bytes));
  CK(cudaMalloc((void**)&q->scales, (size_t)attn_res_mx_scale_bytes(format, rows, K)));
  return 0;
}

int main(void) {
  uint16_t hx[M * XROW], hw[N * XROW], back[M * XROW], ho[M * OROW];
  for (int r = 0; r < M * XROW; ++r) hx[r] = GUARD;
  for (int r = 0; r < N * XROW; ++r) hw[r] = GUARD;
  for (int r = 0; r < M; ++r)
    for (int k = 0; k < K; ++k) hx[r * XROW + k] = bf16((float)entry(r, k, 0));
  for (int r = 0; r < N; ++r)
    for (int k = 0; k < K; ++k) hw[r * XROW + k] = bf16((float)entry(r, k, 3));
  uint16_t *x, *w, *y, *out, *weight;
  CK(cudaMalloc((void**)&x, sizeof hx));
  CK(cudaMalloc((void**)&w, sizeof hw));
  CK(cudaMalloc((void**)&y, sizeof hx));
  CK(cudaMalloc((void**)&out, sizeof ho));
  CK(cudaMalloc((void**)&weight, K * 2));
  CK(cudaMemcpy(w, hw, sizeof hw, cudaMemcpyHostToDevice));
  for (int format = ATTN_RES_MXFP8; format <= ATTN_RES_NVFP4; ++format) {
    CK(cudaMemcpy(x, hx, sizeof hx, cudaMemcpyHostToDevice));
    attn_res_mx_t a, b;
    if (make(format, M, &a) || make(format, N, &b)) return 1;
    OK(attn_res_mx_quantize(x, XROW, &a, 0, NULL));
    OK(attn_res_mx_quantize(w, XROW, &b, ATTN_RES_FLAG_PDL, NULL));
    CK(cudaMemset(y, 0x5A, sizeof hx));
    OK(attn_res_mx_dequantize(&a, y, XROW, 0, NULL));
    CK(cudaMemcpy(back, y, sizeof back, cudaMemcpyDeviceToHost));
    for (int r = 0; r < M; ++r) {
      for (int k = 0; k < K; ++k)
        if (value(back[r * XROW + k]) != (float)entry(r, k, 0)) {
          fprintf(stderr, "format %d: row %d column %d is %g\n", format, r, k, value(back[r * XROW + k]));
          return 1;
        }
      for (int k = K; k < XROW && r < M - 1; ++k)
        if (back[r * XROW + k] != 0x5A5A) return fprintf(stderr, "padding written\n"), 1;
    }
    for (int kernel = 0; kernel <= ATTN_RES_MX_WIDER; ++kernel) {
      CK(cudaMemset(out, 0x5A, sizeof ho));
      OK(attn_res_mx_matmul(&a, &b, out, OROW, ATTN_RES_FLAG_KERNEL(kernel), NULL));
      CK(cudaMemcpy(ho, out, sizeof ho, cudaMemcpyDeviceToHost));
      for (int m = 0; m < M; ++m)
        for (int n = 0; n < OROW; ++n) {
          int sum = 0;
          for (int k = 0; k < K; ++k) sum += n < N ? entry(m, k, 0) * entry(n, k, 3) : 0;
          if (n < N ? ho[m * OROW + n] != bf16((float)sum) : ho[m * OROW + n] != 0x5A5A) {
            fprintf(stderr, "format %d kernel %d: [%d, %d] is %g, wanted %d\n", format, kernel, m, n,
                    value(ho[m * OROW + n]), sum);
            return 1;
          }
        }
    }
    /* prefix + delta in place, with the rows themselves as the addend */
    uint16_t one[K];
    for (int k = 0; k < K; ++k) one[k] = bf16(1.f);
    CK(cudaMemcpy(weight, one, sizeof one, cudaMemcpyHostToDevice));
    CK(cudaMemcpy(y, hx, sizeof hx, cudaMemcpyHostToDevice));
    OK(attn_res_mx_norm(x, XROW, y, XROW, weight, 1e-6f, NULL, 0, &a, 0, NULL));
    CK(cudaMemcpy(back, x, sizeof back, cudaMemcpyDeviceToHost));
    for (int r = 0; r < M; ++r)
      for (int k = 0; k < XROW; ++k) {
        const uint16_t want = k < K ? bf16(2.f * (float)entry(r, k, 0)) : GUARD;
        if (back[r * XROW + k] != want) return fprintf(stderr, "norm: prefix\n"), 1;
      }
    /* refusals leave everything as it is */
    attn_res_mx_t bad = a;
    bad.cols = 40;
    if (attn_res_mx_quantize(x, XROW, &bad, 0, NULL) != ATTN_RES_EINVAL ||
        attn_res_mx_matmul(&a, &bad, out, OROW, 0, NULL) != ATTN_RES_EINVAL ||
        attn_res_mx_matmul(&a, &b, out, 36, 0, NULL) != ATTN_RES_EINVAL ||
        attn_res_mx_matmul(&a, &b, out + 1, OROW, 0, NULL) != ATTN_RES_EALIGN ||
        attn_res_mx_norm(x, XROW, x, XROW, weight, 1e-6f, NULL, 0, &a, 0, NULL) != ATTN_RES_EALIAS ||
        attn_res_mx_dequantize(&a, (attn_res_bf16_t*)a.data, XROW, 0, NULL) != ATTN_RES_EALIAS)
      return fprintf(stderr, "a bad argument was taken\n"), 1;
    CK(cudaFree(a.data));
    CK(cudaFree(a.scales));
    CK(cudaFree(b.data));
    CK(cudaFree(b.scales));
  }
  CK(cudaDeviceSynchronize());
  printf("ok\n");
  return 0;
}
