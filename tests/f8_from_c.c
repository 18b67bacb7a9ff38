/* The 8-bit entry points used from plain C: small integers, which e4m3 holds
 * under a scale of 1, go through quantisation (also transposed) and back
 * unchanged, their product equals the integer product, the gated block with a
 * gate of zero weights makes zeros; guard rows stay as they were; argument
 * errors are returned.  Prints "ok" and exits 0 on success.  Test
 * infrastructure: built and run by tests/test_f8_from_c_gpu.py. */
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "attn_res.h"

#define M 5
#define N 37
#define K 200
#define XROW (K + 8) /* bf16 row stride */
#define OROW 40      /* result row stride */

#define CK(x)                                                         \
  do {                                                                \
    cudaError_t e_ = (x);                                             \
    if (e_ != cudaSuccess) {                                          \
      fprintf(stderr, "%s: %s\n", #x, cudaGetErrorString(e_));        \
      return 1;                                                       \
    }                                                                 \
  } while (0)
#define STATUS(x, want)                                                          \
  do {                                                                           \
    attn_res_status_t s_ = (x);                                                  \
    if (s_ != (want)) {                                                          \
      fprintf(stderr, "%s: %s\n", #x, attn_res_status_string(s_));               \
      return 1;                                                                  \
    }                                                                            \
  } while (0)
#define OK(x) STATUS(x, ATTN_RES_OK)
#define EXPECT(c)                                           \
  do {                                                      \
    if (!(c)) {                                             \
      fprintf(stderr, "line %d: %s\n", __LINE__, #c);       \
      return 1;                                             \
    }                                                       \
  } while (0)

static uint16_t bf16(float f) {
  uint32_t u;
  memcpy(&u, &f, 4);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

/* every group holds a 448, so a scale of 1 stands, and the others are elements */
static float entry(int r, int k, int salt) {
  static const float v[8] = {0, 1, -1, 2, -3, 4, -6, 3};
  return k % 64 == 5 ? 448.f : v[(r * 7 + k * 5 + salt) % 8];
}

static int make(int block, int64_t rows, int64_t cols, attn_res_f8_t* q) {
  const int64_t b = (cols + 127) / 128;
  memset(q, 0, sizeof *q);
  q->block = block;
  q->rows = rows;
  q->cols = cols;
  q->row_bytes = (cols + 15) / 16 * 16 + 16;
  q->scales_row = block == ATTN_RES_F8_ROWS ? (rows + 3) / 4 * 4 : b;
  CK(cudaMalloc(&q->data, (size_t)(rows * q->row_bytes)));
  CK(cudaMemset(q->data, 0x5A, (size_t)(rows * q->row_bytes)));
  CK(cudaMalloc((void**)&q->scales,
                (size_t)((block == ATTN_RES_F8_ROWS ? b : (rows + 127) / 128) * q->scales_row * 4)));
  return 0;
}

int main(void) {
  static uint16_t hx[M * XROW], hw[N * XROW], back[M * XROW], ho[M * OROW];
  static uint8_t codes[M * (K + 32)];
  uint16_t *x, *w, *y, *out;
  attn_res_f8_t qx, qxt, qw, zero, h, s[2];
  for (int r = 0; r < M; ++r)
    for (int k = 0; k < XROW; ++k) hx[r * XROW + k] = k < K ? bf16(entry(r, k, 0)) : 0x7FA1u;
  for (int r = 0; r < N; ++r)
    for (int k = 0; k < XROW; ++k) hw[r * XROW + k] = k < K ? bf16(entry(r, k, 3)) : 0x7FA1u;
  CK(cudaMalloc((void**)&x, sizeof hx));
  CK(cudaMalloc((void**)&w, sizeof hw));
  CK(cudaMalloc((void**)&y, sizeof hx));
  CK(cudaMalloc((void**)&out, sizeof ho));
  CK(cudaMemcpy(x, hx, sizeof hx, cudaMemcpyHostToDevice));
  CK(cudaMemcpy(w, hw, sizeof hw, cudaMemcpyHostToDevice));
  CK(cudaMemcpy(y, hx, sizeof hx, cudaMemcpyHostToDevice));
  CK(cudaMemset(out, 0x5A, sizeof ho));
  if (make(ATTN_RES_F8_ROWS, M, K, &qx) || make(ATTN_RES_F8_ROWS, K, M, &qxt) || make(ATTN_RES_F8_SQUARE, N, K, &qw) ||
      make(ATTN_RES_F8_SQUARE, N, K, &zero) || make(ATTN_RES_F8_ROWS, M, N, &h) || make(ATTN_RES_F8_ROWS, M, N, &s[0]) ||
      make(ATTN_RES_F8_ROWS, M, N, &s[1]))
    return 1;

  OK(attn_res_f8_quantize(x, XROW, &qx, &qxt, 0, NULL));
  OK(attn_res_f8_quantize(w, XROW, &qw, NULL, 0, NULL));
  OK(attn_res_f8_dequantize(&qx, y, XROW, ATTN_RES_FLAG_PDL, NULL));
  CK(cudaMemcpy(back, y, sizeof back, cudaMemcpyDeviceToHost));
  EXPECT(memcmp(back, hx, sizeof back) == 0);
  CK(cudaMemcpy(codes, qx.data, (size_t)(M * qx.row_bytes), cudaMemcpyDeviceToHost));
  for (int r = 0; r < M; ++r)
    for (int k = K; k < qx.row_bytes; ++k) EXPECT(codes[r * qx.row_bytes + k] == 0x5A);

  for (int kernel = 0; kernel <= 2; ++kernel) {
    CK(cudaMemset(out, 0x5A, sizeof ho));
    OK(attn_res_f8_matmul(&qx, &qw, NULL, NULL, out, OROW, ATTN_RES_OUT_BF16, ATTN_RES_FLAG_KERNEL(kernel), NULL));
    CK(cudaMemcpy(ho, out, sizeof ho, cudaMemcpyDeviceToHost));
    for (int i = 0; i < M; ++i)
      for (int j = 0; j < OROW; ++j) {
        float sum = 0;
        for (int k = 0; k < K && j < N; ++k) sum += entry(i, k, 0) * entry(j, k, 3); /* exact */
        EXPECT(ho[i * OROW + j] == (j < N ? bf16(sum) : 0x5A5A));
      }
  }

  CK(cudaMemset(w, 0, sizeof hw));
  OK(attn_res_f8_quantize(w, XROW, &zero, NULL, 0, NULL));
  OK(attn_res_f8_gated(&qx, &zero, &qw, ATTN_RES_SILU, &h, NULL, 0, &s[0], &s[1], 0, NULL));
  CK(cudaMemcpy(codes, h.data, (size_t)(M * h.row_bytes), cudaMemcpyDeviceToHost));
  for (int r = 0; r < M; ++r)
    for (int j = 0; j < N; ++j) EXPECT((codes[r * h.row_bytes + j] & 0x7F) == 0);

  STATUS(attn_res_f8_gated_backward(out, OROW, &s[0], &s[1], ATTN_RES_GELU, &h, &s[1], NULL, NULL, NULL, 0, NULL),
         ATTN_RES_EALIAS);
  STATUS(attn_res_f8_matmul(&qx, &qw, &qx, NULL, out, OROW, 0, 0, NULL), ATTN_RES_EINVAL);
  STATUS(attn_res_f8_matmul(&qx, &qw, NULL, NULL, out, OROW + 4, 0, 0, NULL), ATTN_RES_EALIGN);
  STATUS(attn_res_f8_quantize(x, XROW, &qx, &qx, 0, NULL), ATTN_RES_EINVAL);
  CK(cudaDeviceSynchronize());
  unsigned bits = 1;
  OK(attn_res_device_status(&bits, 0));
  EXPECT(bits == 0);
  puts("ok");
  return 0;
}
