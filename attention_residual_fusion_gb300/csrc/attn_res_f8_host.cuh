// attn_res_f8_host.cuh -- host side shared by the 8-bit entry points.
#pragma once

#include <cuda_runtime.h>

#include "attn_res_checks.cuh"

namespace attn_res_host {

// A checked product: matmul (a, w, and a2, w2 or null) or the gated block's (a
// = x, w = gate, w2 = up).  Defined in attn_res_f8_product.cu.
struct F8Call {
  const attn_res_f8_t *a, *w, *a2, *w2;
  bool gated;
  int activation;                  // gated
  const attn_res_f8_t *h, *g, *u;  // gated: results in codes, or null
  void* out;                       // bf16 or fp32 rows; null: h in codes
  int64_t out_row;
  int out_type;
  bool pdl;
  int kernel, split;  // overrides, 0 automatic
  int device;
  unsigned* err;
  cudaStream_t stream;
};
// Whether the overrides can be met.
bool f8_overrides_ok(const F8Call& c);
// Chooses what is automatic of form and split; false where the wide form would
// have more tiles than it counts (results beyond any device's memory).
bool f8_choose_form(F8Call* c);
// Of a call with its form chosen.
cudaError_t launch_f8_product(const F8Call& c);

}  // namespace attn_res_host
