// attn_res_mx_host.cuh -- host side shared by the microscaled entry points.
#pragma once

#include <cuda_runtime.h>

#include "attn_res_checks.cuh"
#include "attn_res_launch.cuh"
#include "attn_res_mx_product.cuh"

namespace attn_res_host {

// Defined in attn_res_mx_product.cu: the launch of a checked product.
struct ProductCall {
  const attn_res_mx_t* a;
  const attn_res_mx_t* w;
  attn_res_bf16_t* out;
  int64_t out_row;
  bool pdl;
  int kernel;  // ATTN_RES_MX_*, 0 automatic
  int split;   // of the narrow form, 0 automatic
  int device;
  unsigned* err;
  cudaStream_t stream;
};
cudaError_t launch_mx_product(const ProductCall& c);
// Whether the overrides can be met.
bool product_overrides_ok(const attn_res_mx_t& a, const attn_res_mx_t& w, int kernel, int split);

}  // namespace attn_res_host
