// attn_res_checks.cuh -- host side shared by the microscaled and 8-bit entry
// points: checks of arguments and the launch of row kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attn_res.h"

namespace attn_res_host {

// Defined in attn_res_api.cu: the current device, if it is one the kernels
// run on, and its status word.
attn_res_status_t current_device(int* device);
cudaError_t device_status_word(int device, unsigned** word);

constexpr int64_t kMaxStride = int64_t(1) << 40;

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A byte range an argument covers.
struct Span {
  uintptr_t lo = 0, hi = 0;
  bool written = false;
};
inline Span span(const void* p, int64_t bytes, bool written) {
  Span s;
  if (p != nullptr) {
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + static_cast<uintptr_t>(bytes);
  }
  s.written = written;
  return s;
}
template <int N>
inline bool written_overlap(const Span (&s)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      if (i != j && s[i].written && s[i].lo < s[j].hi && s[j].lo < s[i].hi) return true;
  return false;
}

inline bool known_flags(uint32_t f) { return (f & ~ATTN_RES_FLAG_PDL) == 0; }
// (rows - 1) * stride below 2^60: extents in bytes stay far from overflow.
inline bool span_ok(int64_t rows, int64_t stride) { return rows <= 1 || stride <= (int64_t(1) << 60) / (rows - 1); }

// bf16 rows; `width` columns are used.
inline attn_res_status_t check_rows(const attn_res_bf16_t* x, int64_t rows, int64_t row, int64_t width) {
  if (!x || row < width || row > kMaxStride || !span_ok(rows, row)) return ATTN_RES_EINVAL;
  if (!aligned(x, 16) || row % 8 != 0) return ATTN_RES_EALIGN;
  return ATTN_RES_OK;
}
inline Span rows_span(const attn_res_bf16_t* x, int64_t rows, int64_t row, int64_t width, bool written) {
  return span(x, ((rows - 1) * row + width) * 2, written);
}

inline attn_res_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_RES_OK;
  (void)cudaGetLastError();
  return ATTN_RES_ECUDA;
}

// A programmatic launch: the kernel's start-up overlaps the end of a preceding
// kernel that lets its dependents start, and it waits for that kernel before
// it touches memory.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  Launch(int64_t grid, int threads, void* stream) {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  Launch(const Launch&) = delete;
};

}  // namespace attn_res_host
