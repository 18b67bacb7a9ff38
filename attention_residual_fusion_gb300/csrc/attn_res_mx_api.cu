// attn_res_mx_api.cu -- the microscaled entry points of include/attn_res.h:
// argument checks, launch shapes and the launches of the row kernels (the
// product's are in attn_res_mx_product.cu).  Nothing is launched and nothing
// is written unless every check passes.
#include <cmath>

#include "attn_res_checks.cuh"
#include "attn_res_mx_host.cuh"
#include "attn_res_mx_rows.cuh"

namespace {

using namespace attn_res_dev;
using namespace attn_res_host;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;  // tensor-map coordinates and grids are 32-bit
constexpr int64_t kMaxCols = int64_t(1) << 30;
constexpr int64_t kMaxNormCols = 8 * 8 * kMxNormMaxThreads;

bool known_format(int f) { return f == ATTN_RES_MXFP8 || f == ATTN_RES_MXFP4 || f == ATTN_RES_NVFP4; }
int64_t code_bytes(const attn_res_mx_t& q) { return q.cols * mx_bits(q.format) / 8; }
int64_t scale_bytes(const attn_res_mx_t& q) {
  return (q.rows + 127) / 128 * mx_group_tiles(q.format, q.cols) * 512;
}

// What a matrix holds whatever its pointers: format and sizes.
bool scalars_ok(const attn_res_mx_t* q) {
  return q != nullptr && known_format(q->format) && q->rows >= 0 && q->rows <= kMaxRows && q->cols > 0 &&
         q->cols <= kMaxCols && q->cols % 32 == 0 &&
         (q->tensor_scale == nullptr || q->format == ATTN_RES_NVFP4);
}
attn_res_status_t check_matrix(const attn_res_mx_t& q) {
  if (!q.data || !q.scales || q.row_bytes < code_bytes(q) || q.row_bytes >= kMaxStride ||
      !span_ok(q.rows, q.row_bytes))
    return ATTN_RES_EINVAL;
  if (!aligned(q.data, 16) || !aligned(q.scales, 16) || q.row_bytes % 16 != 0 ||
      !aligned(q.tensor_scale, 4))
    return ATTN_RES_EALIGN;
  return ATTN_RES_OK;
}
Span data_span(const attn_res_mx_t& q, bool written) {
  return span(q.data, (q.rows - 1) * q.row_bytes + code_bytes(q), written);
}
Span scales_span(const attn_res_mx_t& q, bool written) { return span(q.scales, scale_bytes(q), written); }
Span tensor_scale_span(const attn_res_mx_t& q) { return span(q.tensor_scale, 4, false); }

MxView view(const attn_res_mx_t& q) {
  MxView v;
  v.data = static_cast<uint8_t*>(q.data);
  v.scales = q.scales;
  v.tensor_scale = q.tensor_scale;
  v.row_bytes = q.row_bytes;
  v.rows = q.rows;
  v.cols = q.cols;
  v.group_tiles = mx_group_tiles(q.format, q.cols);
  return v;
}

// Both directions of the conversion share their checks and their grid.
template <class Kern>
attn_res_status_t run_rows(Kern pick, const attn_res_bf16_t* x, int64_t x_row, const attn_res_mx_t* q,
                           bool to_codes, uint32_t flags, void* stream) {
  if (!scalars_ok(q) || !known_flags(flags)) return ATTN_RES_EINVAL;
  if (q->rows == 0) return ATTN_RES_OK;
  attn_res_status_t st = check_matrix(*q);
  if (st == ATTN_RES_OK) st = check_rows(x, q->rows, x_row, q->cols);
  if (st != ATTN_RES_OK) return st;
  const Span spans[4] = {rows_span(x, q->rows, x_row, q->cols, !to_codes), data_span(*q, to_codes),
                         scales_span(*q, to_codes), tensor_scale_span(*q)};
  if (written_overlap(spans)) return ATTN_RES_EALIAS;
  int device;
  st = current_device(&device);
  if (st != ATTN_RES_OK) return st;
  MxRowsParams p = {};
  p.x = x;
  p.out = const_cast<attn_res_bf16_t*>(x);
  p.x_row = x_row;
  p.q = view(*q);
  const int64_t padded = p.q.group_tiles * 4 * mx_group(q->format);
  const int64_t chunks = (padded + kMxWarpCols - 1) / kMxWarpCols;
  const int64_t jobs = (q->rows + 127) / 128 * 32 * chunks;
  if (jobs > INT32_MAX) return ATTN_RES_EINVAL;  // beyond any device's memory
  p.col_chunks = static_cast<uint32_t>(chunks);
  p.jobs = static_cast<uint32_t>(jobs);
  const int64_t ctas = (jobs + kMxThreads / 32 - 1) / (kMxThreads / 32);
  Launch l(ctas, kMxThreads, stream);
  return launched(cudaLaunchKernelEx(&l.cfg, pick(q->format), p));
}

// The norm's launch for `rows` rows of `nv` vectors (with the groups that fill
// the last scale tile).
struct NormShape {
  void (*kernel)(MxNormParams);
  int threads;
  int64_t ctas;
};
template <int VPT, int MAX_THREADS, int MIN_CTAS, bool WARP_ROWS>
NormShape norm_shape(int format, int64_t nv, int64_t rows) {
  NormShape s;
  const int64_t padded = (rows + 127) / 128 * 128;
  if (WARP_ROWS) {
    s.threads = 32 * kMxWarpRows;
    s.ctas = padded / kMxWarpRows;
  } else {
    s.threads = static_cast<int>(((nv + VPT - 1) / VPT + 31) / 32 * 32);
    s.ctas = rows + (padded - rows + kMxPadRows - 1) / kMxPadRows;
  }
  switch (format) {
    case ATTN_RES_MXFP8: s.kernel = attn_res_mx_norm_kernel<ATTN_RES_MXFP8, VPT, MAX_THREADS, MIN_CTAS, WARP_ROWS>; break;
    case ATTN_RES_MXFP4: s.kernel = attn_res_mx_norm_kernel<ATTN_RES_MXFP4, VPT, MAX_THREADS, MIN_CTAS, WARP_ROWS>; break;
    default: s.kernel = attn_res_mx_norm_kernel<ATTN_RES_NVFP4, VPT, MAX_THREADS, MIN_CTAS, WARP_ROWS>; break;
  }
  return s;
}
// Vectors per thread by the rows' number and width.  With few rows, more
// threads a row.  With many (from kNormManyRows on), up to 1024 columns a warp a
// row -- CTAs of a warp or two would start no faster than an SM takes CTAs --
// and above, four vectors a thread at 64 registers, which keeps the most bytes
// of rows on their way.  Graph replay, mxfp8 with an addend, us (few / many):
//   rows x H         few    many         rows x H         few    many
//   256 x 512        1.65   1.83         8192 x 512       9.25   5.28
//   512 x 4096       3.10   3.29         8192 x 2048     22.9   20.8
//   512 x 7168       5.99   5.35         8192 x 4096     40.1   37.9
//   1024 x 1024      2.64   2.20         8192 x 7168     78.3   63.3
//   1024 x 4096      6.07   5.72         (95 % of the copy rate)
//   1024 x 7168     11.1    9.28
// The many-row shapes in the other formats: 8192 x 7168 59.5 us to mxfp4 and
// 64.9 to nvfp4 (16 bytes of spills a thread).  Above 32768 columns 1024
// threads of 64 registers spill about 150 bytes each: 512 x 65536 to mxfp8
// 55.2 us, for 34.7 us of bytes.
constexpr int64_t kNormManyRows = 1024;
NormShape norm_shape(int format, int64_t nv, int64_t rows) {
  if (rows >= kNormManyRows) {
    if (nv <= 32) return norm_shape<1, 256, 1, true>(format, nv, rows);
    if (nv <= 64) return norm_shape<2, 256, 1, true>(format, nv, rows);
    if (nv <= 128) return norm_shape<4, 256, 1, true>(format, nv, rows);
    if (nv <= 256) return norm_shape<4, 64, 16, false>(format, nv, rows);
    if (nv <= 512) return norm_shape<4, 128, 8, false>(format, nv, rows);
    if (nv <= 1024) return norm_shape<4, 256, 4, false>(format, nv, rows);
  }
  if (nv <= 256) return norm_shape<1, 256, 1, false>(format, nv, rows);
  if (nv <= 1024) return norm_shape<2, 512, 2, false>(format, nv, rows);
  if (nv <= 4096) return norm_shape<8, 512, 1, false>(format, nv, rows);
  return norm_shape<8, 1024, 1, false>(format, nv, rows);
}

}  // namespace

extern "C" {

int64_t attn_res_mx_scale_bytes(int format, int64_t rows, int64_t cols) {
  attn_res_mx_t q = {};
  q.format = format;
  q.rows = rows;
  q.cols = cols;
  return scalars_ok(&q) ? scale_bytes(q) : -1;
}

attn_res_status_t attn_res_mx_quantize(const attn_res_bf16_t* x, int64_t x_row,
                                       const attn_res_mx_t* q, uint32_t flags, void* stream) {
  auto pick = [](int f) -> void (*)(MxRowsParams) {
    return f == ATTN_RES_MXFP8   ? attn_res_mx_quantize_kernel<ATTN_RES_MXFP8>
           : f == ATTN_RES_MXFP4 ? attn_res_mx_quantize_kernel<ATTN_RES_MXFP4>
                                 : attn_res_mx_quantize_kernel<ATTN_RES_NVFP4>;
  };
  return run_rows(pick, x, x_row, q, true, flags, stream);
}

attn_res_status_t attn_res_mx_dequantize(const attn_res_mx_t* q, attn_res_bf16_t* x, int64_t x_row,
                                         uint32_t flags, void* stream) {
  auto pick = [](int f) -> void (*)(MxRowsParams) {
    return f == ATTN_RES_MXFP8   ? attn_res_mx_dequantize_kernel<ATTN_RES_MXFP8>
           : f == ATTN_RES_MXFP4 ? attn_res_mx_dequantize_kernel<ATTN_RES_MXFP4>
                                 : attn_res_mx_dequantize_kernel<ATTN_RES_NVFP4>;
  };
  return run_rows(pick, x, x_row, q, false, flags, stream);
}

attn_res_status_t attn_res_mx_norm(attn_res_bf16_t* prefix, int64_t prefix_row,
                                   const attn_res_bf16_t* delta, int64_t delta_row,
                                   const attn_res_bf16_t* weight, float eps,
                                   attn_res_bf16_t* norm_out, int64_t norm_row,
                                   const attn_res_mx_t* q, uint32_t flags, void* stream) {
  if (!scalars_ok(q) || q->cols > kMaxNormCols || !known_flags(flags) || !std::isfinite(eps) || eps < 0.f)
    return ATTN_RES_EINVAL;
  if (q->rows == 0) return ATTN_RES_OK;
  const int64_t T = q->rows, H = q->cols;
  attn_res_status_t st = check_matrix(*q);
  if (st == ATTN_RES_OK) st = check_rows(prefix, T, prefix_row, H);
  if (st == ATTN_RES_OK && delta) st = check_rows(delta, T, delta_row, H);
  if (st == ATTN_RES_OK) st = check_rows(weight, 1, H, H);
  if (st == ATTN_RES_OK && norm_out) st = check_rows(norm_out, T, norm_row, H);
  if (st != ATTN_RES_OK) return st;
  const Span spans[7] = {rows_span(prefix, T, prefix_row, H, delta != nullptr),
                         rows_span(delta, T, delta_row, H, false),
                         rows_span(weight, 1, H, H, false),
                         rows_span(norm_out, T, norm_row, H, true),
                         data_span(*q, true),
                         scales_span(*q, true),
                         tensor_scale_span(*q)};
  if (written_overlap(spans)) return ATTN_RES_EALIAS;
  int device;
  st = current_device(&device);
  if (st != ATTN_RES_OK) return st;
  MxNormParams p = {};
  p.prefix = prefix;
  p.delta = delta;
  p.weight = weight;
  p.norm_out = norm_out;
  p.prefix_row = prefix_row;
  p.delta_row = delta_row;
  p.norm_row = norm_row;
  p.eps = eps;
  p.width = static_cast<float>(H);
  p.q = view(*q);
  const NormShape shape = norm_shape(q->format, p.q.group_tiles * 4 * mx_group(q->format) / 8, T);
  Launch l(shape.ctas, shape.threads, stream);
  return launched(cudaLaunchKernelEx(&l.cfg, shape.kernel, p));
}

attn_res_status_t attn_res_mx_matmul(const attn_res_mx_t* a, const attn_res_mx_t* w,
                                     attn_res_bf16_t* out, int64_t out_row, uint32_t flags,
                                     void* stream) {
  const int kernel = static_cast<int>((flags >> 16) & 0xfu), split = static_cast<int>((flags >> 8) & 0xffu);
  if (!scalars_ok(a) || !scalars_ok(w) || a->format != w->format || a->cols != w->cols ||
      !known_flags(flags & ~(ATTN_RES_FLAG_KERNEL(0xf) | ATTN_RES_FLAG_SPLIT(0xff))) ||
      !product_overrides_ok(*a, *w, kernel, split))
    return ATTN_RES_EINVAL;
  if (a->rows == 0 || w->rows == 0) return ATTN_RES_OK;
  attn_res_status_t st = check_matrix(*a);
  if (st == ATTN_RES_OK) st = check_matrix(*w);
  if (st == ATTN_RES_OK) st = check_rows(out, a->rows, out_row, w->rows);
  if (st != ATTN_RES_OK) return st;
  const Span spans[7] = {rows_span(out, a->rows, out_row, w->rows, true),
                         data_span(*a, false),
                         scales_span(*a, false),
                         tensor_scale_span(*a),
                         data_span(*w, false),
                         scales_span(*w, false),
                         tensor_scale_span(*w)};
  if (written_overlap(spans)) return ATTN_RES_EALIAS;
  ProductCall c;
  st = current_device(&c.device);
  if (st != ATTN_RES_OK) return st;
  cudaError_t e = device_status_word(c.device, &c.err);
  if (e != cudaSuccess) return launched(e);
  c.a = a;
  c.w = w;
  c.out = out;
  c.out_row = out_row;
  c.pdl = (flags & ATTN_RES_FLAG_PDL) != 0;
  c.kernel = kernel;
  c.split = split;
  c.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_mx_product(c));
}

}  // extern "C"
