// attn_res_f8_api.cu -- the 8-bit entry points of include/attn_res.h: argument
// checks and the launches of the row kernels (the products' are in
// attn_res_f8_product.cu).  Nothing is launched and nothing is written unless
// every check passes.
#include "attn_res_f8_host.cuh"
#include "attn_res_f8_rows.cuh"
#include "attn_res_tensor_host.cuh"

namespace {

using namespace attn_res_dev;
using namespace attn_res_host;

constexpr int64_t kMaxSide = (int64_t(1) << 31) - 1024;  // places of tensor maps and grids are 32-bit

// What a matrix is whatever its pointers: kind and sizes.
bool scalars_ok(const attn_res_f8_t* q, int block = 0) {
  return q != nullptr && (block == 0 ? q->block == ATTN_RES_F8_ROWS || q->block == ATTN_RES_F8_SQUARE : q->block == block) &&
         q->rows >= 0 && q->rows <= kMaxSide && q->cols >= 0 && q->cols <= kMaxSide;
}
bool shaped(const attn_res_f8_t* q, int block, int64_t rows, int64_t cols) {
  return scalars_ok(q, block) && q->rows == rows && q->cols == cols;
}
bool known_activation(int a) { return a == ATTN_RES_SILU || a == ATTN_RES_GELU; }

// Rows of scales, and scales in one.
int64_t scale_rows(const attn_res_f8_t& q) { return f8_blocks(q.block == ATTN_RES_F8_ROWS ? q.cols : q.rows); }
int64_t scale_cols(const attn_res_f8_t& q) { return q.block == ATTN_RES_F8_ROWS ? q.rows : f8_blocks(q.cols); }

attn_res_status_t check_matrix(const attn_res_f8_t& q) {
  if (q.rows == 0 || q.cols == 0) return ATTN_RES_OK;
  if (!q.data || !q.scales || q.row_bytes < q.cols || q.row_bytes >= kMaxStride || !span_ok(q.rows, q.row_bytes) ||
      q.scales_row < scale_cols(q) || q.scales_row >= kMaxStride || !span_ok(scale_rows(q), q.scales_row))
    return ATTN_RES_EINVAL;
  if (!aligned(q.data, 16) || q.row_bytes % 16 != 0) return ATTN_RES_EALIGN;
  const bool rows = q.block == ATTN_RES_F8_ROWS;
  if (!aligned(q.scales, rows ? 16 : 4) || (rows && q.scales_row % 4 != 0)) return ATTN_RES_EALIGN;
  return ATTN_RES_OK;
}
attn_res_status_t check_f32_rows(const float* x, int64_t rows, int64_t row, int64_t width) {
  if (!x || row < width || row > kMaxStride || !span_ok(rows, row)) return ATTN_RES_EINVAL;
  if (!aligned(x, 16) || row % 4 != 0) return ATTN_RES_EALIGN;
  return ATTN_RES_OK;
}

constexpr uint32_t kOverrides = ATTN_RES_FLAG_KERNEL(0xf) | ATTN_RES_FLAG_SPLIT(0xff);
void overrides(uint32_t flags, F8Call* c) {
  c->kernel = static_cast<int>((flags >> 16) & 0xfu);
  c->split = static_cast<int>((flags >> 8) & 0xffu);
}

// The ranges of a call's arguments, two for a matrix.
template <int N>
struct Spans {
  Span at[N];
  int used = 0;
  void add(const attn_res_f8_t* q, bool written) {
    if (q == nullptr || q->rows == 0 || q->cols == 0) return;
    at[used++] = span(q->data, (q->rows - 1) * q->row_bytes + q->cols, written);
    at[used++] = span(q->scales, ((scale_rows(*q) - 1) * q->scales_row + scale_cols(*q)) * 4, written);
  }
  void add(Span s) { at[used++] = s; }
  bool clash() const { return written_overlap(at); }
};

F8View view(const attn_res_f8_t& q) {
  return {static_cast<uint8_t*>(q.data), q.scales, q.row_bytes, q.scales_row, q.rows, q.cols};
}

// CTAs of a kernel with a warp for each strip, or a CTA for each tile; -1 where
// they are too many (beyond any device's memory).
int64_t strip_ctas(int64_t rows, int64_t cols) {
  const int64_t jobs = (rows + kF8Strip - 1) / kF8Strip * f8_blocks(cols);
  const int64_t ctas = (jobs + kF8Threads / 32 - 1) / (kF8Threads / 32);
  return ctas <= INT32_MAX ? ctas : -1;
}
int64_t tile_ctas(int64_t rows, int64_t cols) {
  const int64_t ctas = f8_blocks(rows) * f8_blocks(cols);
  return ctas <= INT32_MAX ? ctas : -1;
}

template <class... Params>
attn_res_status_t run(void (*kern)(Params...), int64_t ctas, void* stream, const Params&... p) {
  int device;
  const attn_res_status_t st = current_device(&device);
  if (st != ATTN_RES_OK) return st;
  Launch l(ctas, kF8Threads, stream);
  return launched(cudaLaunchKernelEx(&l.cfg, kern, p...));
}

template <int ACT, bool TRANSPOSED>
cudaError_t launch_backward(const F8BackwardParams& p, const F8BackwardMaps& maps, int device, void* stream) {
  const auto kern = attn_res_f8_gated_backward_kernel<ACT, TRANSPOSED>;
  static std::atomic<uint64_t> enabled{0};
  static std::atomic<int> sms[64];
  cudaError_t e = allow_smem(kern, sizeof(F8BackShared), device, enabled);
  int ctas = sms[device].load(std::memory_order_acquire);
  if (e == cudaSuccess && ctas == 0) {
    e = cudaDeviceGetAttribute(&ctas, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) sms[device].store(ctas, std::memory_order_release);
  }
  if (e != cudaSuccess) return e;
  Launch l(p.tiles < ctas ? p.tiles : ctas, kF8BackThreads, stream);
  l.cfg.dynamicSmemBytes = sizeof(F8BackShared);
  return cudaLaunchKernelEx(&l.cfg, kern, p, maps);
}

}  // namespace

extern "C" {

attn_res_status_t attn_res_f8_quantize(const attn_res_bf16_t* x, int64_t x_row, const attn_res_f8_t* q,
                                       const attn_res_f8_t* qt, uint32_t flags, void* stream) {
  if (!scalars_ok(q) || !known_flags(flags) || (qt != nullptr && !shaped(qt, q->block, q->cols, q->rows)))
    return ATTN_RES_EINVAL;
  if (q->rows == 0 || q->cols == 0) return ATTN_RES_OK;
  attn_res_status_t st = check_matrix(*q);
  if (st == ATTN_RES_OK && qt) st = check_matrix(*qt);
  if (st == ATTN_RES_OK) st = check_rows(x, q->rows, x_row, q->cols);
  if (st != ATTN_RES_OK) return st;
  Spans<5> spans;
  spans.add(rows_span(x, q->rows, x_row, q->cols, false));
  spans.add(q, true);
  spans.add(qt, true);
  if (spans.clash()) return ATTN_RES_EALIAS;
  F8QuantizeParams p = {};
  p.x = x;
  p.x_row = x_row;
  p.q = view(*q);
  if (qt) p.t = view(*qt);
  const bool square = q->block == ATTN_RES_F8_SQUARE, strips = !square && !qt;
  const int64_t ctas = strips ? strip_ctas(q->rows, q->cols) : tile_ctas(q->rows, q->cols);
  if (ctas < 0) return ATTN_RES_EINVAL;
  if (strips) return run(attn_res_f8_quantize_rows_kernel, ctas, stream, p);
  if (!square) return run(attn_res_f8_quantize_tile_kernel<false, true>, ctas, stream, p);
  return qt ? run(attn_res_f8_quantize_tile_kernel<true, true>, ctas, stream, p)
            : run(attn_res_f8_quantize_tile_kernel<true, false>, ctas, stream, p);
}

attn_res_status_t attn_res_f8_dequantize(const attn_res_f8_t* q, attn_res_bf16_t* x, int64_t x_row, uint32_t flags,
                                         void* stream) {
  if (!scalars_ok(q) || !known_flags(flags)) return ATTN_RES_EINVAL;
  if (q->rows == 0 || q->cols == 0) return ATTN_RES_OK;
  attn_res_status_t st = check_matrix(*q);
  if (st == ATTN_RES_OK) st = check_rows(x, q->rows, x_row, q->cols);
  if (st != ATTN_RES_OK) return st;
  Spans<3> spans;
  spans.add(rows_span(x, q->rows, x_row, q->cols, true));
  spans.add(q, false);
  if (spans.clash()) return ATTN_RES_EALIAS;
  const int64_t ctas = strip_ctas(q->rows, q->cols);
  if (ctas < 0) return ATTN_RES_EINVAL;
  const F8DequantizeParams p = {view(*q), x, x_row};
  return q->block == ATTN_RES_F8_SQUARE ? run(attn_res_f8_dequantize_kernel<true>, ctas, stream, p)
                                        : run(attn_res_f8_dequantize_kernel<false>, ctas, stream, p);
}

attn_res_status_t attn_res_f8_matmul(const attn_res_f8_t* a, const attn_res_f8_t* w, const attn_res_f8_t* a2,
                                     const attn_res_f8_t* w2, void* out, int64_t out_row, int out_type,
                                     uint32_t flags, void* stream) {
  if (!scalars_ok(a, ATTN_RES_F8_ROWS) || !scalars_ok(w) || a->cols != w->cols || !known_flags(flags & ~kOverrides) ||
      out_type < ATTN_RES_OUT_BF16 || out_type > ATTN_RES_OUT_F32_ADD || (a2 == nullptr) != (w2 == nullptr))
    return ATTN_RES_EINVAL;
  if (a2 != nullptr && (!scalars_ok(a2, ATTN_RES_F8_ROWS) || !scalars_ok(w2, w->block) || a2->rows != a->rows ||
                        w2->rows != w->rows || a2->cols != w2->cols))
    return ATTN_RES_EINVAL;
  F8Call c = {};
  c.a = a;
  c.w = w;
  c.a2 = a2;
  c.w2 = w2;
  overrides(flags, &c);
  if (!f8_overrides_ok(c)) return ATTN_RES_EINVAL;
  if (a->rows == 0 || w->rows == 0) return ATTN_RES_OK;
  attn_res_status_t st = check_matrix(*a);
  if (st == ATTN_RES_OK) st = check_matrix(*w);
  if (st == ATTN_RES_OK && a2) st = check_matrix(*a2);
  if (st == ATTN_RES_OK && a2) st = check_matrix(*w2);
  const bool f32 = out_type != ATTN_RES_OUT_BF16;
  if (st == ATTN_RES_OK)
    st = f32 ? check_f32_rows(static_cast<const float*>(out), a->rows, out_row, w->rows)
             : check_rows(static_cast<const attn_res_bf16_t*>(out), a->rows, out_row, w->rows);
  if (st != ATTN_RES_OK) return st;
  Spans<9> spans;
  spans.add(span(out, ((a->rows - 1) * out_row + w->rows) * (f32 ? 4 : 2), true));
  spans.add(a, false);
  spans.add(w, false);
  spans.add(a2, false);
  spans.add(w2, false);
  if (spans.clash()) return ATTN_RES_EALIAS;
  if (!f8_choose_form(&c)) return ATTN_RES_EINVAL;
  st = current_device(&c.device);
  if (st != ATTN_RES_OK) return st;
  cudaError_t e = device_status_word(c.device, &c.err);
  if (e != cudaSuccess) return launched(e);
  c.out = out;
  c.out_row = out_row;
  c.out_type = out_type;
  c.pdl = (flags & ATTN_RES_FLAG_PDL) != 0;
  c.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_f8_product(c));
}

attn_res_status_t attn_res_f8_gated(const attn_res_f8_t* x, const attn_res_f8_t* gate, const attn_res_f8_t* up,
                                    int activation, const attn_res_f8_t* h, attn_res_bf16_t* h_rows, int64_t h_row,
                                    const attn_res_f8_t* save_g, const attn_res_f8_t* save_u, uint32_t flags,
                                    void* stream) {
  if (!scalars_ok(x, ATTN_RES_F8_ROWS) || !scalars_ok(gate, ATTN_RES_F8_SQUARE) || gate->cols != x->cols ||
      !shaped(up, ATTN_RES_F8_SQUARE, gate->rows, gate->cols) || !known_activation(activation) ||
      !known_flags(flags & ~kOverrides) || (h != nullptr && h_rows != nullptr) || (save_g == nullptr) != (save_u == nullptr))
    return ATTN_RES_EINVAL;
  const int64_t T = x->rows, F = gate->rows;
  for (const attn_res_f8_t* q : {h, save_g, save_u})
    if (q != nullptr && !shaped(q, ATTN_RES_F8_ROWS, T, F)) return ATTN_RES_EINVAL;
  F8Call c = {};
  c.a = x;
  c.w = gate;
  c.w2 = up;
  c.gated = true;
  overrides(flags, &c);
  if (!f8_overrides_ok(c)) return ATTN_RES_EINVAL;
  if (T == 0 || F == 0) return ATTN_RES_OK;
  attn_res_status_t st = check_matrix(*x);
  for (const attn_res_f8_t* q : {gate, up, h, save_g, save_u})
    if (st == ATTN_RES_OK && q != nullptr) st = check_matrix(*q);
  if (st == ATTN_RES_OK && h == nullptr) st = check_rows(h_rows, T, h_row, F);
  if (st != ATTN_RES_OK) return st;
  Spans<13> spans;
  for (const attn_res_f8_t* q : {x, gate, up}) spans.add(q, false);
  for (const attn_res_f8_t* q : {h, save_g, save_u}) spans.add(q, true);
  spans.add(rows_span(h_rows, T, h_row, F, true));
  if (spans.clash()) return ATTN_RES_EALIAS;
  if (!f8_choose_form(&c)) return ATTN_RES_EINVAL;
  st = current_device(&c.device);
  if (st != ATTN_RES_OK) return st;
  cudaError_t e = device_status_word(c.device, &c.err);
  if (e != cudaSuccess) return launched(e);
  c.activation = activation;
  c.h = h;
  c.g = save_g;
  c.u = save_u;
  c.out = h_rows;
  c.out_row = h_row;
  c.pdl = (flags & ATTN_RES_FLAG_PDL) != 0;
  c.stream = static_cast<cudaStream_t>(stream);
  return launched(launch_f8_product(c));
}

attn_res_status_t attn_res_f8_gated_backward(const attn_res_bf16_t* dh, int64_t dh_row, const attn_res_f8_t* g,
                                             const attn_res_f8_t* u, int activation, const attn_res_f8_t* dg,
                                             const attn_res_f8_t* du, const attn_res_f8_t* dg_t,
                                             const attn_res_f8_t* du_t, const attn_res_f8_t* h_t, uint32_t flags,
                                             void* stream) {
  if (!scalars_ok(g, ATTN_RES_F8_ROWS) || !known_activation(activation) || !known_flags(flags)) return ATTN_RES_EINVAL;
  const int64_t T = g->rows, F = g->cols;
  for (const attn_res_f8_t* q : {u, dg, du})
    if (!shaped(q, ATTN_RES_F8_ROWS, T, F)) return ATTN_RES_EINVAL;
  const bool transposed = dg_t != nullptr;
  for (const attn_res_f8_t* q : {dg_t, du_t, h_t})
    if ((q != nullptr) != transposed || (q != nullptr && !shaped(q, ATTN_RES_F8_ROWS, F, T))) return ATTN_RES_EINVAL;
  if (T == 0 || F == 0) return ATTN_RES_OK;
  attn_res_status_t st = check_rows(dh, T, dh_row, F);
  for (const attn_res_f8_t* q : {g, u, dg, du, dg_t, du_t, h_t})
    if (st == ATTN_RES_OK && q != nullptr) st = check_matrix(*q);
  if (st != ATTN_RES_OK) return st;
  // (these are read through tensor maps, which hold strides below 2^40 bytes)
  if (dh_row * 2 >= kMaxStride || g->scales_row * 4 >= kMaxStride || u->scales_row * 4 >= kMaxStride)
    return ATTN_RES_EINVAL;
  Spans<15> spans;
  spans.add(rows_span(dh, T, dh_row, F, false));
  for (const attn_res_f8_t* q : {g, u}) spans.add(q, false);
  for (const attn_res_f8_t* q : {dg, du, dg_t, du_t, h_t}) spans.add(q, true);
  if (spans.clash()) return ATTN_RES_EALIAS;
  const int64_t tiles = tile_ctas(T, F);
  if (tiles < 0 || tiles > INT32_MAX / 2) return ATTN_RES_EINVAL;
  F8BackwardParams p = {};
  F8BackwardMaps maps;
  int device;
  st = current_device(&device);
  if (st != ATTN_RES_OK) return st;
  cudaError_t e = device_status_word(device, &p.err);
  auto map = [&](CUtensorMapDataType type, const void* at, int64_t cols, int64_t rows, int64_t row_bytes,
                 uint32_t box_rows, CUtensorMap* m) {
    if (e == cudaSuccess) e = map_2d(type, at, cols, rows, row_bytes, 128, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE, m);
  };
  map(CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dh, F, T, dh_row * 2, 128, &maps.dh);
  map(CU_TENSOR_MAP_DATA_TYPE_UINT8, g->data, F, T, g->row_bytes, 128, &maps.g);
  map(CU_TENSOR_MAP_DATA_TYPE_UINT8, u->data, F, T, u->row_bytes, 128, &maps.u);
  map(CU_TENSOR_MAP_DATA_TYPE_FLOAT32, g->scales, T, f8_blocks(F), g->scales_row * 4, 1, &maps.g_scales);
  map(CU_TENSOR_MAP_DATA_TYPE_FLOAT32, u->scales, T, f8_blocks(F), u->scales_row * 4, 1, &maps.u_scales);
  if (e != cudaSuccess) return launched(e);
  p.dg = view(*dg);
  p.du = view(*du);
  if (transposed) {
    p.dg_t = view(*dg_t);
    p.du_t = view(*du_t);
    p.h_t = view(*h_t);
  }
  p.tiles = (int)tiles;
  p.col_tiles = (int)f8_blocks(F);
  const bool silu = activation == ATTN_RES_SILU;
  if (transposed)
    e = silu ? launch_backward<ATTN_RES_SILU, true>(p, maps, device, stream)
             : launch_backward<ATTN_RES_GELU, true>(p, maps, device, stream);
  else
    e = silu ? launch_backward<ATTN_RES_SILU, false>(p, maps, device, stream)
             : launch_backward<ATTN_RES_GELU, false>(p, maps, device, stream);
  return launched(e);
}

}  // extern "C"
