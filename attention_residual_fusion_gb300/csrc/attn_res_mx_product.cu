// attn_res_mx_product.cu -- launches of the microscaled product.
#include "attn_res_mx_host.cuh"

namespace attn_res_host {
namespace {

using namespace attn_res_dev;

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_tiled(EncodeTiled* out) {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult state;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                     cudaEnableDefault, &state);
    if (e != cudaSuccess) return e;
    if (state != cudaDriverEntryPointSuccess || f == nullptr) return cudaErrorNotSupported;
    found.store(f, std::memory_order_release);
  }
  *out = reinterpret_cast<EncodeTiled>(f);
  return cudaSuccess;
}

// Tensor map of an operand's codes as bytes: boxes of 128 bytes x `rows`,
// 128-byte swizzle; bytes past the row's end and rows past the last read as 0.
cudaError_t operand_map(const attn_res_mx_t& x, uint32_t rows, CUtensorMap* map) {
  EncodeTiled enc;
  cudaError_t e = encode_tiled(&enc);
  if (e != cudaSuccess) return e;
  const cuuint64_t dim[2] = {(cuuint64_t)(x.cols * mx_bits(x.format) / 8), (cuuint64_t)x.rows};
  const cuuint64_t stride[1] = {(cuuint64_t)x.row_bytes};
  const cuuint32_t box[2] = {128, rows};
  const cuuint32_t one[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x.data, dim, stride, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Of its scales: rows of 512 bytes (one tile of 128 rows x 4 groups), boxes of
// the tiles of one 128-byte block of codes.
cudaError_t scales_map(const attn_res_mx_t& x, uint32_t tiles, CUtensorMap* map) {
  EncodeTiled enc;
  cudaError_t e = encode_tiled(&enc);
  if (e != cudaSuccess) return e;
  const cuuint64_t dim[2] = {128, (cuuint64_t)((x.rows + 127) / 128 * mx_group_tiles(x.format, x.cols))};
  const cuuint64_t stride[1] = {512};
  const cuuint32_t box[2] = {128, tiles};
  const cuuint32_t one[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, x.scales, dim, stride, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int FMT>
ProductParams params(const ProductCall& c) {
  ProductParams p = {};
  p.a_scales = c.a->scales;
  p.w_scales = c.w->scales;
  p.a_g = c.a->tensor_scale;
  p.w_g = c.w->tensor_scale;
  p.out = c.out;
  p.out_row = c.out_row;
  p.m = c.a->rows;
  p.n = c.w->rows;
  p.group_tiles = mx_group_tiles(FMT, c.a->cols);
  p.row_bytes_used = (int)(c.a->cols * mx_bits(FMT) / 8);
  p.early_weights = c.pdl;
  p.err = c.err;
  return p;
}

// The dynamic shared memory above 48 KB is opt-in, per function and device.
template <class Kern>
cudaError_t allow_smem(Kern kern, uint32_t bytes, int device, std::atomic<uint64_t>& enabled) {
  const uint64_t bit = 1ull << device;
  if (!(enabled.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    enabled.fetch_or(bit, std::memory_order_acq_rel);
  }
  return cudaSuccess;
}

// Every launch is a programmatic one: its start-up overlaps the end of a
// preceding kernel that lets its dependents start (those of this library do,
// after their own wait), and it waits for that kernel before it touches memory.
struct Attributes {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  Attributes(dim3 grid, int threads, uint32_t smem, unsigned cluster, const ProductCall& c) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  Attributes(const Attributes&) = delete;
};

// CTAs that share a tile's K in the narrow form: two CTAs an SM (of 152) if
// that fills at least three quarters of them, else one (so that no SM has twice
// the work of another); at most 6 (clusters of 8 measured slower than of 4..6
// wherever they fit: 128 tokens x 2048 x 4096 9.3 us against 7.6, 64 x 4096 x
// 7168 8.8 against 7.4) and a block of K each.
int64_t narrow_split(int64_t tiles, int64_t blocks) {
  auto per_sm = [&](int64_t ctas) {
    const int64_t s = ctas / tiles;
    return s > kMaxSplit ? kMaxSplit : s < 1 ? 1 : s;
  };
  int64_t s = per_sm(304);
  if (s * tiles < 228) s = per_sm(152);
  return s < blocks ? s : blocks;
}

template <int FMT, int TN>
cudaError_t launch_narrow(const ProductCall& c) {
  using C = NarrowCfg<FMT, TN>;
  void (*kern)(ProductParams, CUtensorMap, CUtensorMap) = attn_res_mx_product_narrow_kernel<FMT, TN>;
  static std::atomic<uint64_t> enabled{0};
  cudaError_t e = allow_smem(kern, C::SMEM, c.device, enabled);
  CUtensorMap map_a, map_w;
  if (e == cudaSuccess) e = operand_map(*c.a, TN, &map_a);
  if (e == cudaSuccess) e = operand_map(*c.w, 128, &map_w);
  if (e != cudaSuccess) return e;
  const ProductParams p = params<FMT>(c);
  const int64_t n_tiles = (p.n + 127) / 128, m_tiles = (p.m + TN - 1) / TN;
  const int blocks = (p.row_bytes_used + 127) / 128;
  const int64_t split = c.split ? c.split : narrow_split(n_tiles * m_tiles, blocks);
  Attributes l(dim3((unsigned)(n_tiles * split), (unsigned)m_tiles, 1), C::THREADS, C::SMEM, (unsigned)split, c);
  return cudaLaunchKernelEx(&l.cfg, kern, p, map_a, map_w);
}

template <int FMT, int HALVES>
cudaError_t launch_wide(const ProductCall& c) {
  using C = WideCfg<FMT, HALVES>;
  void (*kern)(ProductParams, TileWalk, WideMaps) = attn_res_mx_product_wide_kernel<FMT, HALVES>;
  static std::atomic<uint64_t> enabled{0};
  static std::atomic<int> pairs_of[64];
  cudaError_t e = allow_smem(kern, C::SMEM, c.device, enabled);
  WideMaps maps;
  if (e == cudaSuccess) e = operand_map(*c.a, 128, &maps.a);
  if (e == cudaSuccess) e = operand_map(*c.w, C::HN / 2, &maps.w);
  if (e == cudaSuccess) e = scales_map(*c.a, C::F::ATOMS, &maps.a_sf);
  if (e == cudaSuccess) e = scales_map(*c.w, C::F::ATOMS, &maps.w_sf);
  if (e != cudaSuccess) return e;
  const ProductParams p = params<FMT>(c);
  const int64_t m_tiles = (p.m + C::TM - 1) / C::TM, n_tiles = (p.n + C::TN - 1) / C::TN;
  const int64_t tiles = m_tiles * n_tiles;
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  const TileWalk walk{(int)m_tiles, (int)n_tiles};
  Attributes l(dim3(2, 1, 1), C::THREADS, C::SMEM, 2, c);
  int pairs = pairs_of[c.device].load(std::memory_order_acquire);
  if (pairs == 0) {  // that the device holds at once
    e = cudaOccupancyMaxActiveClusters(&pairs, kern, &l.cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    pairs_of[c.device].store(pairs, std::memory_order_release);
  }
  l.cfg.gridDim.x = 2 * (unsigned)(tiles < pairs ? tiles : pairs);
  return cudaLaunchKernelEx(&l.cfg, kern, p, walk, maps);
}

// The forms' times in units of 10 ns, for the choice between them, from graph
// replays on GB300 of 1..8192 tokens x 1024..16384 columns x 1024..8192 (all
// formats, inputs in L2).  A pair of the wide form takes 0.8 us and 0.34 us
// for each 128-byte block of K for a tile of 256 columns, 1.75 us and 0.40 us
// for one of 384; 76 pairs work at once; 6 us for the launch, the first loads
// and the last stores.  The narrow form's 128-token tiles take in 34 KB for
// each block, about 10 TB/s in all, and 5.5 us for the rest:
//   tokens x columns x K       narrow     wide      wider
//   128 x 7168 x 7168 mxfp4    12.1 us    15.2 us        -
//   300 x 2050 x 7200 mxfp8    14.5       25.3      30.0 us
//   256 x 7168 x 7168 mxfp4    14.8       15.6      18.5
//   512 x 7168 x 7168 mxfp4    17.2       16.2      19.1
//   1024 x 7168 x 7168 mxfp4   31.1       26.7      20.2
//   8192 x 8192 x 1024 mxfp4     -        36.2      41.4
//   4096 x 16384 x 2048 nvfp4    -        55.2      55.1
//   8192 x 7168 x 7168 mxfp4     -       129       109
int64_t wide_cost(const ProductCall& c, int64_t blocks, int tile_columns) {
  const int64_t tiles = (c.a->rows + 255) / 256 * ((c.w->rows + tile_columns - 1) / tile_columns);
  const int64_t waves = (tiles + 75) / 76;
  return 600 + waves * (tile_columns == 256 ? 80 + 34 * blocks : 175 + 40 * blocks);
}
int64_t narrow_cost(const ProductCall& c, int64_t blocks) {
  const int64_t tiles = (c.a->rows + 127) / 128 * ((c.w->rows + 127) / 128);
  return 550 + tiles * blocks * 34 / 100;
}

// Token tiles of the narrow form's grid (its y).
constexpr int64_t kNarrowMaxRows = int64_t(65535) * 128;
int64_t k_blocks(const attn_res_mx_t& a) { return (a.cols * mx_bits(a.format) / 8 + 127) / 128; }

template <int FMT>
cudaError_t launch_format(const ProductCall& c) {
  const int64_t rows = c.a->rows, blocks = k_blocks(*c.a);
  int kernel = c.kernel;
  if (kernel == 0) {
    const int64_t one = wide_cost(c, blocks, 256), two = wide_cost(c, blocks, 384);
    // up to 64 tokens the narrow form's time is that of reading the weights
    if (rows <= 64 || (rows <= kNarrowMaxRows && narrow_cost(c, blocks) < (one < two ? one : two)))
      kernel = ATTN_RES_MX_NARROW;
    else
      kernel = one <= two ? ATTN_RES_MX_WIDE : ATTN_RES_MX_WIDER;
  }
  if (kernel == ATTN_RES_MX_WIDE) return launch_wide<FMT, 1>(c);
  if (kernel == ATTN_RES_MX_WIDER) return launch_wide<FMT, 2>(c);
  if (rows <= 16) return launch_narrow<FMT, 16>(c);
  if (rows <= 32) return launch_narrow<FMT, 32>(c);
  if (rows <= 64) return launch_narrow<FMT, 64>(c);
  return launch_narrow<FMT, 128>(c);
}

}  // namespace

cudaError_t launch_mx_product(const ProductCall& c) {
  switch (c.a->format) {
    case ATTN_RES_MXFP8: return launch_format<ATTN_RES_MXFP8>(c);
    case ATTN_RES_MXFP4: return launch_format<ATTN_RES_MXFP4>(c);
    case ATTN_RES_NVFP4: return launch_format<ATTN_RES_NVFP4>(c);
    default: return cudaErrorInvalidValue;
  }
}

bool product_overrides_ok(const attn_res_mx_t& a, int kernel, int split) {
  if (kernel < 0 || kernel > ATTN_RES_MX_WIDER) return false;
  if (kernel == ATTN_RES_MX_NARROW) return a.rows <= kNarrowMaxRows && split <= kMaxSplit && split <= k_blocks(a);
  return split == 0;
}

}  // namespace attn_res_host
