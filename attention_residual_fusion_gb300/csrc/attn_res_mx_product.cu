// attn_res_mx_product.cu -- launches of the microscaled product.
#include "attn_res_mx_host.cuh"
#include "attn_res_tensor_host.cuh"

namespace attn_res_host {
namespace {

using namespace attn_res_dev;

// Tensor map of an operand's codes as bytes: boxes of 128 bytes x `rows`,
// 128-byte swizzle; bytes past the row's end and rows past the last read as 0.
cudaError_t operand_map(const attn_res_mx_t& x, uint32_t rows, CUtensorMap* map) {
  return map_2d(CU_TENSOR_MAP_DATA_TYPE_UINT8, x.data, x.cols * mx_bits(x.format) / 8, x.rows, x.row_bytes, 128, rows,
                CU_TENSOR_MAP_SWIZZLE_128B, map);
}

// Of its scales: rows of 512 bytes (one tile of 128 rows x 4 groups), boxes of
// the tiles of one 128-byte block of codes.
cudaError_t scales_map(const attn_res_mx_t& x, uint32_t tiles, CUtensorMap* map) {
  return map_2d(CU_TENSOR_MAP_DATA_TYPE_UINT32, x.scales, 128, (x.rows + 127) / 128 * mx_group_tiles(x.format, x.cols),
                512, 128, tiles, CU_TENSOR_MAP_SWIZZLE_NONE, map);
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

// The choice of form and split: each one's time by a model of it, in units of
// 10 ns, whose constants were fitted to 414 products behind another small call
// of the library (graph replays on GB300, inputs in L2: 1..8192 tokens x
// 64..16384 columns x 32..8192, all formats, every form and split).  Over these
// the choice takes 0.6 % longer than the best form in the geometric mean, and
// 15 % at most; over 125 others 0.8 % and 11 %.
//
// Narrow form: waves of clusters.  A wave that leaves an SM a single CTA takes
// less for each 128-byte block of K and for the joining of the parts than one
// with two; more than 64 tokens (tiles of 128) cost more in all of these.
// Clusters of three and more leave some SMs without a second CTA: kClusters[s]
// of s CTAs run at once on GB300's 152 SMs, and as a second wave the rest
// takes as long again (3200 x 512 x 2368 mxfp8 in three parts, 100 clusters,
// 16.4 us; whole 10.0).  (Counted by the driver for a kernel of this shape
// without TMEM; for one that takes TMEM it counts a CTA an SM, whatever the
// columns.)
constexpr int kSms = 152;
constexpr int kClusters[kMaxSplit + 1] = {0, 304, 152, 97, 74, 58, 46};
struct NarrowCosts {
  int base;             // launch, first loads, results
  int block, block2;    // a CTA's block of K: one CTA an SM, two
  int two;              // two CTAs an SM: first loads and results
  int join, join2;      // joining: one CTA an SM, two
  int join2_part;       // two: for each part
  int wave;             // a wave before the last one
};
constexpr NarrowCosts kNarrowFew = {220, 28, 28, 65, 50, 55, 28, 173};    // up to 64 tokens
constexpr NarrowCosts kNarrowMany = {420, 26, 46, 128, 105, 151, 0, 410};  // tiles of 128 tokens
int64_t narrow_cost(const NarrowCosts& k, int64_t tiles, int64_t blocks, int split) {
  const int64_t per_cta = (blocks + split - 1) / split, clusters = kClusters[split];
  const int64_t waves = (tiles + clusters - 1) / clusters;
  const bool two = (tiles - (waves - 1) * clusters) * split > kSms;
  int64_t t = k.base + (waves - 1) * (k.wave + k.block2 * per_cta);
  t += two ? k.two + k.block2 * per_cta : k.block * per_cta;
  if (split > 1) t += two ? k.join2 + k.join2_part * split : k.join;
  return t;
}
// Wide forms: waves of pairs, a tile's blocks of K, and the way of all results
// to memory (34000 of them take 10 ns at the copy rate).
//   tokens x columns x K        narrow     wide      wider   (us, the small call's 1.3 us taken off)
//   300 x 2050 x 7200 mxfp8      12.8      23.2       27.6
//   128 x 7168 x 7168 mxfp4      10.2      13.9       16.8
//   256 x 7168 x 7168 mxfp4      12.2      14.0       16.9
//   512 x 7168 x 7168 mxfp4      15.3      14.3       16.9
//   1024 x 7168 x 7168 mxfp4     28.8      24.7       18.4
//   4096 x 256 x 1024 mxfp4       5.3       6.0        7.0
//   4096 x 4096 x 128 mxfp4      18.1      11.6       12.9
//   8192 x 16384 x 128 mxfp4      125      61.2       63.5
//   8192 x 7168 x 32 nvfp4       61.2      31.2       29.4
struct WideCosts {
  int base, tile, block;
  int results;  // for 34000 results, in hundredths
};
constexpr WideCosts kWide = {372, 51, 36, 62}, kWider = {364, 77, 43, 88};
int64_t wide_cost(const WideCosts& k, const ProductCall& c, int64_t blocks, int tile_columns, int64_t pairs) {
  const int64_t tiles = (c.a->rows + 255) / 256 * ((c.w->rows + tile_columns - 1) / tile_columns);
  const int64_t waves = (tiles + pairs - 1) / pairs;
  return k.base + waves * (k.tile + k.block * blocks) + c.a->rows * c.w->rows / 34000 * k.results / 100;
}

// Token tiles of the narrow form's grid (its y).
constexpr int64_t kNarrowMaxRows = int64_t(65535) * 128;
// Weight rows of the wide forms, whose last tile may reach past them by less
// than two tiles: their places are 32-bit (of the tensor maps).
constexpr int64_t kWideMaxColumns = (int64_t(1) << 31) - 2 * 384;
int64_t k_blocks(const attn_res_mx_t& a) { return (a.cols * mx_bits(a.format) / 8 + 127) / 128; }

// The least cost of the splits 1..kMaxSplit, and that split.
int64_t plan_narrow(const ProductCall& c, int tile_tokens, int64_t blocks, int* split) {
  const int64_t tiles = (c.w->rows + 127) / 128 * ((c.a->rows + tile_tokens - 1) / tile_tokens);
  const NarrowCosts& k = tile_tokens == 128 ? kNarrowMany : kNarrowFew;
  int64_t least = narrow_cost(k, tiles, blocks, 1);
  *split = 1;
  for (int s = 2; s <= kMaxSplit && s <= blocks; ++s) {
    const int64_t t = narrow_cost(k, tiles, blocks, s);
    if (t < least) {
      least = t;
      *split = s;
    }
  }
  return least;
}

template <int FMT, int TN>
cudaError_t launch_narrow(const ProductCall& c, int split) {
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
  Attributes l(dim3((unsigned)(n_tiles * split), (unsigned)m_tiles, 1), C::THREADS, C::SMEM, (unsigned)split, c);
  return cudaLaunchKernelEx(&l.cfg, kern, p, map_a, map_w);
}

template <int FMT, int HALVES>
struct Wide {
  using C = WideCfg<FMT, HALVES>;
  static constexpr auto kern = attn_res_mx_product_wide_kernel<FMT, HALVES>;

  // Pairs that the device holds at once.
  static cudaError_t resident(const ProductCall& c, int* pairs) {
    static std::atomic<uint64_t> enabled{0};
    static std::atomic<int> known[64];
    *pairs = known[c.device].load(std::memory_order_acquire);
    if (*pairs != 0) return cudaSuccess;
    cudaError_t e = allow_smem(kern, C::SMEM, c.device, enabled);
    const Attributes l(dim3(2, 1, 1), C::THREADS, C::SMEM, 2, c);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(pairs, kern, &l.cfg);
    if (e != cudaSuccess) return e;
    if (*pairs < 1) return cudaErrorInvalidConfiguration;
    known[c.device].store(*pairs, std::memory_order_release);
    return cudaSuccess;
  }
  static cudaError_t launch(const ProductCall& c, int pairs) {
    WideMaps maps;
    cudaError_t e = operand_map(*c.a, 128, &maps.a);
    if (e == cudaSuccess) e = operand_map(*c.w, C::HN / 2, &maps.w);
    if (e == cudaSuccess) e = scales_map(*c.a, C::F::ATOMS, &maps.a_sf);
    if (e == cudaSuccess) e = scales_map(*c.w, C::F::ATOMS, &maps.w_sf);
    if (e != cudaSuccess) return e;
    const int64_t m_tiles = (c.a->rows + C::TM - 1) / C::TM, n_tiles = (c.w->rows + C::TN - 1) / C::TN;
    const int64_t tiles = m_tiles * n_tiles;
    if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    const TileWalk walk{(int)m_tiles, (int)n_tiles};
    Attributes l(dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs), 1, 1), C::THREADS, C::SMEM, 2, c);
    return cudaLaunchKernelEx(&l.cfg, kern, params<FMT>(c), walk, maps);
  }
};

template <int FMT>
cudaError_t launch_format(const ProductCall& c) {
  using One = Wide<FMT, 1>;
  using Two = Wide<FMT, 2>;
  const int64_t rows = c.a->rows, blocks = k_blocks(*c.a);
  const int tile_tokens = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  int kernel = c.kernel, split = c.split, one_pairs = 0, two_pairs = 0;
  int64_t narrow = INT64_MAX;
  // up to 64 tokens the narrow form's time is that of reading the weights
  if (kernel == 0 && rows <= 64) kernel = ATTN_RES_MX_NARROW;
  if (split == 0 && (kernel == 0 ? rows <= kNarrowMaxRows : kernel == ATTN_RES_MX_NARROW))
    narrow = plan_narrow(c, tile_tokens, blocks, &split);
  cudaError_t e = cudaSuccess;
  if (kernel == 0 || kernel == ATTN_RES_MX_WIDE) e = One::resident(c, &one_pairs);
  if (e == cudaSuccess && (kernel == 0 || kernel == ATTN_RES_MX_WIDER)) e = Two::resident(c, &two_pairs);
  if (e != cudaSuccess) return e;
  if (kernel == 0) {
    const int64_t one = wide_cost(kWide, c, blocks, 256, one_pairs);
    const int64_t two = wide_cost(kWider, c, blocks, 384, two_pairs);
    kernel = narrow < (one < two ? one : two) || c.w->rows > kWideMaxColumns ? ATTN_RES_MX_NARROW
             : one <= two                                                    ? ATTN_RES_MX_WIDE
                                                                             : ATTN_RES_MX_WIDER;
  }
  if (kernel == ATTN_RES_MX_WIDE) return One::launch(c, one_pairs);
  if (kernel == ATTN_RES_MX_WIDER) return Two::launch(c, two_pairs);
  switch (tile_tokens) {
    case 16: return launch_narrow<FMT, 16>(c, split);
    case 32: return launch_narrow<FMT, 32>(c, split);
    case 64: return launch_narrow<FMT, 64>(c, split);
    default: return launch_narrow<FMT, 128>(c, split);
  }
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

bool product_overrides_ok(const attn_res_mx_t& a, const attn_res_mx_t& w, int kernel, int split) {
  if (kernel < 0 || kernel > ATTN_RES_MX_WIDER) return false;
  if (kernel == ATTN_RES_MX_NARROW) return a.rows <= kNarrowMaxRows && split <= kMaxSplit && split <= k_blocks(a);
  return split == 0 && (kernel == 0 || w.rows <= kWideMaxColumns);
}

}  // namespace attn_res_host
