// attn_res_f8_product.cu -- launches of the 8-bit products.
#include <algorithm>

#include "attn_res_f8_host.cuh"
#include "attn_res_f8_product.cuh"
#include "attn_res_tensor_host.cuh"

namespace attn_res_host {
namespace {

using namespace attn_res_dev;

// Tensor map of an operand's codes: boxes of 128 bytes x `rows`, swizzled.
cudaError_t codes_map(const attn_res_f8_t& x, uint32_t rows, CUtensorMap* map) {
  return map_2d(CU_TENSOR_MAP_DATA_TYPE_UINT8, x.data, x.cols, x.rows, x.row_bytes, 128, rows,
                CU_TENSOR_MAP_SWIZZLE_128B, map);
}

F8View view(const attn_res_f8_t* q) {
  F8View v = {};
  if (q != nullptr) v = {static_cast<uint8_t*>(q->data), q->scales, q->row_bytes, q->scales_row, q->rows, q->cols};
  return v;
}

F8ProductParams params(const F8Call& c) {
  F8ProductParams p = {};
  p.a[0] = {c.a->scales, c.a->scales_row};
  p.w[0] = {c.w->scales, c.w->scales_row};
  if (c.a2 != nullptr) p.a[1] = {c.a2->scales, c.a2->scales_row};
  if (c.w2 != nullptr) p.w[1] = {c.w2->scales, c.w2->scales_row};
  p.blocks[0] = (int)f8_blocks(c.a->cols);
  p.blocks[1] = c.a2 != nullptr ? (int)f8_blocks(c.a2->cols) : 0;
  p.m = c.a->rows;
  p.n = c.w->rows;
  p.out = c.out;
  p.out_row = c.out_row;
  p.add = c.out_type == ATTN_RES_OUT_F32_ADD;
  p.h = view(c.h);
  p.g = view(c.g);
  p.u = view(c.u);
  p.err = c.err;
  return p;
}

// Every launch is a programmatic one: its start-up overlaps the end of a
// preceding kernel that lets its dependents start, and it waits for that kernel
// before it touches memory.
struct Attributes {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  Attributes(dim3 grid, int threads, uint32_t smem, unsigned cluster, cudaStream_t stream) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  Attributes(const Attributes&) = delete;
};

// The operands' maps, boxes of `a_rows` and 128 rows.
cudaError_t product_maps(const F8Call& c, uint32_t a_rows, F8ProductMaps* maps) {
  cudaError_t e = cudaSuccess;
  for (int t = 0; t < 2; ++t) {
    const attn_res_f8_t *a = t ? c.a2 : c.a, *w = t ? c.w2 : c.w;
    // (a term of width 0 has no blocks, and maps of nothing are none)
    if (e == cudaSuccess && a != nullptr && a->cols > 0) e = codes_map(*a, a_rows, &maps->a[t]);
    if (e == cudaSuccess && w != nullptr && w->cols > 0) e = codes_map(*w, 128, &maps->w[t]);
  }
  return e;
}

// Tiles of the wide form's walk, rows of `a` and columns.
int64_t wide_m_tiles(const F8Call& c) { return (c.a->rows + F8WideCfg::TM - 1) / F8WideCfg::TM; }
int64_t wide_n_tiles(const F8Call& c) {
  const int64_t columns = c.gated ? 128 : F8WideCfg::TN;
  return (c.w->rows + columns - 1) / columns;
}

template <int OUT, int ACT, bool ROWS_W>
struct Wide {
  using C = F8WideCfg;
  static constexpr auto kern = attn_res_f8_wide_kernel<OUT, ACT, ROWS_W>;

  // Pairs that the device holds at once.
  static cudaError_t resident(const F8Call& c, int* pairs) {
    static std::atomic<uint64_t> enabled{0};
    static std::atomic<int> known[64];
    *pairs = known[c.device].load(std::memory_order_acquire);
    if (*pairs != 0) return cudaSuccess;
    cudaError_t e = allow_smem(kern, C::SMEM, c.device, enabled);
    const Attributes l(dim3(2, 1, 1), C::THREADS, C::SMEM, 2, c.stream);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(pairs, kern, &l.cfg);
    if (e != cudaSuccess) return e;
    if (*pairs < 1) return cudaErrorInvalidConfiguration;
    known[c.device].store(*pairs, std::memory_order_release);
    return cudaSuccess;
  }
  static cudaError_t launch(const F8Call& c) {
    int pairs;
    cudaError_t e = resident(c, &pairs);
    F8ProductMaps maps = {};
    if (e == cudaSuccess) e = product_maps(c, 128, &maps);
    if (e != cudaSuccess) return e;
    const int64_t m_tiles = wide_m_tiles(c), n_tiles = wide_n_tiles(c), tiles = m_tiles * n_tiles;
    const TileWalk walk{(int)m_tiles, (int)n_tiles};
    Attributes l(dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs), 1, 1), C::THREADS, C::SMEM, 2, c.stream);
    return cudaLaunchKernelEx(&l.cfg, kern, params(c), walk, maps);
  }
};

template <int TN, bool GATED, bool ROWS_W>
cudaError_t launch_narrow(const F8Call& c, int split) {
  using C = F8NarrowCfg<TN, GATED, ROWS_W>;
  const auto kern = attn_res_f8_narrow_kernel<TN, GATED, ROWS_W>;
  static std::atomic<uint64_t> enabled{0};
  cudaError_t e = allow_smem(kern, C::SMEM, c.device, enabled);
  F8ProductMaps maps = {};
  if (e == cudaSuccess) e = product_maps(c, TN, &maps);
  if (e != cudaSuccess) return e;
  const int64_t n_tiles = (c.w->rows + 127) / 128, m_tiles = (c.a->rows + TN - 1) / TN;
  Attributes l(dim3((unsigned)(n_tiles * split), (unsigned)m_tiles, 1), C::THREADS, C::SMEM, (unsigned)split, c.stream);
  return cudaLaunchKernelEx(&l.cfg, kern, params(c), c.out_type, c.activation, c.pdl, maps);
}

int64_t k_blocks(const F8Call& c) { return f8_blocks(c.a->cols) + (c.a2 != nullptr ? f8_blocks(c.a2->cols) : 0); }
// Tokens of a narrow tile.
int tile_tokens(const F8Call& c) {
  const int most = c.gated ? 64 : 128;
  for (int t = 16; t < most; t *= 2)
    if (c.a->rows <= t) return t;
  return most;
}

// The choice of form and split: each one's time by a model of it, in ns, whose
// constants were fitted to 79 products (45 with block scales, 6 with row scales on
// both sides, 28 gated; 1..1024 tokens x 512..16384 columns x 512..7200; each in
// the wide form and the narrow one's splits; graph replays on GB300, inputs in L2).
// Over these the choice takes 2.4 % longer than the best form in the geometric
// mean, and 25 % at most (512 x 512 x 2048: 8.0 us in eight parts, 6.4 in six).  Over 96
// others, drawn at random (1..1400 x 128..12000 x 256..8000, 24 of each kind): block
// scales 3.6 % (18 % at most), gated 1.6 % (17 %), row scales 0.8 % (13 %; the narrow
// form's second multiplication is not in its model), sums of two products, which
// were not fitted, 2.0 % (33 %, 872 x 324 x 3012 twice: 12.0 us in seven parts, 9.0 in six).
//
// Narrow: waves of clusters, kClusters[s] of s CTAs of which the 152 SMs hold at
// once, two CTAs an SM.  A block of K takes as long as its weights' way from L2,
// or the sums' way through registers, more of either with a second CTA beside.
//   tokens x columns x K        parts: 1     2     4     5     8    wide   (us)
//   1 x 7168 x 7168              16.0   9.5   8.6   8.0  10.2   27.6
//   128 x 7168 x 7168            30.1  18.7  16.2  15.3  21.4   29.8
//   333 x 2050 x 7200            30.9  19.1  15.8  14.7  19.2   29.6
//   512 x 16384 x 1024           27.1  36.9  52.0  66.3  93.5   15.3
//   64 x 4096 x 7168 gated       38.4  22.5  13.8  16.9  14.5   31.2
constexpr int kSms = 152;
constexpr int kClusters[kF8MaxSplit + 1] = {0, 304, 152, 97, 74, 58, 46, 39, 36};
int64_t narrow_cost(const F8Call& c, int64_t tiles, int64_t blocks, int tokens, int split) {
  const int64_t per_cta = (blocks + split - 1) / split, clusters = kClusters[split];
  const int64_t waves = (tiles + clusters - 1) / clusters;
  const bool two = (tiles - (waves - 1) * clusters) * split > kSms;
  const int64_t weights = c.gated ? 2 : 1, sums = weights * tokens;
  const int64_t one_cta = std::max<int64_t>(159 * weights, 141 + 33 * sums / 10);
  const int64_t two_ctas = std::max<int64_t>(306 * weights, 287 + 48 * sums / 10);
  int64_t t = 2320 + 21 * sums + (waves - 1) * (4380 + two_ctas * per_cta) + (two ? two_ctas : one_cta) * per_cta;
  if (split > 1) t += 270 + 13 * split * sums / 10;
  return t;
}
int64_t plan_narrow(const F8Call& c, int64_t blocks, int* split) {
  const int tokens = tile_tokens(c);
  const int64_t tiles = (c.w->rows + 127) / 128 * ((c.a->rows + tokens - 1) / tokens);
  int64_t least = narrow_cost(c, tiles, blocks, tokens, 1);
  *split = 1;
  for (int s = 2; s <= kF8MaxSplit && s <= blocks; ++s) {
    const int64_t t = narrow_cost(c, tiles, blocks, tokens, s);
    if (t < least) {
      least = t;
      *split = s;
    }
  }
  return least;
}
// Wide: waves of pairs.
int64_t wide_cost(const F8Call& c, int64_t blocks) {
  const int64_t tiles = wide_m_tiles(c) * wide_n_tiles(c);
  return 1630 + (tiles + kSms / 2 - 1) / (kSms / 2) * (3190 + (c.w->block == ATTN_RES_F8_ROWS ? 820 : 471) * blocks);
}

// Token tiles of the narrow form's grid (its y).
int64_t narrow_max_rows(const F8Call& c) { return int64_t(65535) * (c.gated ? 64 : 128); }

template <bool GATED, bool ROWS_W>
cudaError_t launch_narrow(const F8Call& c, int split) {
  switch (tile_tokens(c)) {
    case 16: return launch_narrow<16, GATED, ROWS_W>(c, split);
    case 32: return launch_narrow<32, GATED, ROWS_W>(c, split);
    case 64: return launch_narrow<64, GATED, ROWS_W>(c, split);
    default:
      if constexpr (GATED) return cudaErrorInvalidValue;
      else return launch_narrow<128, GATED, ROWS_W>(c, split);
  }
}

}  // namespace

bool f8_overrides_ok(const F8Call& c) {
  if (c.kernel < 0 || c.kernel > ATTN_RES_F8_WIDE) return false;
  if (c.kernel != ATTN_RES_F8_NARROW) return c.split == 0;
  return c.a->rows <= narrow_max_rows(c) && c.split <= kF8MaxSplit && (c.split <= 1 || c.split <= k_blocks(c));
}

bool f8_choose_form(F8Call* call) {
  F8Call& c = *call;
  if (c.kernel != ATTN_RES_F8_WIDE && c.split == 0 && c.a->rows <= narrow_max_rows(c)) {
    const int64_t blocks = k_blocks(c), narrow = plan_narrow(c, blocks, &c.split);
    if (c.kernel == 0 && narrow <= wide_cost(c, blocks)) c.kernel = ATTN_RES_F8_NARROW;
  }
  if (c.kernel == 0) c.kernel = ATTN_RES_F8_WIDE;
  return c.kernel == ATTN_RES_F8_NARROW || wide_m_tiles(c) * wide_n_tiles(c) <= INT32_MAX / 2;
}

cudaError_t launch_f8_product(const F8Call& c) {
  const bool rows = c.w->block == ATTN_RES_F8_ROWS;
  if (c.kernel == ATTN_RES_F8_NARROW) {
    if (c.gated) return launch_narrow<true, false>(c, c.split);
    return rows ? launch_narrow<false, true>(c, c.split) : launch_narrow<false, false>(c, c.split);
  }
  if (c.gated) {
    const bool silu = c.activation == ATTN_RES_SILU;
    if (c.out == nullptr)
      return silu ? Wide<kF8GatedCodes, ATTN_RES_SILU, false>::launch(c) : Wide<kF8GatedCodes, ATTN_RES_GELU, false>::launch(c);
    return silu ? Wide<kF8GatedBf16, ATTN_RES_SILU, false>::launch(c) : Wide<kF8GatedBf16, ATTN_RES_GELU, false>::launch(c);
  }
  if (c.out_type == ATTN_RES_OUT_BF16)
    return rows ? Wide<kF8OutBf16, 0, true>::launch(c) : Wide<kF8OutBf16, 0, false>::launch(c);
  return rows ? Wide<kF8OutF32, 0, true>::launch(c) : Wide<kF8OutF32, 0, false>::launch(c);
}

}  // namespace attn_res_host
