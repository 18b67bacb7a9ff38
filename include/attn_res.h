/*
 * attn_res.h -- C ABI of the GB300-native Kimi-K3 attention-residual
 * (AttnRes) mixture.
 *
 * The operation (implementation walkthrough of vllm-ascend PR #14840 "Add
 * Kimi K3 attention residual fusion"; key source excerpts of the prhub summary
 * of vllm PR #54261 "SM100 Kimi-K3 AttnRes defaults to native CUDA"): for each
 * token row t of width H = 7168,
 *
 *   c      = bf16_rn(prefix[t] + delta[t])      (c = prefix[t] if no delta)
 *   x_i    = blocks[t, i]  for i < num_blocks,  x_S = c        (S = num_blocks)
 *   q      = rms_w * res_w
 *   l_i    = <x_i, q> / sqrt(mean(x_i^2) + eps)
 *   w      = softmax(l_0 .. l_S)
 *   acc    = sum_i w_i x_i                      (raw rows, fp32)
 *   out[t] = bf16_rn(acc * out_norm_w / sqrt(mean(acc^2) + out_eps))
 *            or bf16_rn(acc) when out_norm_w == NULL
 *   prefix[t] = c                  when delta != NULL          (in place)
 *   blocks[t, block_write_idx] = c when block_write_idx >= 0   (in place)
 *
 * All reads of a token see the values from before the call, so a write-back
 * slot may also be one of the sources (block_write_idx < num_blocks).
 *
 * Element type: every tensor is bf16, passed as a pointer to its 16-bit
 * patterns (uint16_t).  Strides are in elements.  All tensor pointers are
 * DEVICE pointers of the current CUDA device; the caller owns every buffer.
 * The library allocates no memory, keeps no per-call state and is
 * re-entrant.
 */
#ifndef ATTN_RES_H_
#define ATTN_RES_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Hidden size the kernels are built for (the Kimi-K3 width named in the
 * dispatch gate of vllm PR #54261). */
#define ATTN_RES_HIDDEN 7168
/* Largest num_blocks (same gate: 0 <= num_blocks <= 8). */
#define ATTN_RES_MAX_BLOCKS 8

typedef uint16_t attn_res_bf16_t; /* bf16 bit pattern */

typedef enum {
  ATTN_RES_OK = 0,
  ATTN_RES_EINVAL = 1,  /* a size, index, stride, eps or required pointer is invalid */
  ATTN_RES_EALIGN = 2,  /* a pointer is not 16-byte aligned or a stride is not a multiple of 8 */
  ATTN_RES_EALIAS = 3,  /* a written region overlaps another argument's region */
  ATTN_RES_ECUDA = 4,   /* the CUDA runtime reported an error (query, attribute or launch) */
  ATTN_RES_EDEVICE = 5  /* the current device is not a compute capability 10.3 GPU */
} attn_res_status_t;

/* Launch options, in attn_res_layout_t.flags. */

/* Programmatic dependent launch: the kernel may start while the previous
 * kernel of the stream is still running.  It loads the bank rows and the
 * weights first, then waits for that kernel (griddepcontrol.wait) before
 * reading prefix and delta, and lets its own dependents launch once those
 * loads are issued (the stream kernel and its staged form: once it has run
 * out of tokens).  Contract: no grid that may still be running when this
 * call's grid starts may write the bank rows it reads or the weights.  That
 * is the preceding kernel of the stream, and also any earlier one that the
 * preceding kernel lets run on -- a kernel that releases its dependents
 * before its own grid-dependency wait.  The kernels here wait before they
 * release, so in a chain of these calls only the immediately preceding
 * call counts: between a call that writes a bank slot and a later PDL call
 * that reads it, put a kernel launched without PDL (or any fully
 * stream-ordered operation), or make the reading call without the flag.
 * Placement of the wait: PDL discipline in the key source excerpts of vllm
 * PR #54261. */
#define ATTN_RES_FLAG_PDL 0x1u

/* Hidden-sharded calls only (attn_res_tp_*; attn_res and attn_res_h reject
 * it): the single-exchange form, see attn_res_tp_sums below. */
#define ATTN_RES_FLAG_TP_GRAM 0x2u

/* Tuning overrides (0 = automatic).  Results do not depend on them beyond
 * fp32 summation order.
 *   KERNEL(k): ATTN_RES_KERNEL_SPLIT -- one cluster per token row, rows held
 *              in registers (latency path for few tokens);
 *              ATTN_RES_KERNEL_STREAM -- persistent clusters that stream many
 *              tokens through a TMA-filled shared-memory ring of bank rows,
 *              prefix and delta loaded into registers one token ahead;
 *              ATTN_RES_KERNEL_STAGED -- the stream kernel with prefix and
 *              delta also in the ring, as deep as shared memory allows;
 *              ATTN_RES_KERNEL_ROW -- one CTA per token row holding the whole
 *              row in registers, no cluster (up to 2 bank rows);
 *              ATTN_RES_KERNEL_ROW_SMEM -- the same with the rows in shared
 *              memory, brought in by bulk copies (1..8 bank rows).
 *   SPLIT(k):  CTAs (one thread-block cluster) a token row is split over;
 *              split kernel 4, 7, 8, 14 or 16; stream kernel see below; the
 *              row kernels 1.
 *   STAGES(n): ring depth of the stream kernel; CTAs per SM the staged
 *              form's ring is sized for.
 *   VPT(n):    16-byte vectors per thread and row (split kernel: 1; row
 *              kernels: 4 or 7).
 * Stream kernel shapes (split, vpt, stages): (7,1,2) (7,2,2) (7,2,3) (7,4,2)
 * (4,2,2) (4,2,3) (2,4,2) (14,2,2) (2,8,2).  Unset fields default to:
 * split 2 with no bank rows (4 if VPT 2 is given, 7 for VPT 1), else 7;
 * stages 2; VPT 8 with split 2 and no bank rows, 4 with split 2 and bank
 * rows, or with split 7 and 1..5 bank rows and an output norm or 3..6 bank
 * rows from 512 token rows, else 2 -- so (7,4,2) there, (2,8,2) with no
 * bank rows, and (7,2,2) otherwise.
 * Staged shapes (split, vpt, CTAs per SM): (4,4,5) (7,4,7) (4,4,4); the
 * ring holds as many stages of the S + 1 (+1 with delta) row slices as fit,
 * and a shape whose ring cannot hold two is ATTN_RES_EINVAL for that S.
 * Without overrides: (4,4,5) for 3 bank rows, (7,4,7) for 4, (4,4,4) for 5.
 * Automatic choice (shape overrides without KERNEL keep to the split and
 * stream kernels), measured per case on GB300:
 *   T < 80, or shared bank rows below 80: the split kernel;
 *   shared bank rows (B > 1) from 80 rows: the stream kernel;
 *   otherwise, with an output norm: no bank row, the row kernel; 1 bank row,
 *   the row kernel below 512 rows and the shared-memory row kernel from
 *   512; 2, the row kernel below 4096 rows and the shared-memory one from
 *   4096; 3..5, the shared-memory row kernel below 512 rows and the staged
 *   form from 512; 6, the shared-memory row kernel below 512 rows and the
 *   stream kernel from 512; 7..8, the stream kernel;
 *   without an output norm, below 512 rows: no bank row, the split kernel;
 *   1..2, the row kernel; 3, the staged form; 4..5, the shared-memory row
 *   kernel; 6..8, the stream kernel; from 512 rows: 0..1 bank rows, the row
 *   kernel, else the stream kernel.
 * (The exact table is attn_res_launch_shape's answer.) */
#define ATTN_RES_FLAG_SPLIT(k) (((uint32_t)(k) & 0xffu) << 8)
#define ATTN_RES_FLAG_KERNEL(k) (((uint32_t)(k) & 0xfu) << 16)
#define ATTN_RES_FLAG_STAGES(n) (((uint32_t)(n) & 0xfu) << 20)
#define ATTN_RES_FLAG_VPT(n) (((uint32_t)(n) & 0xfu) << 24)
#define ATTN_RES_KERNEL_SPLIT 1
#define ATTN_RES_KERNEL_STREAM 2
#define ATTN_RES_KERNEL_GENERIC 3 /* one CTA per row, any H (see attn_res_h) */
#define ATTN_RES_KERNEL_STAGED 4  /* stream kernel with prefix and delta staged in the ring */
#define ATTN_RES_KERNEL_ROW 5     /* one CTA per token row, the whole row */
#define ATTN_RES_KERNEL_ROW_SMEM 6 /* the same with the rows in shared memory */

/* Memory layout of the tensors, in elements.  A row is H contiguous
 * elements; columns H .. stride-1 are padding that is never read or
 * written. */
typedef struct {
  int64_t prefix_row;      /* between token rows of prefix (>= H) */
  int64_t delta_row;       /* between token rows of delta (>= H; ignored if delta == NULL) */
  int64_t blocks_token;    /* between token rows of the bank (>= (capacity-1)*blocks_slot + H
                              when the call touches more than one bank row) */
  int64_t blocks_slot;     /* between slots of one token (>= H) */
  int64_t out_row;         /* between token rows of out (>= H) */
  int32_t blocks_capacity; /* slots allocated per token (blocks.shape[1]); >= num_blocks */
  uint32_t flags;          /* ATTN_RES_FLAG_* */
  int32_t blocks_group;    /* B: token rows per bank row (0 or 1: one bank row per
                              token); see "Shared bank rows" below */
} attn_res_layout_t;

/* Shared bank rows (B = layout.blocks_group > 1).  The attn_res_kernel.cu
 * excerpt of vllm PR #54261 addresses the bank at row tb / B for token row
 * tb; the pages never say what B stands for.  Here: token row t reads bank
 * row t / B (integer division), so the bank holds ceil(T / B) token rows of
 * blocks_token elements.  Several rows then share one write-back slot; it
 * ends holding c of the last row of each group (the value sequential writes
 * in token order would leave), and only that row writes it.  Because the
 * other rows of the group would read a slot that is being written,
 * 0 <= block_write_idx < num_blocks is ATTN_RES_EINVAL when B > 1; a
 * negative blocks_group is ATTN_RES_EINVAL too.  With B > 1 the stream
 * kernel is built in one shape, (7,2,2); other stream overrides are
 * ATTN_RES_EINVAL. */

/*
 * attn_res -- enqueue the AttnRes mixture for T token rows on `stream`.
 *
 *   prefix          [T, H] at prefix_row.  Read; overwritten with c when
 *                   delta != NULL.
 *   delta           [T, H] at delta_row, or NULL.
 *   blocks          bank [T, capacity, H] at (blocks_token, blocks_slot)
 *                   ([ceil(T / B), capacity, H] with shared bank rows).
 *                   Slots 0 .. num_blocks-1 are read; slot block_write_idx
 *                   (if >= 0) is overwritten with c; nothing else is touched.
 *                   May be NULL only when num_blocks == 0 and
 *                   block_write_idx == -1.
 *   num_blocks      valid bank slots S, 0 <= S <= min(8, capacity).
 *   block_write_idx -1 (no write-back) or 0 <= idx < capacity.
 *   res_w, rms_w    [H] weights (the reference's proj / qk weight and norm
 *                   weight); q = rms_w * res_w.
 *   out_norm_w      [H] output RMSNorm weight, or NULL for no output norm.
 *   eps, out_eps    finite, >= 0.
 *   out             [T, H] at out_row.
 *   T               token rows, >= 0.  T == 0 checks the scalar arguments
 *                   and returns OK; pointers and strides are not examined.
 *   layout          strides, capacity and flags (see above).  Not NULL.
 *   stream          a cudaStream_t of the current device (NULL = legacy
 *                   default stream).
 *
 * Requirements: all pointers 16-byte aligned; all strides multiples of 8;
 * the address range [ptr, ptr + extent) of each written tensor (out always,
 * prefix when delta != NULL, blocks when block_write_idx >= 0) does not
 * overlap the range of any other argument.
 *
 * Returns ATTN_RES_OK once the work is enqueued (the call is asynchronous).
 * Any other status is returned before anything is launched, and nothing is
 * written.  Faults during execution surface from later CUDA calls on the
 * stream, as for any kernel.
 */
attn_res_status_t attn_res(attn_res_bf16_t* prefix, const attn_res_bf16_t* delta,
                           attn_res_bf16_t* blocks, int num_blocks,
                           int block_write_idx, const attn_res_bf16_t* res_w,
                           const attn_res_bf16_t* rms_w,
                           const attn_res_bf16_t* out_norm_w, float eps,
                           float out_eps, attn_res_bf16_t* out, int64_t T,
                           const attn_res_layout_t* layout, void* stream);

/*
 * attn_res_h -- the same operation for any hidden size H > 0 that is a
 * multiple of 8 (one 16-byte vector); every [H]- and row-sized argument above
 * is then H elements wide and strides must be >= H.  H == ATTN_RES_HIDDEN
 * behaves exactly like attn_res.  Other widths:
 *   - H at most 16384, with bank rows or an output norm: any-width forms of
 *     the fast kernels with ceil(H / 1024) CTAs per token row (one cluster)
 *     of 1024 columns each, the last CTA owning the remainder -- below 80
 *     token rows and up to H = 8192 the split kernel (one vector per
 *     thread), else the stream kernel (the per-CTA layout of the (7,2,2)
 *     shape); KERNEL(SPLIT) or KERNEL(STREAM) force one of them; shape
 *     overrides are ATTN_RES_EINVAL;
 *   - otherwise (wider rows, or neither bank rows nor an output norm) a
 *     general kernel (one CTA of 256 threads per token row, same fp32
 *     arithmetic, the rows read three times through L2), a functional
 *     path.  ATTN_RES_FLAG_KERNEL(ATTN_RES_KERNEL_GENERIC) forces it, also at
 *     H == ATTN_RES_HIDDEN.  Forcing a fast kernel where no form of it fits
 *     the width (or the row has no exchange) is ATTN_RES_EINVAL; the row
 *     kernels and the staged form are built for H == ATTN_RES_HIDDEN only
 *     (forced at another width: ATTN_RES_EINVAL).
 * Returns ATTN_RES_EINVAL for a bad H.  (No counterpart on the pages, whose
 * kernel is built for H = 7168 only.)
 */
attn_res_status_t attn_res_h(int64_t H, attn_res_bf16_t* prefix,
                             const attn_res_bf16_t* delta, attn_res_bf16_t* blocks,
                             int num_blocks, int block_write_idx,
                             const attn_res_bf16_t* res_w, const attn_res_bf16_t* rms_w,
                             const attn_res_bf16_t* out_norm_w, float eps, float out_eps,
                             attn_res_bf16_t* out, int64_t T,
                             const attn_res_layout_t* layout, void* stream);

/*
 * Hidden-sharded (tensor-parallel) mixture.  The Kimi-K3 deployments the
 * prhub summary of vllm PR #54261 evaluates (impact section: TP8, TEP8,
 * DEP16, ...) may hold a column shard of each row per rank.  The logits need
 * full-row sums and the output norm a full-row sum of squares, so the
 * operation above splits at those two points; the caller all-reduces (sums)
 * the small float buffers between the calls:
 *
 *   attn_res_tp_sums   -> all-reduce sums [T, 2N]   (N = num_blocks + 1)
 *   attn_res_tp_sq     -> all-reduce sq [T]         (output norm only)
 *   attn_res_tp_finish
 *
 * Each rank passes its own shard: every row-sized argument (prefix, delta,
 * blocks rows, res_w, rms_w, out_norm_w, out) is the Hs columns that rank
 * owns, with the strides and layout rules of attn_res_h for width Hs (a
 * multiple of 8); H is the full hidden size (the sum of the shard widths),
 * used in mean(x^2) and mean(acc^2).  With one rank (Hs == H) the three calls
 * compute the same result as attn_res_h.  Float buffers are fp32 device
 * memory owned by the caller, 4-byte aligned; sums has sums_row >=
 * attn_res_tp_sums_width(num_blocks, gram) floats between token rows:
 * entries 0..N-1 are sum(x_i^2), N..2N-1 are <x_i, q> over the shard
 * (x_S = c).  layout->flags accepts ATTN_RES_FLAG_PDL, ATTN_RES_FLAG_TP_GRAM,
 * ATTN_RES_FLAG_KERNEL and ATTN_RES_FLAG_STAGES.  Two kernel forms, the same
 * results up to fp32 summation order:
 *   ring (ATTN_RES_KERNEL_STREAM) -- persistent CTAs (as many as fit on the
 *     device, at most T) each streaming every G-th token row's rows through
 *     a shared-memory ring filled by bulk copies (TMA), ATTN_RES_FLAG_STAGES
 *     2..4 deep (default 2); the Gram sums on warp-level tensor-core tiles;
 *   one CTA of 32..256 threads per token row (ATTN_RES_KERNEL_GENERIC).
 * Automatic: the ring from 1024 token rows when it fits in 220 KB of shared
 * memory (2 stages of num_blocks + 1 (+1 with delta) rows of Hs columns, plus
 * 4*Hs bytes and the warps' tiles for the Gram sums), else one CTA per row.
 * A forced ring that does not fit, another KERNEL value, or STAGES with
 * ATTN_RES_KERNEL_GENERIC is ATTN_RES_EINVAL; with the automatic form
 * STAGES applies only when the ring runs.  Errors as for attn_res (nothing
 * is launched unless ATTN_RES_OK is returned); a written float buffer that
 * overlaps any other argument is ATTN_RES_EALIAS.
 *
 * Single exchange (ATTN_RES_FLAG_TP_GRAM set on attn_res_tp_sums and
 * attn_res_tp_finish): attn_res_tp_sums also writes g_ij = <x_i, x_j> over
 * the shard for i < j (entries 2N.., row-major over i), and
 * attn_res_tp_finish takes sum(acc^2) = sum_i w_i^2 ss_i + 2 sum_{i<j} w_i
 * w_j g_ij from the reduced entries: one all-reduce and no attn_res_tp_sq
 * call (which rejects the flag).  Exact in real arithmetic; in fp32 the
 * output norm loses relative accuracy where the weighted rows cancel
 * (|acc| << sum_i w_i |x_i|), so the default is the two-exchange form.
 * The ring form computes the Gram products on warp-level tensor-core tiles
 * (mma.sync m16n8k16, bf16 in, fp32 accumulate; q split exactly into two
 * bf16 rows): the one dense contraction in this library, confined to this
 * opt-in form -- the mixture itself, like the pages' kernels, uses no tensor
 * cores (a bandwidth-bound mix of a few rows per token).
 */

/* Floats per token row of `sums`: 2N, plus N(N-1)/2 with gram != 0
 * (N = num_blocks + 1); -1 for num_blocks outside 0..8. */
int attn_res_tp_sums_width(int num_blocks, int gram);

/* Per-shard sums; reads prefix, delta, blocks[t, 0..num_blocks), res_w,
 * rms_w; writes sums[t, 0..attn_res_tp_sums_width(num_blocks, gram)). */
attn_res_status_t attn_res_tp_sums(int64_t Hs, const attn_res_bf16_t* prefix,
                                   const attn_res_bf16_t* delta, const attn_res_bf16_t* blocks,
                                   int num_blocks, const attn_res_bf16_t* res_w,
                                   const attn_res_bf16_t* rms_w, float* sums, int64_t sums_row,
                                   int64_t T, const attn_res_layout_t* layout, void* stream);

/* Output-norm partial: softmax from the reduced sums, acc over the shard,
 * sq[t] = sum(acc^2) over the shard.  Reads prefix, delta, blocks, sums;
 * writes sq[0..T).  sq must not be NULL. */
attn_res_status_t attn_res_tp_sq(int64_t Hs, int64_t H, const attn_res_bf16_t* prefix,
                                 const attn_res_bf16_t* delta, const attn_res_bf16_t* blocks,
                                 int num_blocks, float eps, const float* sums, int64_t sums_row,
                                 float* sq, int64_t T, const attn_res_layout_t* layout,
                                 void* stream);

/* Output and write-backs of the shard: softmax from the reduced sums, acc,
 * out (normalised with the reduced sq, or with the Gram entries under
 * ATTN_RES_FLAG_TP_GRAM, when out_norm_w != NULL; sq may be NULL otherwise),
 * prefix[t] = c when delta != NULL, blocks[t, block_write_idx] = c when
 * block_write_idx >= 0. */
attn_res_status_t attn_res_tp_finish(int64_t Hs, int64_t H, attn_res_bf16_t* prefix,
                                     const attn_res_bf16_t* delta, attn_res_bf16_t* blocks,
                                     int num_blocks, int block_write_idx,
                                     const attn_res_bf16_t* out_norm_w, float eps, float out_eps,
                                     const float* sums, int64_t sums_row, const float* sq,
                                     attn_res_bf16_t* out, int64_t T,
                                     const attn_res_layout_t* layout, void* stream);

/*
 * Microscaled rows: a row is held as 8- or 4-bit elements with a scale for
 * each group of 16 or 32 neighbours (the OCP Microscaling Formats
 * specification's MXFP8 and MXFP4, and the NVFP4 variant), the form in which
 * a projection after the mixture takes its input.  The calls below bring
 * rows into it (after a residual addition and RMSNorm, or as they are), back
 * to bf16, and multiply two such matrices.  (No counterpart on the pages,
 * whose mixture ends with a bf16 row.)
 *
 *   format            element  group  scale of a group         scale of the tensor
 *   ATTN_RES_MXFP8    e4m3     32     e8m0 (a power of two)    none
 *   ATTN_RES_MXFP4    e2m1     32     e8m0                     none
 *   ATTN_RES_NVFP4    e2m1     16     e4m3                     fp32, optional
 *
 * An element x of a group with scale s in a tensor with scale g (1 without
 * one) stands for code * s * g.  Quantisation, with TOP = 448 (e4m3) or 6
 * (e2m1), amax the group's largest |x|, rn = round to nearest, ties to even:
 *   MXFP8, MXFP4: s = the smallest power of two >= 2^-127 with
 *                 amax <= TOP * s (so nothing is clipped); code = rn(x / s);
 *   NVFP4:        s = rn_e4m3(min(448, amax / (6 g))), code = rn(x / (s g)),
 *                 0 where s g == 0, clipped to +-6 (fp32 operations, each
 *                 correctly rounded: 6 g, the two quotients and s g).
 * A group that holds a NaN or an infinity gets the scale NaN and zero
 * elements: it stands for NaN throughout.  g must be finite and > 0.
 *
 * Data: element k of row r is the byte data[r * row_bytes + k] (8 bits), or
 * the low (even k) or high (odd k) half of data[r * row_bytes + k / 2] (4
 * bits).  cols must be a multiple of 32, data 16-byte aligned and row_bytes
 * a multiple of 16; bytes past the row's last are neither read nor written.
 * Scales: tiles of 128 rows x 4 groups, 512 bytes each, row tiles outermost
 * and without gaps: the scale of row r and group j is byte
 *   ((r / 128) * ceil(groups / 4) + j / 4) * 512
 *     + (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4,
 * the order in which the tensor cores take them.  The buffer holds
 * attn_res_mx_scale_bytes(format, rows, cols) bytes, 16-byte aligned; the
 * entries past the last row and the last group are written as 0, and
 * attn_res_mx_matmul wants those past the last group to be 0.
 */
#define ATTN_RES_MXFP8 1
#define ATTN_RES_MXFP4 2
#define ATTN_RES_NVFP4 3

typedef struct {
  int32_t format;            /* ATTN_RES_MXFP8, ATTN_RES_MXFP4 or ATTN_RES_NVFP4 */
  int64_t rows, cols;        /* 0 <= rows <= 2^31 - 256; 0 < cols <= 2^30, a multiple of 32 */
  void* data;                /* element codes */
  int64_t row_bytes;         /* between rows of data */
  uint8_t* scales;           /* tiled scales */
  const float* tensor_scale; /* g: one fp32 on the device (4-byte aligned), or NULL;
                                NULL unless format is ATTN_RES_NVFP4 */
} attn_res_mx_t;

/* Bytes of the scale buffer; -1 for an unknown format, or rows or cols out of
 * the ranges above. */
int64_t attn_res_mx_scale_bytes(int format, int64_t rows, int64_t cols);

/*
 * The calls below take device pointers of the current device and enqueue on
 * `stream` as attn_res does.  They are launched so that a kernel's start-up
 * overlaps the end of a preceding kernel that lets its dependents start, and
 * touch no memory before that kernel is complete: fully stream ordered.  flags
 * is 0 or ATTN_RES_FLAG_PDL, which lets attn_res_mx_matmul read w before then
 * (the contract of that flag, with w in the place of the bank rows; the other
 * calls take the flag and do as without it).
 *
 * bf16 rows have unit inner stride, 16-byte aligned pointers and row strides
 * that are multiples of 8 elements and >= the row width.  A written range that
 * overlaps another argument's is ATTN_RES_EALIAS; the other errors are as for
 * attn_res, before any launch.  With no rows (for the product: no rows in a or
 * in w) a call checks the scalar arguments and returns OK.
 */

/* q = x [q->rows, q->cols] in q's format; writes q's data and scales. */
attn_res_status_t attn_res_mx_quantize(const attn_res_bf16_t* x, int64_t x_row,
                                       const attn_res_mx_t* q, uint32_t flags, void* stream);

/* x = the bf16 values that q stands for (element * s, then * g, in fp32,
 * rounded to bf16 once). */
attn_res_status_t attn_res_mx_dequantize(const attn_res_mx_t* q, attn_res_bf16_t* x,
                                         int64_t x_row, uint32_t flags, void* stream);

/*
 * attn_res_mx_norm -- residual addition, RMSNorm and quantisation of q->rows
 * token rows of width H = q->cols (at most 65536):
 *
 *   c = bf16_rn(prefix[t] + delta[t])   (c = prefix[t] if delta == NULL)
 *   y = c * weight / sqrt(mean(c^2) + eps)
 *   prefix[t] = c                       when delta != NULL (in place)
 *   norm_out[t] = bf16_rn(y)            when norm_out != NULL
 *   q[t] = y in q's format              (from the fp32 y)
 *
 * the mixture's current row and output norm (as attn_res with no bank rows),
 * its result in the microscaled form.  eps is finite and >= 0.  y is held to
 * fp32 accuracy for rows of any finite magnitude (squares that fp32 does not
 * hold are taken of the row times a power of two) and weights of up to 2^60
 * and from 2^-60 on (or 0); a row with an infinity or a NaN, and with eps = 0
 * a row of zeros, is what the formula makes of it.
 */
attn_res_status_t attn_res_mx_norm(attn_res_bf16_t* prefix, int64_t prefix_row,
                                   const attn_res_bf16_t* delta, int64_t delta_row,
                                   const attn_res_bf16_t* weight, float eps,
                                   attn_res_bf16_t* norm_out, int64_t norm_row,
                                   const attn_res_mx_t* q, uint32_t flags, void* stream);

/*
 * attn_res_mx_matmul -- out[m, n] = sum_k a[m, k] w[n, k], out
 * [a->rows, w->rows] bf16 at out_row, for two matrices of one format and
 * width (a->cols == w->cols); fp32 sums on the tensor cores (tcgen05, block
 * scaled), times the tensor scales, rounded to bf16 once: a result is out of
 * range only if its value is, whatever the scales.  Any number of rows on both sides.
 * Repeated calls give the same bits.
 *
 * Beside ATTN_RES_FLAG_PDL, flags takes tuning overrides (0 = automatic; the
 * results do not depend on them beyond fp32 summation order):
 *   KERNEL(k): ATTN_RES_MX_NARROW -- a CTA for 128 rows of w and up to 128 of
 *              a, K split over a cluster (few tokens, or few tiles);
 *              ATTN_RES_MX_WIDE, ATTN_RES_MX_WIDER -- persistent CTA pairs,
 *              256 rows of a and 256 or 384 of w at a time (w->rows up to
 *              2^31 - 768);
 *   SPLIT(s):  with ATTN_RES_MX_NARROW, the CTAs that share a tile's K: 1..6,
 *              at most the 128-byte blocks of a row of codes.
 * An override that cannot be met is ATTN_RES_EINVAL.
 */
#define ATTN_RES_MX_NARROW 1
#define ATTN_RES_MX_WIDE 2
#define ATTN_RES_MX_WIDER 3
attn_res_status_t attn_res_mx_matmul(const attn_res_mx_t* a, const attn_res_mx_t* w,
                                     attn_res_bf16_t* out, int64_t out_row, uint32_t flags,
                                     void* stream);

/*
 * Rows in 8 bits with scales for blocks of 128: e4m3 elements, an fp32 scale for
 * 128 of them along a row (activations and gradients) or for a block of 128 x
 * 128 (weights), the form in which a feed-forward block is run and trained in 8
 * bits.  The calls below bring rows into it, also transposed, multiply two such
 * matrices, and make the gated block's first half and its backward pass.  (No
 * counterpart on the pages.)
 *
 * An element of a group with scale s stands for code * s.  Quantisation, with
 * amax the group's largest |x|:
 *   s = max(amax / 448, 2^-126), 1 for a group of zeros;
 *   code = rn_e4m3(x / s), saturating at +-448
 * (fp32 quotients, correctly rounded; rn: to nearest, ties to even).  A group
 * that holds a NaN or an infinity gets the scale NaN and zero codes: it stands
 * for NaN throughout.  Scales that a caller makes may be any fp32 values.  So
 * attn_res_f8_quantize, to the bit; results that attn_res_f8_gated and its
 * backward make in codes come from fp32 values that carry roundings of their
 * own, and their x / s may be off by two units of its last place more.
 *
 * Data: element k of row r is the byte data[r * row_bytes + k].  Any number of
 * columns; data 16-byte aligned, row_bytes a multiple of 16 and at least cols.
 * Bytes past a row's last are neither read nor written.
 * Scales, with b = k / 128:
 *   ATTN_RES_F8_ROWS    scales[b * scales_row + r]: blocks of columns outermost,
 *                       scales_row >= rows and a multiple of 4, 16-byte aligned;
 *   ATTN_RES_F8_SQUARE  scales[(r / 128) * scales_row + b], scales_row >= the
 *                       blocks of a row, 4-byte aligned.
 * Floats between the last of a row of scales and the next row are neither read
 * nor written.  A matrix without elements (rows or cols 0) may have null
 * pointers.
 */
#define ATTN_RES_F8_ROWS 1
#define ATTN_RES_F8_SQUARE 128

typedef struct {
  int32_t block;       /* ATTN_RES_F8_ROWS or ATTN_RES_F8_SQUARE */
  int64_t rows, cols;  /* 0 .. 2^31 - 1024 each */
  void* data;          /* e4m3 codes */
  int64_t row_bytes;   /* between rows of data */
  float* scales;
  int64_t scales_row;  /* floats between rows of scales */
} attn_res_f8_t;

/* Enqueueing, flags, alignment of bf16 rows, aliasing and errors are as for the
 * microscaled calls above; all outputs of a call are disjoint from each other
 * and from its inputs.  Where nothing is to be written, a call checks the scalar
 * arguments and returns OK. */

/* q = x [q->rows, q->cols], and, if qt is not NULL, qt = the transposed x
 * [q->cols, q->rows], quantised by itself: with ATTN_RES_F8_ROWS in groups along
 * the columns of x.  Both have one kind of block. */
attn_res_status_t attn_res_f8_quantize(const attn_res_bf16_t* x, int64_t x_row,
                                       const attn_res_f8_t* q, const attn_res_f8_t* qt,
                                       uint32_t flags, void* stream);

/* x = the bf16 values that q stands for (code * s in fp32, rounded once). */
attn_res_status_t attn_res_f8_dequantize(const attn_res_f8_t* q, attn_res_bf16_t* x,
                                         int64_t x_row, uint32_t flags, void* stream);

/*
 * attn_res_f8_matmul -- out[m, n] = sum_k a[m, k] w[n, k] for a with row scales
 * and w with row or block scales, out [a->rows, w->rows]; with a2 and w2 (both
 * or neither; rows and kinds of block as a's and w's, a width of their own) plus
 * their product: the gradient of what two projections share, say.  Per block of
 * 128 columns the codes' products are summed on the tensor cores (tcgen05, fp32)
 * and then multiplied by the fp32 product of the two scales; the blocks' sums
 * are added in fp32, and the result is rounded once.  (A product of scales below
 * 2^-126 has fewer bits and is 0 below 2^-149; one above 2^128 is infinite, and
 * NaN comes of it where a block's sum is 0.)  Repeated calls give the same bits.
 *
 * out_type: ATTN_RES_OUT_BF16, ATTN_RES_OUT_F32, or ATTN_RES_OUT_F32_ADD, which
 * adds to the fp32 rows that are there.  fp32 rows: 16-byte aligned, out_row a
 * multiple of 4.  A width of 0 makes zeros.
 *
 * ATTN_RES_FLAG_PDL lets the narrow form read w and w2 before the preceding
 * kernel is complete (the contract of that flag, with them in the place of the
 * bank rows); elsewhere it does nothing.  Beside it, flags takes tuning overrides
 * (0 = automatic; the results do not depend on them beyond fp32 summation order):
 *   KERNEL(k): ATTN_RES_F8_NARROW -- a CTA for 128 rows of w and up to 128 of a
 *              (the gated block: 64), K split over a cluster;
 *              ATTN_RES_F8_WIDE -- persistent CTA pairs, 256 rows of a and 256
 *              of w at a time;
 *   SPLIT(s):  with ATTN_RES_F8_NARROW, the CTAs that share a tile's K: 1..8, at
 *              most the 128-column blocks of K.
 * An override that cannot be met is ATTN_RES_EINVAL.
 */
#define ATTN_RES_F8_NARROW 1
#define ATTN_RES_F8_WIDE 2
#define ATTN_RES_OUT_BF16 0
#define ATTN_RES_OUT_F32 1
#define ATTN_RES_OUT_F32_ADD 2
attn_res_status_t attn_res_f8_matmul(const attn_res_f8_t* a, const attn_res_f8_t* w,
                                     const attn_res_f8_t* a2, const attn_res_f8_t* w2, void* out,
                                     int64_t out_row, int out_type, uint32_t flags, void* stream);

/*
 * attn_res_f8_gated -- the first half of a gated feed-forward block, both
 * projections in one kernel:
 *
 *   g = x gate^T,  u = x up^T,  h = act(g) * u       [x->rows, gate->rows]
 *
 * x with row scales, gate and up of one shape with block scales; products as
 * attn_res_f8_matmul's, h in fp32 from the fp32 sums.  The result is h in codes
 * with row scales or, with h NULL, h_rows in bf16.  save_g and save_u (both or
 * neither) receive g and u in codes with row scales: the checkpoint that
 * attn_res_f8_gated_backward takes.
 * activation: ATTN_RES_SILU, act(g) = g / (1 + exp(-g)), or ATTN_RES_GELU, the
 * tanh form g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2, as g / (1 +
 * exp(-z)) too.  (Fast exponential: act(g) to 2^-16 of itself where it is small
 * -- GELU's, whose z carries fp32 roundings of its own, to 2^-14 --, to a few
 * 2^-23 elsewhere; 0 where exp(-z) overflows, below z = -88.7.  The backward pass
 * has 1 / (1 + exp(-z)) of its fp32 z to a few 2^-23 throughout.)
 */
#define ATTN_RES_SILU 1
#define ATTN_RES_GELU 2
attn_res_status_t attn_res_f8_gated(const attn_res_f8_t* x, const attn_res_f8_t* gate,
                                    const attn_res_f8_t* up, int activation,
                                    const attn_res_f8_t* h, attn_res_bf16_t* h_rows, int64_t h_row,
                                    const attn_res_f8_t* save_g, const attn_res_f8_t* save_u,
                                    uint32_t flags, void* stream);

/*
 * attn_res_f8_gated_backward -- from the gradient dh [T, F] of h and the saved g
 * and u (row scales), in fp32:
 *
 *   dg = dh * u * act'(g),  du = dh * act(g),  h = act(g) * u
 *
 * dg and du in codes with row scales, for the input's gradient dx = dg gate + du
 * up (attn_res_f8_matmul of them and the transposed weights); and, if not NULL
 * (all three or none), the transposed dg_t, du_t and h_t [F, T], quantised by
 * themselves in groups along the tokens, for the gradients of the weights.
 * Rows of dh, and of g's and u's scales, lie less than 2^40 bytes apart.
 */
attn_res_status_t attn_res_f8_gated_backward(const attn_res_bf16_t* dh, int64_t dh_row,
                                             const attn_res_f8_t* g, const attn_res_f8_t* u,
                                             int activation, const attn_res_f8_t* dg,
                                             const attn_res_f8_t* du, const attn_res_f8_t* dg_t,
                                             const attn_res_f8_t* du_t, const attn_res_f8_t* h_t,
                                             uint32_t flags, void* stream);

/* Static text for a status code. */
const char* attn_res_status_string(attn_res_status_t status);

/* ATTN_RES_HIDDEN, for callers that load the library dynamically. */
int attn_res_hidden_size(void);

/* ATTN_RES_MAX_BLOCKS. */
int attn_res_max_blocks(void);

/*
 * attn_res_launch_shape -- the launch attn_res would make for T rows with
 * num_blocks sources, a delta row or not, output norm on/off and the given
 * flags: the kernel (ATTN_RES_KERNEL_*), CTAs per token row (`split`), ring
 * depth (`stages`: the stream kernel's STAGES; the staged form's depth,
 * which follows from the rows of a stage; 0 for the other kernels), threads
 * per CTA, CTAs in the grid (0 for the persistent stream kernel and its
 * staged form, whose grid is as many clusters as fit on the device, at most
 * T) and the thread-block cluster size (1 when the CTAs of a row never
 * exchange sums -- no bank rows and no output norm -- and for the row and
 * general kernels, which hold a row in one CTA).  Any output pointer may be
 * NULL.  Pure host computation, no CUDA call.  Returns ATTN_RES_EINVAL for
 * T < 0, num_blocks outside 0..8 or an unsupported override.
 */
attn_res_status_t attn_res_launch_shape(int64_t T, int num_blocks, int has_delta,
                                        int has_out_norm, uint32_t flags,
                                        int* kernel, int* split, int* stages,
                                        int* threads_per_cta, int64_t* ctas,
                                        int* cluster);

/*
 * attn_res_device_status -- error bits the kernels recorded on the current
 * device since the last clear (0 = none).  Bit 0: a wait for a shared-memory
 * stage of row data timed out; bit 1: a wait for the partial sums of another
 * CTA of the cluster timed out.  The kernel then finished without waiting
 * further and that call's outputs are not valid.  With `clear` != 0 the word is reset.  Synchronous
 * (cudaMemcpy); a diagnostic, not for the hot path.
 */
attn_res_status_t attn_res_device_status(unsigned int* bits, int clear);

/*
 * attn_res_selftest_wait_timeout -- exercise the kernels' time-out path on
 * the current device: three warps wait at once, each with one of the bounded
 * waits that the kernels use, on an mbarrier that nothing ever completes;
 * after about `limit_us` microseconds (1 .. 1 000 000) they give up, and when
 * all have, bit 0 of the device status word is set.  Synchronous: returns after the kernel
 * finished, with the status word (not cleared) in *bits.  A diagnostic for
 * tests; it does not touch any caller buffer.
 */
attn_res_status_t attn_res_selftest_wait_timeout(unsigned int limit_us, unsigned int* bits);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_RES_H_ */
