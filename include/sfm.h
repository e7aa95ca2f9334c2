/*
 * sfm.h -- C-ABI of the GB300 (sm_103a) sparse shared-KV MLA attention library.
 *
 * The library computes, for every query row and head,
 *
 *     O   = softmax(Q . K~^T . softmax_scale) . V~,      K~ = V~,  kv_n = 1, d = 512
 *     LSE = log sum exp(S - max S) + max S,              S  = Q K~^T . softmax_scale
 *
 * ("sparse_flash_mla" doc (zh), 功能说明 / 计算公式; the English doc's
 * "Function" section and the SparseAttnSharedkv README give the same formula),
 * where the attended rows K~ of one query row are the union of two sources:
 *
 *   ori_kv  a sliding window [p - ori_win_left, p + ori_win_right] cut to
 *           [0, kv_len) (ori_mask_mode 4), the causal prefix [0, p] (mode 3)
 *           or all rows (mode 0); -1 for a window side means unbounded.  With
 *           ori_topk > 0 the ori source is instead the valid entries of
 *           ori_sparse_indices inside that set (the token-wise sparse form of
 *           the kv_quant_sparse_flash_attention guide, 属性参数:
 *           sparse_block_size = 1, sparse_mode 0 / 3).
 *   cmp_kv  compressed rows; slot j is visible iff (j + 1) * cmp_ratio <=
 *           p_cmp + 1 (cmp_mask_mode 3) or always (mode 0).  HCA (cmp_topk = 0)
 *           attends every visible slot; CSA (cmp_topk > 0) the valid entries of
 *           cmp_sparse_indices (-1 = invalid, valid entries first).
 *
 * with p = kv_len - q_len + i for query row i (right-down alignment, CP切分示例)
 * and p_cmp = cmp_len * cmp_ratio + cmp_residual_kv - q_len + i (参数说明: the
 * residual recovers the cmp-side mask length; equal to p under the documented
 * contract).
 * Optional per-head fp32 sinks add exp(sink - m) to the softmax denominator
 * only; the LSE excludes them.  An empty attended set gives O = 0 and
 * LSE = -inf.
 *
 * Two-call contract ("sparse_flash_mla" doc, 功能说明 and 函数原型): first
 * sfm_metadata() builds the split-KV work plan on the device, then
 * sfm_forward() consumes it.  Both calls take the SAME sfm_params; the plan
 * carries a fingerprint of them and sfm_forward() refuses (status bit
 * SFM_STATUS_METADATA_MISMATCH, outputs zeroed) a plan made for other params.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers of the current CUDA device,
 *     except the sfm_params / sfm_tensors structs themselves, which live in
 *     host memory and are read during the call only.
 *   - The caller owns every buffer (inputs, outputs, metadata, workspace,
 *     status).  The library allocates nothing on the device and never
 *     synchronises: work is enqueued on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream) and completes in stream order.
 *   - Return value: SFM_OK or an sfm_error code for a host-side rejection
 *     (nothing is enqueued then).  Tensor VALUES are checked on the device
 *     (indices, block ids, lengths); a bad value never faults: the row is
 *     skipped and a bit is OR-ed into *status (if status != NULL).
 *   - Element types: q / out / plain KV rows are bf16 or fp16 (sfm_params.dtype).
 *     Packed KV rows are bytes (see SFM_KV_INT8_PACKED).  Indices, lengths and
 *     block tables are int32; sinks and LSE are fp32.
 */
#ifndef SFM_H
#define SFM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SFM_ABI_VERSION 4

/* A cudaStream_t, passed as an untyped pointer so this header needs no CUDA headers. */
typedef void *sfm_stream_t;

/* Layouts ("sparse_flash_mla" doc, 参数说明: layout_q / layout_kv and the
 * layout匹配关系表).  SFM_LAYOUT_PAGED is the pages' PA_BBND / PA_BSND / PA_ND:
 * (blocks, block_size, 1, row) addressed through a block table. */
enum sfm_layout { SFM_LAYOUT_BSND = 0, SFM_LAYOUT_TND = 1, SFM_LAYOUT_PAGED = 2 };

/* E4M3: index queries and keys only (sfm_index_scores). */
enum sfm_dtype { SFM_DTYPE_BF16 = 0, SFM_DTYPE_FP16 = 1, SFM_DTYPE_E4M3 = 2 };

/* KV row formats.
 *   SFM_KV_PLAIN        512 bf16/fp16 values per row (1024 bytes).
 *   SFM_KV_INT8_PACKED  kv_quant_sparse_flash_attention guide, "A2/A3 C8 NoPE"
 *                       table: bytes [0,512) int8 NoPE, then rope_head_dim
 *                       (0 or 64) bf16/fp16 rope values, then 4 fp32 scales,
 *                       one per 128-dim tile: 656 bytes (rope 64) or 528 bytes
 *                       (rope 0).  K~[d] = int8[d] * scale[d / 128] for
 *                       d < 512, followed by the rope values; V~ = K~[0:512];
 *                       q has 512 + rope_head_dim dims, out has 512.
 *   SFM_KV_FP8_PACKED   the same guide, "Ascend 950 INT8/FP8 C8 NoPE" section:
 *                       the same 528 / 656-byte rows with the 512 NoPE bytes
 *                       FLOAT8_E4M3FN values (sign, 4 exponent bits biased by
 *                       7, 3 mantissa bits, no infinity, S.1111.111 = NaN):
 *                       K~[d] = e4m3(byte d) * scale[d / 128].
 *   SFM_KV_FP8_ROWS     index rows: FLOAT8_E4M3FN values only, one fp32 scale
 *                       per row in an array of its own.  Written by
 *                       sfm_kv_store() for sfm_index_scores(); sfm_forward()
 *                       does not take it. */
enum sfm_kv_format { SFM_KV_PLAIN = 0, SFM_KV_INT8_PACKED = 1, SFM_KV_FP8_PACKED = 2, SFM_KV_FP8_ROWS = 3 };

/* How sfm_metadata sizes the split-KV chunks of a query row ("sparse_flash_mla"
 * doc, 确定性计算: deterministic results and batch invariance are the default).
 *   SFM_SPLIT_BATCH_INVARIANT  a row is cut into chunks whose size depends
 *       only on the head count and the query shape (max_seqlen_q): a row's O
 *       and LSE are bit for bit the same whatever other rows share the batch
 *       and however many there are.  Batches much smaller than one row per
 *       SM leave SMs idle (a 128-head row of 1152 positions is two work
 *       units, so 8 such rows keep 16 SMs busy).
 *   SFM_SPLIT_OCCUPANCY        where the batch-invariant plan has fewer work
 *       units than the kernel has CTAs, the chunk size is chosen from the
 *       number of query rows and the SM count as well, so the units fill the
 *       SMs; otherwise the plan is the batch-invariant one.  Results are
 *       deterministic for given params and lengths, but a row's rounding can
 *       change with the batch size. */
enum sfm_split_policy { SFM_SPLIT_BATCH_INVARIANT = 0, SFM_SPLIT_OCCUPANCY = 1 };

/* Host-side return codes. */
enum sfm_error {
    SFM_OK = 0,
    SFM_ERR_INVALID_ARG = 1,   /* a scalar out of range or a required pointer missing */
    SFM_ERR_UNSUPPORTED = 2,   /* a combination the library does not implement */
    SFM_ERR_LAYOUT = 3,        /* layout pair / stride / alignment rule broken */
    SFM_ERR_WORKSPACE = 4,     /* workspace or metadata buffer too small */
    SFM_ERR_CUDA = 5           /* a CUDA runtime call failed (launch, attribute query) */
};

/* Device status bits, OR-ed into *status by the kernels (never reset by the
 * library: the caller zeroes the word before a call it wants to inspect). */
#define SFM_STATUS_BAD_INDEX          0x01  /* an index entry >= its source length: skipped */
#define SFM_STATUS_BAD_BLOCK          0x02  /* a block id / row outside the cache: row skipped */
#define SFM_STATUS_BAD_LENGTH         0x04  /* a length above its tensor's capacity: clamped */
#define SFM_STATUS_METADATA_MISMATCH  0x08  /* metadata built for other params: outputs zeroed */
#define SFM_STATUS_WORKSPACE_OVERFLOW 0x10  /* plan needs more workspace than given: outputs zeroed */
#define SFM_STATUS_PLAN_OVERFLOW      0x20  /* plan larger than int32 counters allow: outputs zeroed */
#define SFM_STATUS_TIMEOUT            0x40  /* a kernel pipeline wait gave up (bounded spin): outputs undefined */

/* Scalar attributes shared by sfm_metadata() and sfm_forward().  Field names
 * follow the pages' parameter tables ("sparse_flash_mla" doc, 参数说明). */
typedef struct sfm_params {
    int32_t num_heads_q;       /* q_n, 1..128 */
    int32_t num_heads_kv;      /* kv_n, must be 1 */
    int32_t head_dim;          /* d of V~ and of the output, must be 512 */
    int32_t rope_head_dim;     /* packed rows only: 0 or 64 extra score dims; plain rows: 0 */
    int32_t batch_size;        /* b (> 0) */
    int32_t max_seqlen_q;      /* BSND: q_s, the q tensor's S dim; TND: max q length */
    int32_t total_q;           /* TND: q_t, rows of q; ignored for BSND */
    int32_t max_seqlen_ori_kv; /* BSND: S dim of ori_kv; TND / paged: max ori length */
    int32_t max_seqlen_cmp_kv; /* BSND: S dim of cmp_kv; TND / paged: max cmp length */
    int32_t ori_topk;          /* 0: window over ori_kv; > 0: ori_sparse_indices last dim */
    int32_t cmp_topk;          /* CSA: cmp_sparse_indices last dim (> 0); SWA / HCA: 0 */
    int32_t cmp_ratio;         /* SWA: 1; CSA / HCA: > 0 */
    int32_t ori_mask_mode;     /* 0 no mask, 3 right-down causal, 4 band (window) */
    int32_t cmp_mask_mode;     /* 0 no mask, 3 right-down causal */
    int32_t ori_win_left;      /* -1 (unbounded) or >= 0 past rows */
    int32_t ori_win_right;     /* -1 (unbounded) or >= 0 future rows */
    int32_t layout_q;          /* SFM_LAYOUT_BSND or SFM_LAYOUT_TND */
    int32_t layout_kv;         /* BSND, TND or PAGED; non-paged must equal layout_q */
    int32_t has_ori_kv;        /* must be 1 (every supported mode reads ori_kv) */
    int32_t has_cmp_kv;        /* 0: SWA; 1: CSA or HCA */
    int32_t dtype;             /* enum sfm_dtype of q, out and plain KV rows */
    int32_t kv_format;         /* enum sfm_kv_format */
    int32_t ori_block_size;    /* paged: rows per ori block, multiple of 16, <= 1024 */
    int32_t cmp_block_size;    /* paged with cmp_kv: rows per cmp block, multiple of 16, <= 1024 */
    int32_t return_lse;        /* 1: write LSE (fp32, token-major x q_n) */
    int32_t kernel_hint;       /* 0 or 2: the tensor-core kernel, which takes every supported
                                  shape (up to 128 heads, plain or packed rows; packed rows
                                  are computed with fp16 operands, bf16 q converted exactly,
                                  and rope-0 packed rows with a zero rope block, as if
                                  padded); 1 (the former CUDA-core kernel): SFM_ERR_UNSUPPORTED */
    int32_t sparse_block_size; /* ori_topk > 0 only: tokens per selected block; 0 or 1 =
                                  token-wise (each ori_sparse_indices entry is a token),
                                  2..128 (a power of two, dividing ori_block_size when
                                  paged) = block-wise: entry e selects tokens
                                  [e * sparse_block_size, (e + 1) * sparse_block_size),
                                  each still under the ori mask ([QSFA] / [SFA] 属性参数:
                                  sparse_block_size; the tokens of a block share the
                                  selection decision) */
    int32_t split_policy;      /* enum sfm_split_policy (0 = batch invariant) */
} sfm_params;

/* Device tensors of one call.  Shapes (row = one KV row of row_stride bytes):
 *   q                    BSND (b, q_s, q_n, dq) / TND (q_t, q_n, dq), dq = 512 + rope_head_dim
 *   ori_kv, cmp_kv       BSND (b, S, 1, row) / TND (t, 1, row) / PAGED (blocks, block_size, 1, row)
 *   ori_sparse_indices   (tokens, 1, ori_topk) int32, -1 = invalid (ori_topk > 0 only)
 *   cmp_sparse_indices   (tokens, 1, cmp_topk) int32, -1 = invalid (CSA only)
 *   *_block_table        (b, block_table_stride) int32 block ids (PAGED only)
 *   cu_seqlens_*         (b + 1) int32 prefix sums (TND)
 *   seqused_*            (b) int32 valid counts (seqused_ori_kv required for PAGED,
 *                        seqused_cmp_kv required for PAGED cmp_kv; each overrides the
 *                        length taken from the shape or cu_seqlens)
 *   cmp_residual_kv      (b) int32, 0 <= r < cmp_ratio (required when cmp_mask_mode = 3)
 *   sinks                (q_n) fp32 or NULL
 * Row strides are in bytes, >= the row size and a multiple of 16 (rows may be
 * padded between rows, 公共参数组); *_rows is the number of rows
 * the buffer holds (used to bounds-check every resolved row; at most
 * 2^31 - 2, SFM_ERR_UNSUPPORTED above).  Base pointers must be 16-byte
 * aligned. */
typedef struct sfm_tensors {
    const void *q;
    const void *ori_kv;
    int64_t ori_row_stride;
    int64_t ori_rows;
    const void *cmp_kv;
    int64_t cmp_row_stride;
    int64_t cmp_rows;
    const int32_t *ori_sparse_indices;
    const int32_t *cmp_sparse_indices;
    const int32_t *ori_block_table;
    int32_t ori_block_table_stride;
    const int32_t *cmp_block_table;
    int32_t cmp_block_table_stride;
    const int32_t *cu_seqlens_q;
    const int32_t *cu_seqlens_ori_kv;
    const int32_t *cu_seqlens_cmp_kv;
    const int32_t *seqused_q;
    const int32_t *seqused_ori_kv;
    const int32_t *seqused_cmp_kv;
    const int32_t *cmp_residual_kv;
    const float *sinks;
} sfm_tensors;

/* Number of int32 metadata elements sfm_metadata() writes for these params on
 * the current device (>= 1024, the pages' fixed size; larger when the number
 * of query rows or SMs needs more).  Host only, enqueues nothing. */
int sfm_metadata_size(const sfm_params *params, size_t *n_int32);

/* Device workspace bytes sfm_forward() needs for these params (split-KV
 * partial results; 0 when no query row is split).  Host only. */
int sfm_workspace_size(const sfm_params *params, size_t *bytes);

/* "sparse_flash_mla_metadata": enqueue the device-side planner.  It reads the
 * length tensors of `lengths` (cu_seqlens_*, seqused_*, cmp_residual_kv; other
 * fields are ignored and may be NULL), computes every query row's attended-row
 * count, cuts it into equal splits of at most a fixed size (by default a
 * function of that row's own count and the params only, so a row's result
 * does not depend on the rest of the batch: 确定性计算 / batch invariance;
 * see sfm_params.split_policy) and balances the splits over the SMs.
 * metadata: device int32[metadata_n], 16-byte aligned (SFM_ERR_LAYOUT
 * otherwise), metadata_n >= sfm_metadata_size().
 * Ordering: the planner is launched as a programmatic dependent of the kernel
 * before it in the stream and reads the length tensors before waiting for
 * that kernel to finish (it waits before writing `metadata`).  The kernels
 * of this library never write length tensors, except for sfm_index_scores(),
 * whose `visible` may be one: it is in place before that kernel's CTAs end.
 * Copies and ordinary kernels finish before the planner starts; a kernel of the caller's that triggers its
 * dependents early (griddepcontrol.launch_dependents) must not write the
 * length tensors after that trigger. */
int sfm_metadata(const sfm_params *params, const sfm_tensors *lengths, int32_t *metadata, size_t metadata_n,
                 sfm_stream_t stream);

/* "sparse_flash_mla": enqueue the attention for every query row.
 * out: device, q's token-major layout with 512 dims per head, dtype of q.
 * lse: device fp32 (tokens x q_n), required iff params->return_lse (NULL
 *      otherwise; replaces the pages' scalar placeholder).
 * workspace: device, >= sfm_workspace_size() bytes, 256-byte aligned.
 * status: device int32 or NULL (see SFM_STATUS_*).
 * Deterministic: the same inputs give bitwise the same outputs. */
int sfm_forward(const sfm_params *params, const sfm_tensors *inputs, const int32_t *metadata, size_t metadata_n,
                float softmax_scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                int32_t *status, sfm_stream_t stream);

/* Size of the fixed device workspace used by sfm_forward_noalloc(): 32 MiB. */
#define SFM_NOALLOC_WORKSPACE_BYTES ((size_t)32 << 20)

/* sfm_forward() for callers that cannot allocate device memory.  The pages
 * have no counterpart to this entry point; it exists because some callers of
 * this library cannot call cudaMalloc when they run attention -- a graph
 * replayed with its memory frozen, a plug-in whose host framework owns every
 * allocation, a latency-critical path that must not allocate -- yet
 * sfm_forward() needs sfm_workspace_size() bytes of scratch for split-KV
 * partial results.
 *
 * Same arguments and behaviour as sfm_forward() minus the workspace: the
 * scratch comes from a fixed SFM_NOALLOC_WORKSPACE_BYTES device array that is
 * part of the library's module (every GPU that loads the module keeps it
 * until the process exits).  Nothing is allocated by this call: no cudaMalloc,
 * no cudaFree, no allocating library routine.  The caller still owns and
 * passes the inputs, the metadata, out, lse and status.
 *   - Returns SFM_ERR_WORKSPACE, enqueuing nothing, when these params need
 *     more than SFM_NOALLOC_WORKSPACE_BYTES of workspace.
 *   - Each call that needs scratch looks up the array's device address on
 *     the current device (cudaGetSymbolAddress, which allocates nothing); the
 *     first such call on a device loads the module, so make it before any
 *     stream capture.  The address is not cached, so calls made after a
 *     device reset use the array of the re-loaded module.
 *   - All calls on a device share the array and it keeps the last call's
 *     contents: calls whose kernels may overlap on the GPU (unordered
 *     streams) race on it.  Every scratch word is written before it is read
 *     within a call, so nothing needs clearing between calls. */
int sfm_forward_noalloc(const sfm_params *params, const sfm_tensors *inputs, const int32_t *metadata,
                        size_t metadata_n, float softmax_scale, void *out, float *lse, int32_t *status,
                        sfm_stream_t stream);

/* Test hook: sfm_forward() (same arguments, same kernels, same outputs)
 * that also records every KV row the attention kernel's resolver hands to
 * its copy warps, so the attended sets of the kernel that computes O can be
 * compared exactly with a reference.  For query row t and attended position
 * k (ori positions first, then cmp, in index order; k < cap):
 *   rows[t * cap + k] = -1                       the entry is skipped (masked,
 *                                                 invalid or out of range),
 *                     = r (>= 0)                 row r of the ori_kv buffer,
 *                     = (int32_t)(r | 1u << 31)  row r of the cmp_kv buffer,
 * where r counts rows of row_stride bytes from the buffer's base (for PAGED
 * caches: block id * block_size + offset, after the block table).
 * counts[t] = attended positions of row t (clamped to cap); rows with no
 * position and entries at k >= counts[t] are left as the caller filled them
 * (fill counts with 0).  Positions at or beyond cap are not recorded and set
 * SFM_STATUS_BAD_LENGTH.  rows / counts: device int32, caller-owned. */
int sfm_debug_attended(const sfm_params *params, const sfm_tensors *inputs, const int32_t *metadata,
                       size_t metadata_n, float softmax_scale, void *out, float *lse, void *workspace,
                       size_t workspace_bytes, int32_t *rows, int64_t cap, int32_t *counts, int32_t *status,
                       sfm_stream_t stream);

/* Optional instrumentation for benchmarks: with both handles non-NULL (two
 * cudaEvent_t of the current device), every following sfm_forward() records
 * `begin` on its stream right before its main attention kernel and `end`
 * right after it, so the caller can time that kernel alone with
 * cudaEventElapsedTime.  (NULL, NULL) turns it off.  Process-wide setting,
 * not synchronised: set it from the thread that calls sfm_forward(). */
int sfm_set_profile_events(void *begin, void *end);

/* ---------------------------------------------------------------------------
 * Around the attention: rotary positions, the rows of the caches, and the
 * scores and selection that make sparse indices.
 *
 * The conventions above hold for these entry points too: device pointers of
 * the current device, caller-owned buffers, no allocation, no
 * synchronisation, work in stream order, SFM_ERR_* for what the host can see
 * and status bits for tensor values.  Results are deterministic.  A call with
 * no rows (tokens, rows or total_q of 0) enqueues nothing and returns SFM_OK.
 * ------------------------------------------------------------------------- */

/* Which values of a head form the rotated pairs: (2i, 2i + 1), or
 * (i, i + rope_dim / 2) ("half"). */
enum sfm_rope_layout { SFM_ROPE_INTERLEAVED = 0, SFM_ROPE_HALF = 1 };

/* How sfm_rope_frequencies() stretches the positions of a long context by
 * `factor` (>= 1):
 *   NONE    f_i = base^(-2i / rope_dim)
 *   LINEAR  f_i / factor
 *   NTK     base replaced by base * factor^(rope_dim / (rope_dim - 2)):
 *           the slowest pair slows down by factor, the fastest not at all
 *   YARN    pairs that turn more than beta_fast times within
 *           original_max_position keep f_i, those that turn fewer than
 *           beta_slow times get f_i / factor, a linear ramp over the pair
 *           index between; the amplitude is 0.1 ln(factor) + 1. */
enum sfm_rope_scaling { SFM_ROPE_SCALING_NONE = 0, SFM_ROPE_SCALING_LINEAR = 1, SFM_ROPE_SCALING_NTK = 2,
                        SFM_ROPE_SCALING_YARN = 3 };

typedef struct sfm_rope_spec {
    int32_t rope_dim;               /* even, > 0 (NTK: > 2) */
    int32_t scaling;                /* enum sfm_rope_scaling */
    double base;                    /* > 1 */
    double factor;                  /* >= 1; NONE ignores it */
    double beta_fast, beta_slow;    /* YARN: beta_fast > beta_slow > 0 */
    int32_t original_max_position;  /* YARN: > 0 */
    int32_t reserved;               /* 0 */
} sfm_rope_spec;

/* Angles per position in radians (HOST array of rope_dim / 2 doubles) and the
 * amplitude (HOST) of the rotated values.  Host only, needs no GPU. */
int sfm_rope_frequencies(const sfm_rope_spec *spec, double *inv_freq, float *amplitude);

/* sfm_rope(): strides are in elements. */
typedef struct sfm_rope_params {
    int32_t tokens, heads;          /* >= 0, 1.. */
    int32_t head_dim;               /* values per head, 1..4096 */
    int32_t rope_dim, rope_offset;  /* the rotated values [rope_offset, rope_offset + rope_dim), rope_dim even */
    int32_t rope_layout;            /* enum sfm_rope_layout */
    int32_t inverse;                /* 1: the transpose of the forward map */
    int32_t dtype;                  /* enum sfm_dtype of x and y: BF16 or FP16 */
    float amplitude;                /* finite */
    int32_t reserved;               /* 0 */
    int64_t x_token_stride, x_head_stride, y_token_stride, y_head_stride;
} sfm_rope_params;

/* Rotary positions.  For every pair (a, b) of the rotated part and its angle
 * t = position * inv_freq[i]:
 *     a' = amplitude (a cos t - b sin t),   b' = amplitude (b cos t + a sin t);
 * inverse = 1 changes the sign of t, which is the forward map's transpose: it
 * gives the gradient of x from the gradient of y, and for amplitude 1 it
 * undoes the rotation (of an attention output whose values carried positions).
 * x, y: tokens x heads x head_dim; y == x rotates in place (same strides) and
 * touches the rotated part only, otherwise every value of y is written and the
 * two must not overlap.  positions: (tokens) int32, any sign.  inv_freq:
 * DEVICE array of rope_dim / 2 doubles, |inv_freq| < 2^53.  The angle is reduced
 * to one turn in integers, to 2^-31 of a turn at every position, and then rounded
 * to fp32. */
int sfm_rope(const sfm_rope_params *params, const void *x, const int32_t *positions, const double *inv_freq, void *y,
             sfm_stream_t stream);

/* sfm_kv_store(): x_*_stride in elements (multiples of 8), row_stride in bytes. */
typedef struct sfm_store_params {
    int32_t tokens, heads;          /* rows of x: tokens x heads */
    int32_t head_dim;               /* values per row of x: PLAIN and FP8_ROWS a multiple of 16 up to 512;
                                       packed: 512 or 576 (512 NoPE values, then 64 rope values) */
    int32_t dtype;                  /* enum sfm_dtype of x (and of PLAIN rows / packed rope parts): BF16 or FP16 */
    int32_t kv_format;              /* enum sfm_kv_format of the cache rows */
    int32_t norm;                   /* 1: RMS norm over the row's first min(head_dim, 512) values */
    float norm_eps;                 /* >= 0, finite */
    int32_t rope_dim;               /* 0: no rotation; else a multiple of 16 */
    int32_t rope_offset;            /* a multiple of 8 */
    int32_t rope_layout;            /* enum sfm_rope_layout */
    float amplitude;                /* of the rotated values */
    int32_t reserved;               /* 0 */
    int64_t x_token_stride, x_head_stride;
    int64_t row_stride;             /* bytes between cache rows: >= the row, a multiple of 16 */
    int64_t rows;                   /* rows the cache (and `scales`) holds */
} sfm_store_params;

/* Write rows into a cache in the format sfm_forward() (PLAIN and packed rows)
 * or sfm_index_scores() (PLAIN and FP8_ROWS) reads.  Per row, in fp32:
 *     v = x / sqrt(mean(x^2) + eps) * norm_weight      (norm; over the first min(head_dim, 512) values)
 *     v rotated at the token's position as in sfm_rope  (rope_dim > 0)
 * then rounded to the format: PLAIN to dtype; the others per tile (packed:
 * 128 values, FP8_ROWS: the row)
 *     scale = max(max |v| / M, 2^-126),   code = round(v / scale),   M = 127 (int8) or 448 (E4M3),
 * to nearest, ties to even, both quotients too, so that values which are
 * neither normed nor rotated have the codes that these two lines give in fp32;
 * packed rope values (512..575) are rounded to dtype.  A NaN anywhere in a tile
 * makes its scale NaN.
 *   slots    (tokens) int32 or NULL (identity): head h of token t goes to cache
 *            row slots[t] * heads + h.  A negative slot writes nothing (padding).
 *            A slot of whose rows one lies outside the cache writes none of
 *            them and sets SFM_STATUS_BAD_BLOCK.  Two tokens of one call must
 *            not name the same slot: each 16-byte piece of that row is then one
 *            of the two.  Rows no slot names are left as they were.
 *   norm_weight  (min(head_dim, 512)) fp32 or NULL (ones)
 *   positions, inv_freq  as in sfm_rope (NULL without rotation)
 *   scales   (rows) fp32, FP8_ROWS only
 * x and cache are 16-byte aligned. */
int sfm_kv_store(const sfm_store_params *params, const void *x, const float *norm_weight, const int32_t *positions,
                 const double *inv_freq, const int32_t *slots, void *cache, float *scales, int32_t *status,
                 sfm_stream_t stream);

typedef struct sfm_index_params {
    int32_t num_heads;          /* index heads, 1..128 */
    int32_t index_dim;          /* 128 */
    int32_t batch_size;         /* b (> 0) */
    int32_t max_seqlen_q;       /* BSND: q_s; TND: max q length, or any bound above it */
    int32_t total_q;            /* TND: rows of q; ignored for BSND */
    int32_t max_seqlen_kv;      /* columns of the scores, at most 2^31 - 257; BSND: S dim of k; TND / paged: max key count */
    int32_t cmp_ratio;          /* tokens per key (1: one key per token) */
    int32_t mask_mode;          /* 0 no mask, 3 right-down causal */
    int32_t layout_q;           /* SFM_LAYOUT_BSND or SFM_LAYOUT_TND */
    int32_t layout_kv;          /* BSND, TND or PAGED; non-paged must equal layout_q */
    int32_t dtype;              /* of q and k: BF16, FP16 or E4M3 */
    int32_t block_size;         /* paged: rows per block, multiple of 16, <= 1024 */
} sfm_index_params;

/*   q              BSND (b, q_s, num_heads, 128) / TND (q_t, num_heads, 128), 16-byte aligned
 *   k              BSND (b, S, row) / TND (t, row) / PAGED (blocks, block_size, row), 16-byte aligned;
 *                  k_row_stride bytes apart (multiple of 16), k_rows rows in all
 *   k_scales       (k_rows) fp32 or NULL (ones), >= 0
 *   weights        (tokens, num_heads) fp32.  Quantised queries come with a scale
 *                  per token and head (sfm_kv_store writes them beside E4M3
 *                  rows), which this call does not take: multiply it into the
 *                  head's weight, w s max(0, q.k) = w max(0, (s q).k) for s >= 0
 *   the length tensors as in sfm_tensors (seqused_kv required for PAGED;
 *   cmp_residual_kv required for mask mode 3 with cmp_ratio > 1) */
typedef struct sfm_index_tensors {
    const void *q;
    const void *k;
    int64_t k_row_stride;
    int64_t k_rows;
    const float *k_scales;
    const float *weights;
    const int32_t *block_table;
    int32_t block_table_stride;
    const int32_t *cu_seqlens_q;
    const int32_t *cu_seqlens_kv;
    const int32_t *seqused_q;
    const int32_t *seqused_kv;
    const int32_t *cmp_residual_kv;
} sfm_index_tensors;

/* The cheap score that picks what a query attends to:
 *     scores[t][j] = sum_h weights[t][h] * max(0, k_scales[j] * (q[t][h] . k[j])),   j < visible(t)
 *     scores[t][j] = -inf                                                            visible(t) <= j < max_seqlen_kv
 * with visible(t) = the keys of t's sequence under the compressed source's
 * mask of sfm_forward: j is visible iff (j + 1) * cmp_ratio <= p + 1,
 * p = len * cmp_ratio + residual - q_len + i (mode 3), or always (mode 0).
 * Products are exact, sums are in fp32.  A key whose block id is outside the
 * cache scores -inf and sets SFM_STATUS_BAD_BLOCK (as does one behind the
 * cache's last row, with up to three neighbours).  Rows of q at or beyond
 * seqused_q score -inf everywhere; rows behind the last sequence (TND), and
 * those of a sequence beyond max_seqlen_q (SFM_STATUS_BAD_LENGTH), are left as
 * they were.
 * scores: device fp32, score_stride (>= max_seqlen_kv) elements apart.
 * visible: device int32 (tokens) or NULL: visible(t). */
int sfm_index_scores(const sfm_index_params *params, const sfm_index_tensors *tensors, float *scores,
                     int64_t score_stride, int32_t *visible, int32_t *status, sfm_stream_t stream);

typedef struct sfm_topk_params {
    int32_t rows;               /* >= 0 */
    int32_t n;                  /* scores per row, > 0 */
    int32_t k;                  /* indices per row, > 0 */
    int32_t block_size;         /* scores per selected block: 1 or a power of two <= 128 */
    int32_t first_blocks;       /* blocks at the row's start that are always selected */
    int32_t last_blocks;        /* blocks at the row's end that are always selected; first + last <= k */
    int64_t score_stride;       /* elements between rows, >= n */
} sfm_topk_params;

/* The k best positions (block_size 1) or blocks of every row, as the sparse
 * indices that sfm_forward() takes (cmp_sparse_indices, ori_sparse_indices
 * with sparse_block_size = block_size).  Row r has lengths[r] scores (NULL: n;
 * a length outside [0, n] is clamped and sets SFM_STATUS_BAD_LENGTH), and
 * ceil(length / block_size) blocks, the last one possibly short; a block's
 * value is its largest score.  A NaN or -inf counts as no score: a block of
 * nothing else is selected only if it is one of the row's first_blocks or
 * last_blocks.  Equal values (-0 = 0) go to the lower index.
 * indices: device int32 (rows, k): ascending, then -1 where a row has fewer. */
int sfm_topk_select(const sfm_topk_params *params, const float *scores, const int32_t *lengths, int32_t *indices,
                    int32_t *status, sfm_stream_t stream);

/* ---------------------------------------------------------------------------
 * Attention of many queries over the same rows: prompts, single tokens over a
 * cache, and trees of drafted tokens, with more kinds of scores and masks than
 * sfm_forward(); the joining of attention results over separate sets of keys;
 * and the moving of an accepted path's rows.  The conventions of the calls
 * above hold here too.
 * ------------------------------------------------------------------------- */

typedef struct sfm_dense_params {
    int32_t num_heads;          /* query heads, 1..128 */
    int32_t head_dim;           /* 512 */
    int32_t batch_size;         /* b (> 0) */
    int32_t max_seqlen_q;       /* BSND: q_s; TND: ignored */
    int32_t total_q;            /* TND: rows of q (>= 0); BSND: ignored */
    int32_t max_seqlen_kv;      /* BSND: S dim of kv (>= 0); TND (>= 0) / paged (> 0): max key count (longer sequences are cut, SFM_STATUS_BAD_LENGTH) */
    int32_t mask_mode;          /* 0 no mask, 3 right-down causal, 4 window */
    int32_t win_left;           /* mode 4: -1 (unbounded) or >= 0 past keys */
    int32_t win_right;          /* mode 4: -1 (unbounded) or >= 0 future keys */
    int32_t layout_q;           /* SFM_LAYOUT_BSND or SFM_LAYOUT_TND */
    int32_t layout_kv;          /* BSND, TND or PAGED; non-paged must equal layout_q */
    int32_t dtype;              /* of q, kv and out: BF16 or FP16 */
    int32_t block_size;         /* paged: rows per block, multiple of 16, <= 1024 */
    int32_t tree_words;         /* 0: no tree; 1..16: 64-bit words per row of tree_mask */
    int32_t split_keys;         /* 0: long key ranges are cut so that the SMs are filled, which depends on the batch;
                                   > 0 (a multiple of 128): into as few pieces of at most this many keys as there can
                                   be, as even as tiles of 128 keys allow, whatever else is in the batch.  A row's result
                                   is then bit for bit the same whatever other sequences there are.  The queries of its
                                   own sequence still have a part in its last bits: 128 consecutive (token, head) rows
                                   share a range of keys, and with a softcap of 128 or less 32 of them a form of the cap */
    int32_t zero_rest;          /* TND, rows of q that belong to no sequence: 0: left as they were; 1: O = 0; 2: LSE = -inf; 3: both */
    float softmax_scale;        /* finite, times log2 e too */
    float softcap;              /* 0: none; 2^-100 to 2^127: scores are capped */
} sfm_dense_params;

/*   q              BSND (b, q_s, num_heads, 512) / TND (q_t, num_heads, 512), dense, 16-byte aligned
 *   kv             BSND (b, S, row) / TND (t, row) / PAGED (blocks, block_size, row), 16-byte aligned; rows of 512
 *                  values, kv_row_stride bytes apart (>= 1024, multiple of 16), kv_rows rows in all
 *                  (paged: a block at least; otherwise 0, with kv NULL or not, is a source without keys)
 *   the length tensors and sinks as in sfm_tensors (seqused_kv required for PAGED; where cu_seqlens_q falls, the
 *                  length is cut to 0, SFM_STATUS_BAD_LENGTH is set and rows of q may be skipped)
 *   bias_slopes    (num_heads) fp32 or NULL
 *   prefix_lens    (b) int32 or NULL
 *   key_begin, key_end   (tokens) int32 or NULL
 *   tree_mask      (tokens, tree_words) int64, with tree_words > 0
 *   positions      (tokens) int32 in [0, 2^30), with tree_words > 0 */
typedef struct sfm_dense_tensors {
    const void *q;
    const void *kv;
    int64_t kv_row_stride;
    int64_t kv_rows;
    const int32_t *block_table;
    int32_t block_table_stride;
    const int32_t *cu_seqlens_q;
    const int32_t *cu_seqlens_kv;
    const int32_t *seqused_q;
    const int32_t *seqused_kv;
    const float *sinks;
    const float *bias_slopes;
    const int32_t *prefix_lens;
    const int32_t *key_begin;
    const int32_t *key_end;
    const int64_t *tree_mask;
    const int32_t *positions;
} sfm_dense_tensors;

/* Device workspace bytes sfm_dense_forward() needs for these params on the
 * current device (0 where no key range is cut).  Host only. */
int sfm_dense_workspace_size(const sfm_dense_params *params, size_t *bytes);

/* Attention over one source of rows, K~ = V~ = kv.  For query i of a sequence
 * of q_len queries and len keys, head h and key j:
 *     x = softmax_scale * (q[i][h] . kv[j])
 *     x = softcap * tanh(x / softcap)                       (softcap > 0)
 *     x = x - bias_slopes[h] * |pos(i) - pos(j)|            (bias_slopes)
 *     O = sum_j e^x kv[j] / (sum_j e^x + e^sinks[h]),   LSE = log sum_j e^x     (over the visible j)
 * Without a tree, pos(i) = p = len - q_len + i and pos(j) = j, and j is visible iff
 *     (j is inside the mask mode's range of p, which is [0, len) (0), [0, p] (3)
 *      or [p - win_left, p + win_right] (4), and key_begin[i] <= j < key_end[i])
 *     or j < prefix_lens[sequence].
 * key_begin / key_end are the document of a query in a packed sequence (or any
 * other range of keys), prefix_lens the keys that every query sees.
 * With a tree (tree_words > 0; neither prefix_lens nor key_begin / key_end) the
 * last q_len keys are the queries' own rows, written before, in the same order.
 * Key j < len - q_len is at pos(j) = j; key j = len - q_len + k at
 * positions[k], and query i at pos(i) = positions[i] (those of the sequence).
 * Every key of the first kind is visible, of the second those whose bit k of
 * tree_mask[i] is set (word k / 64, bit k % 64: the ancestors of token i and
 * itself; bits behind the last word count as 0); mode 4 takes away those outside [pos(i) - win_left, pos(i) + win_right].
 * A row without visible keys has O = 0 and LSE = -inf, as have rows of q at or
 * beyond seqused_q.  Keys that a row does not see have no part in it, whatever
 * they hold (NaN and infinities too); a row that sees a NaN is NaN, and what a row
 * holds that sees an infinity is not specified.  A block outside the cache is not visible and sets
 * SFM_STATUS_BAD_BLOCK.
 * out: q's layout, 16-byte aligned (fastest with 32), apart from the inputs;
 * lse: device fp32 (tokens x num_heads) or NULL; workspace:
 * device, >= sfm_dense_workspace_size() bytes, 256-byte aligned, used by one
 * call at a time.  Products are exact, sums in fp32; weights e^x are rounded to
 * dtype for the product with kv.  A capped score is off by 2^-20 of itself, and
 * with a softcap of 128 or less by 2^-21 of the softcap too. */
int sfm_dense_forward(const sfm_dense_params *params, const sfm_dense_tensors *tensors, void *out, float *lse,
                      void *workspace, size_t workspace_bytes, int32_t *status, sfm_stream_t stream);

#define SFM_MERGE_MAX_PARTS 8

typedef struct sfm_merge_params {
    int32_t tokens, heads;      /* rows: tokens x heads (>= 0, 1..) */
    int32_t head_dim;           /* a multiple of 8 */
    int32_t parts;              /* 1..SFM_MERGE_MAX_PARTS */
    int32_t dtype;              /* of outs and out: BF16 or FP16 */
    int32_t reserved;           /* 0 */
} sfm_merge_params;

/* Join attention results over separate sets of keys.  Per row, with part n's
 * output O_n and LSE_n (natural, without sinks):
 *     LSE = log sum_n e^LSE_n,   O = sum_n e^LSE_n O_n / (sum_n e^LSE_n + e^sinks[head])
 * A part with LSE_n = -inf has no keys: its O_n does not count, whatever it holds.  No keys at all
 * give O = 0 and LSE = -inf.
 * outs, lses: HOST arrays of `parts` device pointers to dense (tokens, heads,
 * head_dim), 16-byte aligned, and fp32 (tokens, heads).  sinks: fp32 (heads) or
 * NULL (the parts must then have been computed without them, or all but one).
 * out may be one of outs; lse is NULL or none of lses. */
int sfm_merge(const sfm_merge_params *params, const void *const *outs, const float *const *lses, const float *sinks,
              void *out, float *lse, sfm_stream_t stream);

typedef struct sfm_move_params {
    int32_t batch_size;         /* b (>= 0) */
    int32_t max_path;           /* entries per sequence of path (>= 0) */
    int32_t row_bytes;          /* a multiple of 16 */
    int32_t block_size;         /* paged: rows per block (> 0); 0: sequence b has rows [b max_seqlen_kv, (b + 1) max_seqlen_kv) */
    int32_t max_seqlen_kv;      /* not paged: rows per sequence */
    int32_t block_table_stride; /* paged: blocks per sequence of block_table */
    int64_t row_stride;         /* bytes between cache rows: >= row_bytes, a multiple of 16 */
    int64_t rows;               /* rows the cache holds */
} sfm_move_params;

/* Move the rows of an accepted path together: for every sequence b,
 *     row(first[b] + i) = what row(first[b] + path[b][i]) was before the call,   i = 0, 1, ...
 * up to the first negative entry of path[b].  Entries are the drafted tokens'
 * numbers along the path and grow (path[i] < path[i + 1]); one that does not
 * ends the path (SFM_STATUS_BAD_INDEX).  A row outside the sequence's blocks or
 * the cache ends it too (SFM_STATUS_BAD_BLOCK).  Rows that are not written stay.
 * Sequences must not share the rows that they move.  cache is 16-byte aligned. */
int sfm_kv_move(const sfm_move_params *params, const int32_t *path, const int32_t *first, const int32_t *block_table,
                void *cache, int32_t *status, sfm_stream_t stream);

/* Static description of an sfm_error code. */
const char *sfm_error_string(int code);

/* SFM_ABI_VERSION of the loaded library. */
int sfm_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SFM_H */
