/*
 * qmm.h -- C ABI of the affine group-quantized matmul library (libqmm.so, gfx950).
 *
 * Operation:  y = x . dequant(W)^T with w[n,k] = s[n,g] * q[n,k] + b[n,g], g = k / group_size.
 * (huggingface/transformers issue 47331, section "Root cause": the kernel call
 *  affine_qmm_t(x, w_packed, scales, biases, group_size, bits) returns y of shape
 *  x.shape[:-1] + [N]; "Fix": a batched input must give the same rows as the same input
 *  flattened to 2D.)
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers.  Descriptors are HOST pointers, read during the
 *     call only.  The caller owns all memory; the library allocates no device memory.  Its
 *     host state is a thread-local error message and, per device, cached launch settings
 *     (kernel LDS limits, occupancies) and the address of its one static device array (the
 *     workspace of qmm_qmv_argmax_noalloc), guarded so that calls from several threads are
 *     safe.
 *   - Strides are in elements.  A tensor pointer points at the view's first element (a view's
 *     storage offset is already applied).
 *   - `stream` is a hipStream_t of the current device (NULL = its default stream).  Work is
 *     enqueued asynchronously; the library never synchronizes.
 *   - Every argument is validated before anything is launched; on error nothing is written,
 *     the call returns a negative QMM_ERR_* code and qmm_last_error() describes it
 *     (candle pitfall page "Metal 上批量 matmul 结果不对", section 现象: a structured error that
 *     names the layout is preferred over a silently wrong result).
 *   - dtype of x, scales, biases and y is one and the same: QMM_BF16 or QMM_FP16.
 *   - bits in {2,3,4,5,6,8}; group_size in {32,64,128}; K % group_size == 0.
 *   - Codes are a little-endian bitstream per weight row: code k of row n sits at bit k*bits
 *     of the row's stream of uint32 words, continuing into the next word when it straddles
 *     one (Metal Kernel Bits=8 final report, section 3.1, gives the 4- and 8-bit cases).
 */
#ifndef QMM_H
#define QMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QMM_ABI_VERSION 1
#define QMM_MAX_DIMS 8
/* Collapsed activation rows up to this count use the decode (qmv) kernels. */
#define QMM_DECODE_MAX_ROWS 32

typedef enum { QMM_BF16 = 1, QMM_FP16 = 2 } qmm_dtype_t;

/* Return codes. */
enum {
  QMM_OK = 0,
  QMM_ERR_NULL = -1,        /* a required pointer is NULL                                  */
  QMM_ERR_UNSUPPORTED = -2, /* bits / group_size / dtype / flag not supported              */
  QMM_ERR_SHAPE = -3,       /* shapes disagree (K, N, y shape, K % group_size, qmv rows)    */
  QMM_ERR_LAYOUT = -4,      /* x batch dims cannot be expressed as <= 2 strided levels, a   */
                            /* negative stride, x last-dim stride != 1, or y not dense      */
  QMM_ERR_ALIGN = -5,       /* pointer / stride / K alignment that the kernels require      */
  QMM_ERR_HIP = -6          /* the HIP runtime reported an error at launch                  */
};

/* Flags for qmv / qmm_t. */
enum {
  /* Do not fold the batch dims: launch one grid slice per batch element, each of which
   * re-reads the whole weight.  Results are bitwise identical to the folded launch; it
   * exists to time the per-batch-element path against the folded one
   * (transformers issue 47331 summary page, 原因分析: 60 ms vs 2.2 ms for [32,1,K]). */
  QMM_FLAG_FORCE_STRIDED = 1u << 0
};

typedef struct {
  int32_t ndim;                   /* 1 .. QMM_MAX_DIMS                                    */
  int64_t shape[QMM_MAX_DIMS];
  int64_t stride[QMM_MAX_DIMS];   /* elements, >= 0                                        */
} qmm_tensor_desc_t;

typedef struct {
  const uint32_t* w_packed; /* device, row n at w_packed + n * w_row_stride                 */
  int64_t w_row_stride;     /* uint32 words, >= K*bits/32; the matmul needs a multiple of 4 */
  const void* scales;       /* device, [N, sb_row_stride] of dtype                          */
  const void* biases;       /* device, [N, sb_row_stride] of dtype                          */
  int64_t sb_row_stride;    /* elements, >= K / group_size                                  */
  int64_t N;                /* output features (weight rows)                                */
  int64_t K;                /* input features                                               */
  int32_t group_size;
  int32_t bits;
  int32_t dtype;            /* qmm_dtype_t                                                  */
} qmm_weight_desc_t;

/* How a call is executed; filled by qmm_plan (host only, no GPU needed).
 * Row r (0 <= r < rows_per_batch) of grid batch z reads x at
 *   x + z*batch_stride + (r / seg_rows)*seg_stride + (r % seg_rows)*row_stride
 * and writes y at y + (z*rows_per_batch + r)*N. */
typedef struct {
  int64_t rows;            /* total collapsed activation rows M                          */
  int64_t batches;         /* grid batch slices (1 unless QMM_FLAG_FORCE_STRIDED)         */
  int64_t batch_stride;
  int64_t rows_per_batch;
  int64_t seg_rows;        /* rows per contiguous-stride segment                          */
  int64_t seg_stride;
  int64_t row_stride;
  int32_t family;          /* 0: decode kernels (rows <= QMM_DECODE_MAX_ROWS), 1: prefill */
  int32_t kind;            /* 0: folded to one 2D matrix, 1: two strided levels,          */
                           /* 2: one grid slice per batch element (forced)                */
} qmm_plan_t;

/* Version of this ABI (QMM_ABI_VERSION). */
int32_t qmm_abi_version(void);

/* Message of the last failed call on this thread ("" if none).  Valid until the next call
 * into the library on the same thread. */
const char* qmm_last_error(void);

/* Quantize W [N, K] (float32, row n at w + n*w_row_stride) per row and per group of
 * group_size columns with min/max affine parameters (transformers issue 47331, "Root
 * cause": quantize, then cast scales and biases to the storage dtype):
 *   s = fl32(fl32(max - min) / (2^bits - 1)),  b = min,
 *   q = clamp(round_half_even(fl32(fl32(w - b) / s)), 0, 2^bits - 1)   (q = 0 when s == 0),
 * scales/biases stored as s, b rounded to nearest-even in dtype.
 * Outputs are dense: w_packed [N, K*bits/32] words, scales and biases [N, K/group_size].
 * Requires K % group_size == 0 and finite inputs.  N == 0 is a no-op. */
int32_t qmm_quantize(const float* w, int64_t N, int64_t K, int64_t w_row_stride,
                     int32_t group_size, int32_t bits, int32_t dtype,
                     uint32_t* w_packed, void* scales, void* biases, void* stream);

/* Matrix-vector form for decode: y = x . dequant(W)^T where the collapsed activation rows
 * number at most QMM_DECODE_MAX_ROWS (otherwise QMM_ERR_SHAPE: use qmm_t).
 * x: shape [..., K] (any rank 1..8), last-dim stride 1, other strides >= 0.  Batch dims
 *    are folded when their strides allow (candle pitfall page, 怎么确认没中招: dims i, i+1
 *    merge iff stride[i] == stride[i+1]*shape[i+1]; size-1 dims always merge); at most two
 *    strided levels may remain, otherwise QMM_ERR_LAYOUT.
 * y: dense row-major, shape x.shape[:-1] + [N].
 * Every row's arithmetic is independent of how many rows share the call, so row i of a
 * batched call is bit-identical to a call on row i alone (MLX pull request 4516,
 * "Correctness": bitwise-identical outputs over decode steps).
 * Sums of x are taken in float32 after widening each element (MLX pull request 4516,
 * first commit: widen each input before adding it to the bias * sum(x) term).
 * Alignment: x, w_packed 16-byte aligned; x strides (except the last) multiples of 8;
 * w_row_stride a multiple of the 32-code run: 4 words for 4- and 8-bit codes, 2 words for
 * 2- and 6-bit codes, 1 word otherwise.
 * Any K that is a multiple of group_size is accepted (e.g. K = 96 with group_size 32): the
 * decode kernels mask a last 128-code slot that ends past K (MLX pull request 4516, second
 * commit text: inputs that are not aligned for the fast qmv kernel need a guarded tail).
 * When w_row_stride is not a multiple of 4 words (rows padded to an odd word count) the
 * call runs the MFMA kernel that qmm_t uses for many rows.
 * M == 0 or N == 0 is a no-op returning QMM_OK. */
int32_t qmv(const void* x, const qmm_tensor_desc_t* x_desc, const qmm_weight_desc_t* w,
            void* y, const qmm_tensor_desc_t* y_desc, uint32_t flags, void* stream);

/* Transposed matrix-matrix form (prefill and batched decode): same operation and contract
 * as qmv, any number of rows.  Up to QMM_DECODE_MAX_ROWS collapsed rows it runs the same
 * kernels as qmv (so the results agree bitwise); beyond that, and at every row count for the
 * shapes the decode kernels do not take, it runs the MFMA prefill kernel, which dequantizes
 * weight tiles to dtype in LDS before the products. */
int32_t qmm_t(const void* x, const qmm_tensor_desc_t* x_desc, const qmm_weight_desc_t* w,
              void* y, const qmm_tensor_desc_t* y_desc, uint32_t flags, void* stream);

/* Gathered-weight decode form (mixture-of-experts decode): a stack of num_experts
 * quantized weights that share N, K, group_size, bits and dtype, expert e's codes at
 * w->w_packed + e*w_expert_stride words and its scales/biases at w->scales / w->biases +
 * e*sb_expert_stride elements; activation row r uses expert e = expert_index[r]:
 *   y[r, :] = x[r, :] . dequant(W_e)^T.
 * (MLX pull request 4516, pull request text: "Gathered QMV" is the expert-indexed variant of
 * the affine qmv; "Correctness": covered with batched weights.  The Bits=8 final report,
 * section 4.3, shows such expert stacks.)
 * x: rows folding to ONE strided level (e.g. [M, K] or [M, 1, K]); y dense [..., N].
 * expert_index: DEVICE array of x's row count int32 values.  Indices are read on the GPU; a
 * row whose index is outside [0, num_experts) gets NaN outputs (nothing is read outside the
 * stack).  Each row runs the decode kernels on its own (at most 65535 rows), and its result
 * is bit-identical to qmv on that row with expert e's weight.
 * Strides: w_expert_stride >= N * w_row_stride (a multiple of 4), sb_expert_stride >=
 * N * sb_row_stride.  w_row_stride must be a multiple of 4 words (the decode kernels' row
 * alignment; QMM_ERR_ALIGN otherwise).  Other requirements as for qmv.  Zero rows or
 * N == 0 is a no-op. */
int32_t qmm_gather_qmv(const void* x, const qmm_tensor_desc_t* x_desc, const qmm_weight_desc_t* w,
                       int64_t num_experts, int64_t w_expert_stride, int64_t sb_expert_stride,
                       const int32_t* expert_index, void* y, const qmm_tensor_desc_t* y_desc, void* stream);

/* Decode form with a fused per-row argmax (e.g. greedy next-token choice on lm_head logits;
 * the failure the transformers issue 47331 report shows is this argmax collapsing to
 * token 0 for every row after the first, section "Reproduction"):
 *   y = x . dequant(W)^T as in qmv, and for every activation row m
 *   out_index[m] = the first n with y[m, n] == max_n y[m, n], out_value[m] = that value
 *   (as float32; NaN counts as larger than any number).
 * The comparison uses the values y holds (rounded to dtype), so out_index equals an argmax
 * over the returned logits.  y may be NULL: the logits are then not written at all.
 * workspace: DEVICE, 8-byte aligned, 8 * (rows + 1) bytes (QMM_ARGMAX_WORKSPACE_BYTES), ALL
 * ZERO when the call's kernel starts: zero-fill it once when it is allocated.  The kernel
 * leaves it all-zero again when it ends (its last workgroup reads the per-row keys out and
 * clears them), so one workspace serves any number of calls in stream order; calls that may
 * run at the same time (different streams) need workspaces of their own.  out_value may be
 * NULL.  Contract otherwise as for qmv (at most QMM_DECODE_MAX_ROWS rows), but w_row_stride
 * must be a multiple of 4 words (QMM_ERR_ALIGN otherwise); 0 < N < 2^31.
 * One kernel is enqueued. */
#define QMM_ARGMAX_WORKSPACE_BYTES(rows) (8 * ((rows) + 1))
int32_t qmm_qmv_argmax(const void* x, const qmm_tensor_desc_t* x_desc, const qmm_weight_desc_t* w, void* y,
                       const qmm_tensor_desc_t* y_desc, int32_t* out_index, float* out_value, void* workspace,
                       void* stream);

/* The same call as qmm_qmv_argmax without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation).  The workspace is a library-owned device array of
 * QMM_NOALLOC_MAX_ROWS + 1 eight-byte words per GPU (512 bytes), kept until the process ends;
 * its device address is looked up once per device, on the first call made there.  Each call
 * enqueues a small kernel that zeroes the words it uses, then the decode kernel; nothing is
 * allocated or freed.  Calls on one GPU share that array: calls in stream order are fine,
 * calls that may run at the same time (different streams) race and give wrong results.
 * More than QMM_NOALLOC_MAX_ROWS collapsed activation rows -> QMM_ERR_SHAPE (the decode
 * family takes at most QMM_DECODE_MAX_ROWS anyway).  Results are bitwise those of
 * qmm_qmv_argmax; contract otherwise as for it. */
#define QMM_NOALLOC_MAX_ROWS 32
int32_t qmm_qmv_argmax_noalloc(const void* x, const qmm_tensor_desc_t* x_desc, const qmm_weight_desc_t* w, void* y,
                               const qmm_tensor_desc_t* y_desc, int32_t* out_index, float* out_value, void* stream);

/* Per-row top-k of stored logits (the top-k form of the decode epilogue on lm_head logits;
 * transformers issue 47331, "Reproduction": the next-token choice that collapses to token
 * 0): for every row m and j < k, out_index[m * k + j] and out_value[m * k + j] are the
 * column and value of the j-th largest entry of logits row m.  Order: larger value first;
 * NaN counts as larger than any number and +0 as larger than -0; equal values by lower
 * column, so k = 1 gives the column qmm_qmv_argmax returns.  A NaN entry is reported as a
 * quiet NaN.
 * logits: DEVICE [rows, row_stride] of dtype (QMM_BF16 or QMM_FP16), 2-byte aligned,
 * row_stride >= n.  out_index: DEVICE int32 [rows, k], 4-byte aligned; out_value: DEVICE
 * float32 [rows, k] or NULL.  Need 0 < n < 2^31, 0 <= rows < 2^31 and
 * 1 <= k <= min(n, QMM_TOPK_MAX) (QMM_ERR_SHAPE otherwise); rows == 0 is a no-op.
 * workspace: NULL, or DEVICE, 8-byte aligned, QMM_TOPK_WORKSPACE_BYTES(rows) bytes of any
 * content (the call writes every word it reads back; one workspace serves any number of
 * calls in stream order; calls that may overlap need workspaces of their own).  With a
 * workspace, long rows are split into column chunks of at least 2048 (about one chunk
 * workgroup per compute unit in all, at most 1024 / k chunks per row): one kernel writes
 * each chunk's k best candidates to the workspace and a second merges them per row.
 * Without one, or when a row is not split, each row is one workgroup and one kernel.  The
 * results are the same either way.
 * One or two kernels are enqueued; nothing is allocated. */
#define QMM_TOPK_MAX 1024
#define QMM_TOPK_WORKSPACE_BYTES(rows) (32776 * (rows))
int32_t qmm_topk(const void* logits, int32_t dtype, int64_t rows, int64_t n, int64_t row_stride, int32_t k,
                 int32_t* out_index, float* out_value, void* workspace, void* stream);

/* Decode with a per-row top-k: y = x . dequant(W)^T exactly as qmv (y is required and
 * dense, contract as for qmv), then qmm_topk over the rows of y (n = N, row_stride = N)
 * into out_index / out_value [rows, k], with `workspace` as for qmm_topk.  k is checked
 * before anything is enqueued.  The decode kernel and the top-k's one or two kernels are
 * enqueued. */
int32_t qmm_qmv_topk(const void* x, const qmm_tensor_desc_t* x_desc, const qmm_weight_desc_t* w, void* y,
                     const qmm_tensor_desc_t* y_desc, int32_t k, int32_t* out_index, float* out_value,
                     void* workspace, void* stream);

/* Dequantize a whole quantized weight to a dense matrix: out[n, k] = RNE_dtype(fl32(fma(s, q, b)))
 * with s, b the (n, k / group_size) scale and bias and q the code (transformers issue 47331,
 * "Root cause": the probe dequantizes the packed weight back to a dense tensor; the
 * float32 multiply-add followed by one rounding to dtype is this library's reading).
 * out: DEVICE [N, out_row_stride] of dtype, 16-byte aligned, out_row_stride >= K and a
 * multiple of 8.  w_packed and w_row_stride aligned to a 32-code run: 4 words (16 bytes)
 * for 4- and 8-bit codes, 2 words for 2- and 6-bit codes, 1 word otherwise.
 * N == 0 is a no-op. */
int32_t qmm_dequantize(const qmm_weight_desc_t* w, void* out, int64_t out_row_stride, void* stream);

/* Quantized embedding lookup: out[r, :] = dequantized row indices[r] of W (same rounding as
 * qmm_dequantize; Metal Kernel Bits=8 final report, section 3.2, dequantizes single rows of
 * a quantized table).  indices: DEVICE int32 [count]; an index outside [0, N) yields a NaN
 * row (nothing is read outside the table).  out as for qmm_dequantize with count rows.
 * count == 0 is a no-op. */
int32_t qmm_embedding(const qmm_weight_desc_t* w, const int32_t* indices, int64_t count, void* out,
                      int64_t out_row_stride, void* stream);

/* Host-only: validate a qmv (entry = 0) or qmm_t (entry = 1) call and report its plan
 * without touching the GPU.  Pointers inside `w` are only checked for NULL/alignment when
 * they are non-NULL (pass NULLs to test layouts alone).  Returns QMM_OK or the same error
 * code the call itself would return. */
int32_t qmm_plan(const qmm_tensor_desc_t* x_desc, const qmm_weight_desc_t* w,
                 const qmm_tensor_desc_t* y_desc, uint32_t flags, int32_t entry,
                 qmm_plan_t* out);

/* ---- A key/value cache held in 4 bits, and attention over it.
 * The cache keeps, per token slot and kv head, one K and one V row of head_dim values in the
 * weights' codec with 4-bit codes: x = s * q + b per group of group_size consecutive values,
 * s and b in dtype (quantizing the K and V rows a decode step appends is the min/max codec of
 * qmm_quantize, row by row).  It is paged: slot = page * page_size + offset, and a block table
 * names each sequence's pages in order.
 * data: DEVICE, 16-byte aligned, pages * heads * QMM_KV_PAGE_WORDS words; the words' order is
 * the library's own (rows go in with qmm_kv_append and come out with qmm_kv_read).  Any
 * content is a valid empty cache: tokens outside a sequence's length are never used.
 * Limits: head_dim in {64, 128, 256}; group_size in {32, 64, 128} and <= head_dim; page_size a
 * multiple of 16, at most 65536; heads 1..4096; pages >= 1 and pages * page_size < 2^31. */
typedef struct {
  uint32_t* data;
  int64_t pages;
  int32_t page_size;   /* tokens per page */
  int32_t heads;       /* kv heads        */
  int32_t head_dim;
  int32_t group_size;
  int32_t dtype;       /* qmm_dtype_t     */
} qmm_kv_cache_t;
/* Words of one page of one head: codes and (s, b) pairs of its K and V rows. */
#define QMM_KV_PAGE_WORDS(page_size, head_dim, group_size) \
  (2 * (int64_t)(page_size) * ((head_dim) / 8 + (head_dim) / (group_size)))

/* Quantize `tokens` new K and V rows per head into the cache: row (t, h) of k and v goes to
 * slots[t] of head h.  Per group, in float32: s = (max - min) / 15, b = min,
 * q = clamp(round_half_even((x - b) / s), 0, 15) (0 when s == 0); s and b are then rounded to
 * dtype.  k, v: DEVICE, dtype, element (t, h, d) at t * token_stride + h * head_stride + d;
 * 16-byte aligned, strides >= 0 and multiples of 8; finite values.  slots: DEVICE int32
 * [tokens], distinct; a slot outside [0, pages * page_size) is skipped (nothing is written for
 * it), so negative slots can pad a batch.  tokens == 0 is a no-op; tokens * heads * head_dim,
 * tokens rounded up to 2048 / head_dim, is below 2^34 (the threads of one launch).  One kernel is enqueued. */
int32_t qmm_kv_append(const qmm_kv_cache_t* cache, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                      const void* v, int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                      int64_t tokens, void* stream);

/* The values the cache stands for at `count` slots: k and v, DEVICE, dense
 * [count, heads, head_dim] of dtype, 16-byte aligned, round(fma(s, q, b)) of each element.  A
 * slot outside [0, pages * page_size) gives NaN rows.  count == 0 is a no-op; count is limited as
 * qmm_kv_append's tokens are.  One kernel. */
int32_t qmm_kv_read(const qmm_kv_cache_t* cache, const int32_t* slots, int64_t count, void* k, void* v,
                    void* stream);

/* Queries of one attention call over the cache.  Query i (0 <= i < q_len) of sequence n sits at
 * position p = lengths[n] - q_len + i (the queries are the last q_len of the sequence's tokens,
 * already appended).  It sees the cached tokens j in [0, lengths[n]); with `causal` only
 * j <= p; with window > 0 (which needs causal) only j > p - window.
 *     out = sum_j softmax_j(scale * q . k_j) v_j   over the tokens it sees, 0 if it sees none
 * (an empty sequence, or p < 0: queries padded on the left).  Query head h reads kv head
 * h / (q_heads / heads). */
typedef struct {
  const void* q;           /* DEVICE, dtype, element (n, i, h, d) at the strides below + d;
                            * 16-byte aligned, strides >= 0 and multiples of 8              */
  int64_t q_batch_stride, q_token_stride, q_head_stride;
  int64_t batch;           /* sequences, at most 65535                                       */
  int64_t q_len;           /* queries per sequence, below 32768                              */
  int32_t q_heads;         /* a multiple of the cache's heads                                */
  int32_t causal;
  int64_t window;
  float scale;
  const int32_t* block_table; /* DEVICE int32 [batch, table_stride]: page of tokens
                            * [j * page_size, (j + 1) * page_size) of sequence n at
                            * n * table_stride + j.  Only entries of tokens that are seen are
                            * read; one outside [0, pages) makes the outputs that need it NaN. */
  int64_t table_stride;
  int64_t max_blocks;      /* entries per sequence, <= table_stride                          */
  const int32_t* lengths;  /* DEVICE int32 [batch]; a length outside [0, max_length] makes
                            * the sequence's outputs NaN                                     */
  int64_t max_length;      /* the most tokens any sequence has, known to the host: sizes the
                            * launch; <= max_blocks * page_size, <= 2^30                      */
} qmm_kv_attend_t;

/* Attention over the cache: out, DEVICE, dense [batch, q_len, q_heads, head_dim] of dtype,
 * 16-byte aligned.  Scores, softmax and sums are float32.  The operands of the product with V
 * have float32's range and 16 bits: p s_g, whose error is at most 2^-16 of it; in calls with 256
 * query rows per kv head (q_len * q_heads / heads) or more p and v, each product within 2^-14 of
 * |p v|.  workspace: DEVICE, 16-byte aligned, any content, at least
 * qmm_kv_attend_workspace_bytes(cache, args) bytes (NULL when that is 0); one workspace serves
 * any number of calls in stream order, calls that may overlap need their own.  The result depends
 * only on the inputs and max_length.  Cached rows that are not finite reach only the queries that
 * see their token: those of K make their outputs NaN, those of V the elements of their group, or
 * the whole outputs in calls with 256 such rows or more.  batch == 0 or q_len == 0 is a no-op.
 * One kernel is enqueued, or two when the tokens are split over workgroups. */
int32_t qmm_kv_attend(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args, void* out, void* workspace,
                      int64_t workspace_bytes, void* stream);

/* Host-only: workspace bytes of a qmm_kv_attend call (its pointers may be NULL), or a negative
 * error code.  Monotone in max_length: the bytes for the longest length serve every shorter
 * one, with any window. */
int64_t qmm_kv_attend_workspace_bytes(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args);

/* ---- Trees of drafted tokens, and the pages of the cache.
 * A tree of a sequence has `nodes` nodes; parents[i] is node i's parent, an earlier node
 * (0 <= parents[i] < i), or -1 for a root.  Anything else there means that i is no node (padding
 * of a smaller tree), and so are its descendants.  The nodes are the last `nodes` tokens of the
 * sequence: node i is appended at position c + i, c = length - nodes, and stands for position
 * c + depth(i) of the text (depth 0: a root). */
#define QMM_TREE_MAX_NODES 1024

/* Which nodes a node sees, once per tree for every layer: bit j of the row of node i
 * ([batch, nodes, ceil(nodes / 32)] words, bit j % 32 of word j / 32) is set for i itself and its
 * ancestors, with window > 0 for the nearest `window` of them.  The row of what is no node is zero.
 * depth: [batch, nodes], the number of ancestors (0 for what is no node), or NULL.  parents:
 * DEVICE int32 [batch, parents_stride].  mask, depth: DEVICE, dense, 4-byte aligned.  batch at most
 * 65535; batch == 0 or nodes == 0 is a no-op.  One kernel. */
int32_t qmm_tree_mask(const int32_t* parents, int64_t parents_stride, int64_t batch, int64_t nodes, int64_t window,
                      uint32_t* mask, int32_t* depth, void* stream);

/* Attention of a tree's nodes over the cache: qmm_kv_attend (arguments, arithmetic, limits,
 * workspace), except for what a query sees.  Query i is node i of its sequence's tree; it sees the
 * tokens j < c before the tree, with a window only j > c + depth[i] - window, and the nodes of its
 * row of `mask`; a row of zeros sees nothing and gives zeros.  mask and depth (read with a window
 * only, which may then not be NULL) are qmm_tree_mask's for this batch and q_len = nodes at most
 * QMM_TREE_MAX_NODES, or the caller's own (a depth may pass the number of nodes; one below 0 counts as
 * 0); a window is applied to a mask by qmm_tree_mask.  causal
 * must be set.  A length of zero gives zeros; another one below q_len, like one above max_length,
 * makes the sequence's outputs NaN. */
int32_t qmm_kv_attend_tree(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args, const uint32_t* mask,
                           const int32_t* depth, void* out, void* workspace, int64_t workspace_bytes, void* stream);

/* Host-only: workspace bytes of a qmm_kv_attend_tree call, as qmm_kv_attend_workspace_bytes. */
int64_t qmm_kv_attend_tree_workspace_bytes(const qmm_kv_cache_t* cache, const qmm_kv_attend_t* args);

/* The path that verification accepts.  tokens[i] is the token that node i drafts, sampled[i] the
 * one that the model draws after it.  The path starts with node 0 (a root: a token that is already
 * certain) and goes on to the lowest child i of its last node l with tokens[i] == sampled[l].
 * path: DEVICE int32 [batch, nodes], its nodes in order, then -1; count: [batch], their number;
 * last: [batch], what is sampled after the path's end, the next certain token.  Where node 0 is no
 * root: count 0, last -1.  At least one node, batch at most 65535; batch == 0 is a no-op.  One
 * kernel. */
typedef struct {
  const int32_t* parents;   /* DEVICE int32 [batch, stride] each, 4-byte aligned */
  const int32_t* tokens;
  const int32_t* sampled;
  int64_t parents_stride, tokens_stride, sampled_stride;
  int64_t batch;
  int64_t nodes;
} qmm_tree_accept_t;
int32_t qmm_tree_accept(const qmm_tree_accept_t* args, int32_t* path, int32_t* count, int32_t* last, void* stream);

/* Move cached rows of a sequence, as they are: the K and V rows of every head at position
 * origin[n] + index[n, i] of sequence n go to position start[n] + i.  Entries whose index is
 * negative, or whose positions are negative or have no page in [0, pages), move nothing.
 * Without to_table the rows stay in the sequence's pages (a path's rows moved up to the tree's
 * first position; kept rows moved together): the indices that move must then ascend and no row may
 * move up, origin[n] + index[n, i] >= start[n] + i; every row arrives as it was before the call.
 * With to_table they go to the pages that it names, none of which the call may read.  Pages that
 * are written belong to one sequence. */
typedef struct {
  const int32_t* block_table;   /* DEVICE int32 [batch, table_stride], as in qmm_kv_attend */
  int64_t table_stride, blocks;
  const int32_t* to_table;      /* DEVICE int32 [batch, to_stride], or NULL                */
  int64_t to_stride, to_blocks;
  const int32_t* index;         /* DEVICE int32 [batch, index_stride]                      */
  int64_t index_stride;
  int64_t batch;                /* at most 65535, batch * heads below 2^24                 */
  int64_t count;                /* entries per sequence, at most 2^30                      */
  const int32_t* origin;        /* DEVICE int32 [batch], or NULL: 0                        */
  const int32_t* start;         /* DEVICE int32 [batch], >= 0                              */
} qmm_kv_move_t;
/* batch == 0 or count == 0 is a no-op.  One kernel. */
int32_t qmm_kv_move(const qmm_kv_cache_t* cache, const qmm_kv_move_t* args, void* stream);

/* Copy pages src[i] to dst[i], all heads, i < count.  A pair with a page outside [0, pages) is
 * skipped.  The dst are distinct and no src.  DEVICE int32 [count]; count == 0 is a no-op.  One
 * kernel. */
int32_t qmm_kv_copy_pages(const qmm_kv_cache_t* cache, const int32_t* src, const int32_t* dst, int64_t count,
                          void* stream);

/* One step of a program's block tables: beams and samples that continue one sequence, sequences
 * that begin, grow or are cut back, and those that end.  refs[p] counts the entries of the
 * program's tables that name page p; 0: the page is free.  The old table (batch rows) is replaced
 * by the new one (rows rows): row i continues row parents[i], or begins empty if that is outside
 * [0, batch).  It keeps the first min(length, want) tokens and has room for want[i] (NULL: the
 * parent's length); with s = page_size
 *   - blocks of which every token stays name the old page, which all such rows share;
 *   - the block that is kept in part, and those after it up to ceil(want / s), are the row's own, to
 *     write to.  The first row (lowest i) of a parent has the old page there if nobody else holds it: no
 *     other table (refs 1), and no other row of the parent, of which the block's every token stays.
 *     Otherwise they are fresh pages: entry number k of these, by row and block, gets the k-th lowest
 *     page that was free before the call.  Rows of a fresh page for a block kept in part are to be copied:
 *     copy_src[i] -> copy_dst[i] with qmm_kv_copy_pages, for each layer's cache (-1: nothing);
 *   - other entries are -1, and so are those for which no page is left or new_blocks is too small:
 *     *short_of counts these, of kept tokens too (of each row at most 16384 past new_blocks).  A kept
 *     block that had no page before the call has none after it, and is not counted.
 * refs is brought up to date: pages that only old rows named become free for the next call.
 * Entries outside [0, pages) name no page.  new_table must not overlap the old one.
 * copy_src, copy_dst: DEVICE int32 [rows]; short_of: DEVICE int32 [1]; workspace: DEVICE, 4-byte
 * aligned, qmm_kv_fork_workspace_bytes(args) bytes of any content; one serves any number of calls
 * in stream order.  Two or three kernels.  batch, rows <= 65535; rows * new_blocks <= 2^30; the limits of
 * pages and page_size are the cache's. */
typedef struct {
  int32_t* refs;                /* DEVICE int32 [pages]                                    */
  int64_t pages;
  int32_t page_size;
  const int32_t* block_table;   /* DEVICE int32 [batch, table_stride]                      */
  int64_t table_stride, blocks;
  const int32_t* lengths;       /* DEVICE int32 [batch]; negative counts as 0              */
  int64_t batch;
  const int32_t* parents;       /* DEVICE int32 [rows]                                     */
  const int32_t* want;          /* DEVICE int32 [rows] or NULL; negative counts as 0       */
  int64_t rows;
  int32_t* new_table;           /* DEVICE int32 [rows, new_stride]                         */
  int64_t new_stride, new_blocks;
} qmm_kv_fork_t;
int32_t qmm_kv_fork(const qmm_kv_fork_t* args, int32_t* copy_src, int32_t* copy_dst, int32_t* short_of, void* workspace,
                    int64_t workspace_bytes, void* stream);

/* Host-only: workspace bytes of a qmm_kv_fork call (its pointers may be NULL), or a negative error code. */
int64_t qmm_kv_fork_workspace_bytes(const qmm_kv_fork_t* args);

/* ---- A mixture-of-experts layer for a few tokens.
 * Expert stack: num_experts quantized weights that share N, K, group_size, bits and dtype
 * (w describes expert 0; expert e's codes are w_expert_stride words further, its scales and
 * biases sb_expert_stride elements), as in qmm_gather_qmv. */
typedef struct {
  qmm_weight_desc_t w;
  int64_t num_experts;
  int64_t w_expert_stride;   /* words, >= N * w_row_stride                  */
  int64_t sb_expert_stride;  /* elements, >= N * sb_row_stride              */
} qmm_expert_stack_t;

/* Per token t, with S_t its top_k largest router logits (equal ones: the lower expert; NaN
 * counts as largest):
 *     p_e = softmax of the router logits over S_t (renormalize) or over all experts,
 *     y_t = sum_{e in S_t} p_e * ( silu(Wg_e x_t) * (Wu_e x_t) ) Wd_e^T,  silu(g) = g / (1 + exp(-g)).
 * gate, up: [inter, hidden] per expert, sharing bits and group_size; down: [hidden, inter],
 * any bits and group_size.  hidden and inter are at most 2^20, the codes of one expert (and of 128
 * rows more) below 1 GiB.  4- and 8-bit codes: w_packed 16-byte aligned, w_row_stride and
 * w_expert_stride multiples of 4 words; other widths: any word. */
typedef struct {
  const void* x;               /* DEVICE [tokens, x_stride] of dtype, 16-byte aligned, x_stride % 8 == 0 */
  int64_t x_stride;
  const void* router_logits;   /* DEVICE [tokens, router_stride] of dtype, 2-byte aligned               */
  int64_t router_stride;
  int64_t tokens;              /* at most QMM_DECODE_MAX_ROWS                                           */
  int32_t top_k;               /* at most QMM_MOE_MAX_TOP_K                                             */
  int32_t renormalize;
  int32_t dtype;
  const qmm_expert_stack_t* gate;
  const qmm_expert_stack_t* up;
  const qmm_expert_stack_t* down;
  int64_t y_stride;            /* elements between rows of y, >= hidden                                 */
} qmm_moe_t;

#define QMM_MOE_MAX_EXPERTS 512
#define QMM_MOE_MAX_TOP_K 32

/* The layer: y DEVICE [tokens, y_stride] of dtype, 2-byte aligned.  Sums in float32;
 * silu(g) * u enters the second product with 16 bits (two bfloat16 parts) and float32's range.
 * workspace: DEVICE, 16-byte aligned, qmm_moe_workspace_bytes(...) bytes of any content; one serves any
 * number of calls in stream order, calls that may overlap need their own.  The result depends
 * only on the inputs (no atomics).  tokens == 0 is a no-op.  Three kernels are enqueued. */
int32_t qmm_moe(const qmm_moe_t* args, void* y, void* workspace, int64_t workspace_bytes, void* stream);

/* Host-only: workspace bytes of qmm_moe for these sizes, or a negative error code.  Grows with
 * every argument. */
int64_t qmm_moe_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter);

/* ---- Matrix products grouped by expert, for any number of rows.
 *     y[r] = x[r] W_e^T   for offsets[e] <= r < offsets[e + 1]
 * over a stack of quantized weights [N, K]; the weight that a code stands for, s * q + b, is not
 * rounded (codes are exact operands, scales and biases enter in float32, as in qmv).
 * x: DEVICE [rows, x_stride] of dtype, 16-byte aligned, x_stride % 8 == 0.
 * offsets: DEVICE int32 [num_experts + 1], ascending; they are taken into [0, rows], and an expert's
 * rows start where those of all before it have ended.  Rows of y that belong to no expert are left
 * as they are.  y: DEVICE [rows, y_stride] of dtype, 2-byte aligned, y_stride >= N.  rows at most
 * 2^20, num_experts at most QMM_MOE_MAX_EXPERTS, N and K at most 2^20; the limits and alignments
 * of qmm_moe's stacks.  Calls that no launch holds are refused: rows * K (K rounded up to 4096) up to
 * 2^35 - 2^15 and (rows / 16 + num_experts) * N (N rounded up to 256) up to 2^32 - 2^11 always fit.  workspace: DEVICE, 16-byte aligned, qmm_grouped_workspace_bytes(rows, weights)
 * bytes of any content; one serves any number of calls in stream order, calls that may overlap need
 * their own.  A row's result depends on nothing but the row and its expert.  rows == 0 is a no-op.  Two kernels. */
int32_t qmm_grouped(const void* x, int64_t x_stride, int64_t rows, const qmm_expert_stack_t* weights,
                    const int32_t* offsets, void* y, int64_t y_stride, void* workspace, int64_t workspace_bytes,
                    void* stream);

/* Host-only: workspace bytes of qmm_grouped for up to `rows` rows (pointers in weights may be
 * NULL), or a negative error code. */
int64_t qmm_grouped_workspace_bytes(int64_t rows, const qmm_expert_stack_t* weights);

/* The layer of qmm_moe for any number of tokens (at most 65535, tokens * top_k at most 2^20,
 * tokens * hidden, each row rounded up to 128, below 2^29; (tokens * top_k / 16 + num_experts) times the
 * larger of hidden and 2 * inter, rounded up to 256, always fits up to 2^32 - 2^11, and calls that no launch
 * holds are refused): arguments, formula, arithmetic and alignments are qmm_moe's, the workspace is
 * qmm_moe_prompt_workspace_bytes(...) bytes.  tokens == 0 is a no-op.  Five kernels.
 * For fewer than about 12 tokens qmm_moe is the faster one (8 experts of 4096 x 14336, 4 bits: 1 token
 * 54 us against 75, 8 tokens 200 / 238, 16 tokens 239 / 242, 32 tokens 345 / 239). */
int32_t qmm_moe_prompt(const qmm_moe_t* args, void* y, void* workspace, int64_t workspace_bytes, void* stream);

/* Host-only: workspace bytes of qmm_moe_prompt for these sizes, or a negative error code.  Grows
 * with every argument. */
int64_t qmm_moe_prompt_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t hidden, int64_t inter);

/* Settings of qmm_sample, per row: each is a DEVICE array [rows] (4-byte aligned) or, where the
 * pointer is NULL, one number for every row. */
typedef struct {
  const float* temperature;   /* T; <= 0 or NaN: the first largest logit, whatever u is        */
  const int32_t* top_k;       /* keep the top_k largest; <= 0: all                             */
  const float* top_p;         /* keep the shortest prefix reaching this share; >= 1: all; NaN,
                               * like 0, the first largest alone                              */
  const float* min_p;         /* keep weights of at least min_p times the largest; <= 0: all;
                               * NaN, like a number above 1, the first largest alone           */
  float temperature_all;
  int32_t top_k_all;
  float top_p_all;
  float min_p_all;
} qmm_sample_params_t;

/* Draw one column per logits row from given uniform numbers.  Logits that are NaN or -inf are
 * never drawn; the others weigh W_i = floor(2^40 * exp((l_i - max l) / T)), the quotient and
 * exponential in float32 (1 for l_i == max l).  In order of descending logit, equal ones by
 * lower column, a row keeps its top_k first columns; of those the shortest prefix whose weights
 * reach floor(top_p * 2^24) / 2^24 of their sum; of those the columns with
 * exp((l_i - max l) / T) >= min_p.  The largest always stays.  The drawn column is the first,
 * in column order, at which the running sum of the kept weights exceeds floor(u * 2^24) / 2^24
 * of their whole sum.  Sums are exact integers: the result depends on nothing but the inputs.
 * out_index: DEVICE int32 [rows], -1 for a row with nothing to draw (all NaN or -inf);
 * out_prob: DEVICE float32 [rows] or NULL, the drawn column's share of the kept weights (0 with
 * index -1).  u: DEVICE float32 [rows], clamped to [0, 1 - 2^-24] (NaN: 0).
 * logits: DEVICE [rows, row_stride] of dtype (QMM_BF16 or QMM_FP16), 2-byte aligned,
 * row_stride >= n.  Need 0 < n <= QMM_SAMPLE_MAX_N and rows <= 65535; rows == 0 is a no-op.
 * workspace: DEVICE, 8-byte aligned, QMM_SAMPLE_WORKSPACE_BYTES(rows) of any content; one
 * serves any number of calls in stream order, calls that may overlap need their own.
 * Four kernels are enqueued; nothing is allocated. */
#define QMM_SAMPLE_MAX_N (1 << 22)
#define QMM_SAMPLE_WORKSPACE_BYTES(rows) (190520 * (int64_t)(rows))
int32_t qmm_sample(const void* logits, int32_t dtype, int64_t rows, int64_t n, int64_t row_stride,
                   const qmm_sample_params_t* params, const float* u, int32_t* out_index, float* out_prob,
                   void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
