/*
 * libq4 -- Q4_0 block-quantised linear layers on AMD Instinct MI355X (gfx950).
 *
 * The C ABI of the library.  Plain pointers and sizes only; no HIP or torch
 * types appear in a signature (a stream is passed as an opaque pointer that
 * is a hipStream_t).
 *
 * The operation
 * -------------
 * "Vertical disaggregation: maximizing throughput on heterogeneous silicon",
 * section "Every cycle counts: custom kernels": the CPU and GPU backends share
 * one Q4_0 weight copy, output is deterministic, and the kernel stages are
 * nibble unpack, dot product, scale application, batched decode and a GPU
 * path onto matrix cores for prefill.  The format itself is not printed on
 * the page; this library fixes it as:
 *
 *   - a weight W[n][k] (row-major, n output features, k input features) is
 *     split along k into blocks of 32 (k must be a multiple of 32);
 *   - each block is 18 bytes: a 2-byte little-endian IEEE fp16 scale d, then
 *     16 code bytes; byte i holds the 4-bit code q of element i in its low
 *     nibble and of element i+16 in its high nibble;
 *   - a weight decodes as w = (q - 8) * d;
 *   - the packed buffer is n rows of k/32 consecutive blocks, rows
 *     contiguous: n * (k/32) * 18 bytes, no padding.
 *
 * Quantiser: m is the block element of largest magnitude (the first on a
 * tie); d = fp16(m / -8) rounded to nearest even, subnormals kept;
 * q = min(15, trunc(x / d + 8.5)) with x / d a correctly rounded fp32 division
 * by the fp16 scale widened to fp32 and the + 8.5 an fp32 addition; every q is
 * 8 when d is zero.
 *
 * Matmul: y[m][n] = sum_k x[m][k] * w[n][k] (x row-major [m][k], y row-major
 * [m][n]), accumulated in fp32.  Results are deterministic: identical inputs,
 * shapes and dtypes on the same device and build give identical bits (no
 * atomics, fixed reduction order).
 *
 * Conventions for every entry point
 * ---------------------------------
 *   - all data pointers are device pointers owned by the caller; the library
 *     never allocates, frees or synchronises, keeps no state, and is safe to
 *     call from several host threads;
 *   - every call is asynchronous on `stream` (NULL = the null stream); errors
 *     detected on the host return before anything is launched; a failed
 *     launch returns Q4_ERR_HIP; faults during execution surface at the
 *     caller's next synchronisation, as for any HIP library;
 *   - every data pointer must be 16-byte aligned (Q4_ERR_ALIGNMENT) and
 *     non-NULL (Q4_ERR_INVALID_ARG); outputs must not overlap inputs
 *     (Q4_ERR_INVALID_ARG);
 *   - shapes: n >= 1, m >= 1, k >= 32 and k % 32 == 0, and n * k below 2^40
 *     (Q4_ERR_SHAPE); for q4_gemv and q4_gemm also k <= 2^24 (the kernels
 *     address a tile's activation rows with 32-bit per-lane byte offsets);
 *   - inputs must be finite; weights must satisfy |w| < 65520 * 8 so that d
 *     is finite.  This is not checked on the device.
 */
#ifndef LIBQ4_Q4_H
#define LIBQ4_Q4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define Q4_ABI_VERSION 1
#define Q4_QK 32            /* weights per block */
#define Q4_BLOCK_BYTES 18   /* bytes per block */
#define Q4_GEMV_MAX_M 32    /* largest batch accepted by q4_gemv */

/* An opaque hipStream_t. */
typedef struct ihipStream_t *q4_stream_t;

typedef enum q4_status {
  Q4_OK = 0,
  Q4_ERR_INVALID_ARG = 1, /* NULL pointer, overlapping buffers */
  Q4_ERR_SHAPE = 2,       /* m, n or k out of range, k % 32 != 0 */
  Q4_ERR_DTYPE = 3,       /* dtype code not supported by this call */
  Q4_ERR_ALIGNMENT = 4,   /* a pointer is not 16-byte aligned */
  Q4_ERR_HIP = 5,         /* the HIP runtime refused a launch */
  Q4_ERR_WORKSPACE = 6,   /* workspace missing or smaller than required */
  Q4_ERR_UNSUPPORTED = 7, /* the host CPU lacks an instruction set the call needs
                             (q4_host.h) */
  Q4_ERR_SCRATCH = 8      /* the call needs more scratch than q4_gemm_noalloc's
                             fixed per-device array holds */
} q4_status;

typedef enum q4_dtype {
  Q4_F32 = 0, /* IEEE binary32 */
  Q4_F16 = 1, /* IEEE binary16 */
  Q4_BF16 = 2 /* bfloat16: the upper 16 bits of a binary32 pattern; accepted
                 for weights and activations, not for the outputs of q4_gemv
                 and q4_gemm */
} q4_dtype;

/* Version of this ABI (Q4_ABI_VERSION). */
int q4_abi_version(void);

/* Static, NUL-terminated description of a status code; never NULL. */
const char *q4_status_string(int status);

/* Size in bytes of a packed [n][k] Q4_0 weight: n * (k/32) * 18.
 * Returns 0 when the shape is invalid (n < 1, k < 32, k % 32 != 0). */
size_t q4_packed_size(int64_t n, int64_t k);

/* Quantise a row-major [n][k] weight `w` of dtype `w_dtype` (Q4_F32, Q4_F16
 * or Q4_BF16; fp16 and bf16 are widened exactly to fp32 first) into `packed`,
 * which must hold q4_packed_size(n, k) bytes.  The result is bit-identical to
 * the rule stated at the top of this header.  Reads 4 (fp32) or 2 (fp16,
 * bf16) bytes and writes 0.5625 bytes per weight. */
q4_status q4_quantize(const void *w, int w_dtype, int64_t n, int64_t k,
                      void *packed, q4_stream_t stream);

/* Batched-decode GEMV: y[m][n] = x[m][k] . dequant(packed)^T for
 * 1 <= m <= Q4_GEMV_MAX_M (the page's batched decode stage).  x is Q4_F32,
 * Q4_F16 or Q4_BF16, y is Q4_F32 or Q4_F16.  Every output is the fp32 sum
 * over blocks of d times the block dot product of x with (q - 8), rounded
 * once to the output dtype.  The block products take the codes as exact
 * integers q - 8, so each product x (q - 8) is exact and the error is fp32
 * summation error relative to sum |x w|, for every in-domain input.  bf16
 * x with k a multiple of 512 is converted to fp16 inside the kernel (round
 * to nearest even); a workgroup whose conversion was inexact anywhere (a
 * value beyond fp16's range or off its subnormal grid) recomputes its
 * outputs with x widened exactly to fp32, so the result is exact for every
 * bf16 value; other bf16 shapes are widened exactly to fp32.  Streams each
 * packed byte from memory once per call. */
q4_status q4_gemv(const void *x, int x_dtype, const void *packed, void *y,
                  int y_dtype, int64_t m, int64_t n, int64_t k,
                  q4_stream_t stream);

/* Bytes of workspace q4_gemm needs for this shape with fp16 activations (0
 * when none). */
size_t q4_gemm_workspace_size(int64_t m, int64_t n, int64_t k);

/* As q4_gemm_workspace_size for activations of dtype x_dtype (0 for fp32
 * activations, an unknown dtype or an invalid shape).  bf16 activations add
 * m * k * 2 bytes (rounded up to 256), where they are staged as fp16. */
size_t q4_gemm_workspace_size_dt(int64_t m, int64_t n, int64_t k, int x_dtype);

/* Prefill GEMM: y[m][n] = x[m][k] . dequant(packed)^T for any m >= 1 (the
 * page's GPU path onto matrix cores).  x is Q4_F32, Q4_F16 or Q4_BF16; y is
 * Q4_F32 or Q4_F16.
 *   - fp16 and bf16 activations: weight tiles are dequantised to fp16
 *     (w = (q - 8) * d rounded once) and contracted on fp16 matrix cores
 *     with fp32 accumulation; bf16 activations are first staged as fp16 in
 *     the workspace (round to nearest even).  Where that is not exact -- a
 *     block scale |d| > 8188, whose dequantised weights leave fp16's range,
 *     or a bf16 activation fp16 cannot hold -- the affected output tiles come
 *     out non-finite inside the kernel and are recomputed there on the exact
 *     route below, so every in-domain input gives a result within tolerance.
 *   - fp32 activations take the exact route for every tile: activations and
 *     dequantised weights in fp32 on fp32 matrix cores (several times slower
 *     than the fp16 tiles).
 * `workspace` must hold q4_gemm_workspace_size_dt(m, n, k, x_dtype) bytes (it
 * may be NULL when that is 0) and must not overlap x, y or packed; its
 * contents on entry are ignored.  A prompt processed in row chunks passes
 * x + c*rows*k and y + c*rows*n for chunk c. */
q4_status q4_gemm(const void *x, int x_dtype, const void *packed, void *y,
                  int y_dtype, int64_t m, int64_t n, int64_t k,
                  void *workspace, size_t workspace_bytes,
                  q4_stream_t stream);

/* Bytes of the fixed per-device scratch array behind q4_gemm_noalloc. */
#define Q4_NOALLOC_SCRATCH_BYTES (64u << 20)

/* q4_gemm for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation): the
 * same computation, kernels and results as q4_gemm, with the workspace taken
 * from a fixed array of Q4_NOALLOC_SCRATCH_BYTES bytes that the library holds
 * on each device it runs on until the process ends.  The array is the current
 * device's (the device of `stream`); the first call on a device looks up its
 * address once.  Calls whose workspace need, q4_gemm_workspace_size_dt(m, n,
 * k, x_dtype), exceeds the array return Q4_ERR_SCRATCH before launching
 * anything.  The call itself allocates nothing.  Every call on one device
 * shares that device's array: calls that may overlap on one device (several
 * streams, several host threads) race on it and must be serialised by the
 * caller; its contents after a call are unspecified, and each call writes
 * every scratch byte it reads.  Arguments, errors and layouts are q4_gemm's. */
q4_status q4_gemm_noalloc(const void *x, int x_dtype, const void *packed, void *y,
                          int y_dtype, int64_t m, int64_t n, int64_t k,
                          q4_stream_t stream);

/* ------------------------------------------------------------------------
 * Fused linear layer
 * ------------------------------------------------------------------------
 * The calls below also write Q4_BF16 outputs and take any m >= 1 (one entry
 * for decode and prefill).  Conventions are those at the top of this header
 * except where stated.  A call with a launch that a grid does not hold (more
 * than 65535 tiles of 128 to 256 rows, or 2^32 threads) is refused with
 * Q4_ERR_SHAPE before the first launch, and its workspace size is 0. */

typedef enum q4_activation {
  Q4_ACT_NONE = 0,
  Q4_ACT_RELU = 1,     /* max(z, 0) */
  Q4_ACT_GELU = 2,     /* z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
  Q4_ACT_GELU_ERF = 3, /* z / 2 (1 + erf(z / sqrt(2))) */
  Q4_ACT_SILU = 4      /* z / (1 + exp(-z)) */
} q4_activation;

/* What follows a product z = x . dequant(packed)^T of n weight rows:
 *   z += bias                             (n values of bias_dtype; NULL: none)
 *   gated == 0:  v = act(z)               n output columns
 *   gated != 0:  v = act(z[:n/2]) z[n/2:] n / 2 output columns (n even): the
 *                first half of the weight rows is the gate, the second the
 *                factor ("up") rows
 *   y = v + residual                      (shape and dtype of y; NULL: none)
 * all in fp32 with one rounding to y.  residual may be y itself (the same
 * pointer: accumulation in place) but not overlap it otherwise.  bias and
 * residual are 16-byte aligned. */
typedef struct q4_epilogue {
  const void *bias;
  int bias_dtype;  /* q4_dtype; read only with a bias */
  int activation;  /* q4_activation */
  int gated;       /* 0 or 1 */
  const void *residual;
} q4_epilogue;

/* Bytes of workspace q4_linear needs (0 when none, or for an invalid shape
 * or dtype). */
size_t q4_linear_workspace_size(int64_t m, int64_t n, int64_t k, int x_dtype, int gated);

/* Fused linear layer: y = epilogue(x[m][k] . dequant(packed[n])^T) for any
 * m >= 1; y is [m][n], or [m][n / 2] with a gate, of any q4_dtype.
 * `epilogue` may be NULL (the plain product).
 *   - fp32 x: fp32 products of the exactly decoded weights.
 *   - fp16 and bf16 x on matrix cores: for m <= 32 the weight codes enter as
 *     exact integers and the block scales in fp32, as in q4_gemv; above, the
 *     weights are dequantised to fp16 (one rounding, 2^-11 relative) as in
 *     q4_gemm, with the exact route for tiles where that overflows.
 *   - bf16 x may be staged as fp16, every row or part of a row multiplied by
 *     the power of two that brings its largest magnitude to [2^15, 2^16):
 *     exact for every value of at least 2^-32 of that magnitude; a smaller one
 *     is rounded to a multiple of 2^-39 of it.
 * `workspace` holds q4_linear_workspace_size bytes (NULL when that is 0),
 * overlaps no other buffer and is shared by no call that may run at the same
 * time (calls on several streams, graphs replayed at once). */
q4_status q4_linear(const void *x, int x_dtype, const void *packed,
                    const q4_epilogue *epilogue, void *y, int y_dtype, int64_t m,
                    int64_t n, int64_t k, void *workspace, size_t workspace_bytes,
                    q4_stream_t stream);

/* ------------------------------------------------------------------------
 * Experts
 * ------------------------------------------------------------------------ */

#define Q4_MAX_EXPERTS 1024
#define Q4_MAX_TOPK 32
#define Q4_MAX_GROUPS 64

typedef enum q4_score { Q4_SCORE_SOFTMAX = 0, Q4_SCORE_SIGMOID = 1 } q4_score;
typedef enum q4_group_score {
  Q4_GROUP_MAX = 0, /* a group counts as its best expert */
  Q4_GROUP_TOP2 = 1 /* a group counts as the sum of its two best experts */
} q4_group_score;

/* How experts are chosen.  For a token with logits l[experts]:
 *   s    = softmax(l) or sigmoid(l), element by element
 *   key  = s + bias; without a bias and with Q4_GROUP_MAX the logit itself
 *          (the same order)
 *   groups > 1: the experts are `groups` consecutive groups of equal size;
 *          only those in the group_topk best groups remain
 *   the topk largest keys are chosen, in descending order
 *   weight = s of the chosen (without bias); with renormalise divided by the
 *          sum over the chosen (0 if that sum is 0); times scale
 * Keys are formed and compared in 64 bits; ties go to the lowest index
 * (experts and groups alike).  An expert whose logit is -infinity or NaN, or
 * whose bias is -infinity or NaN, is never chosen for that token and counts 0
 * in a group's sum; where fewer than topk experts remain the rest of the row
 * is id -1, weight 0.  +infinity counts as the largest finite fp32. */
typedef struct q4_routing {
  int score;         /* q4_score */
  const float *bias; /* [experts] fp32 device array, 4-byte aligned; NULL: none */
  int groups;        /* 1 .. Q4_MAX_GROUPS, divides experts */
  int group_topk;    /* 1 .. groups */
  int group_score;   /* q4_group_score; used when groups > 1 */
  int renormalise;   /* 0 or 1 */
  float scale;       /* finite */
} q4_routing;

/* Bytes of a plan for m tokens with topk of `experts` experts each: int32
 * words, first offsets[experts + 1] (expert e's pairs are order[offsets[e]] ..
 * order[offsets[e + 1] - 1]; padded to a multiple of 4 words), then
 * order[m topk]: the pair numbers i topk + j, by expert and ascending within
 * one, then -1 for pairs whose id names no expert.  What follows is the
 * library's own.  0 for an invalid shape. */
size_t q4_route_plan_size(int64_t m, int64_t topk, int64_t experts);

/* Routing: ids[m][topk] (int32), weights[m][topk] (fp32) and, unless NULL, a
 * plan of q4_route_plan_size bytes from logits[m][experts] (Q4_F32, Q4_F16 or
 * Q4_BF16). */
q4_status q4_route(const void *logits, int logits_dtype, int64_t m, int64_t experts,
                   int64_t topk, const q4_routing *routing, int32_t *ids, float *weights,
                   void *plan, q4_stream_t stream);

/* The plan of given ids[m][topk]; an id outside 0 .. experts - 1 names no
 * expert.  A token may name the same expert more than once. */
q4_status q4_route_plan(const int32_t *ids, int64_t m, int64_t topk, int64_t experts,
                        void *plan, q4_stream_t stream);

/* Bytes of workspace q4_experts needs (0 when none or for an invalid shape).
 * `x_rows` and `combine` as below. */
size_t q4_experts_workspace_size(int64_t m, int64_t topk, int64_t experts, int64_t n, int64_t k,
                                 int64_t x_rows, int x_dtype, int gated, int combine);

/* The products of the chosen experts.  packed is [experts][n][k] Q4_0 (each
 * expert's rows as in q4_packed_size, experts contiguous), the epilogue's bias
 * [experts][n].  Pair p = i topk + j is token i's j-th expert e:
 *   row p = act((x_p . dequant(packed[e])^T) + bias[e])   (gated: as above)
 * with x_p = x[i] for x_rows == m and x_p = x[p] for x_rows == m topk.
 *   weights == NULL: y is [m topk][nout], y[p] = row p + residual[p]; a pair
 *     without an expert leaves its row of y as it was (no residual either).
 *   weights != NULL (fp32 [m][topk]): y is [m][nout],
 *     y[i] = sum_j weights[i][j] row(i topk + j) + residual[i], summed in fp32
 *     in the order of j; pairs without an expert count 0.
 * `plan` is what q4_route or q4_route_plan wrote for the same m, topk and
 * experts.  Types, routes and the workspace are q4_linear's; which route runs
 * goes by the mean number of rows per expert. */
q4_status q4_experts(const void *x, int x_dtype, int64_t x_rows, const void *packed,
                     const q4_epilogue *epilogue, const void *plan, const float *weights,
                     void *y, int y_dtype, int64_t m, int64_t topk, int64_t experts,
                     int64_t n, int64_t k, void *workspace, size_t workspace_bytes,
                     q4_stream_t stream);

/* Bytes of workspace q4_moe needs (0 for an invalid shape). */
size_t q4_moe_workspace_size(int64_t m, int64_t topk, int64_t experts, int64_t hidden,
                             int64_t inter, int x_dtype, int gated);

/* A whole expert layer: q4_route on logits[m][experts], q4_experts on x[m][hidden]
 * with `up` ([experts][inter or, gated, 2 inter][hidden]) into rows of x's dtype,
 * and q4_experts on those with `down` ([experts][hidden][inter]), combined by the
 * routing weights into y[m][hidden].  up_epilogue carries the activation, the
 * gate and [experts][..] bias (no residual); down_epilogue (may be NULL) the
 * bias and the residual (no activation, no gate).  ids and weights receive the
 * routing unless NULL. */
q4_status q4_moe(const void *x, int x_dtype, const void *logits, int logits_dtype,
                 const q4_routing *routing, const void *up, const q4_epilogue *up_epilogue,
                 const void *down, const q4_epilogue *down_epilogue, void *y, int y_dtype,
                 int64_t m, int64_t topk, int64_t experts, int64_t hidden, int64_t inter,
                 int32_t *ids, float *weights, void *workspace, size_t workspace_bytes,
                 q4_stream_t stream);

/* ------------------------------------------------------------------------
 * Cache of keys and values, and attention over it
 * ------------------------------------------------------------------------
 * A paged cache in Q4_0 and the attention that reads it: what stands between
 * the q/k/v product of a decoder layer and its output product.  Conventions
 * are those at the top of this header except where stated.
 *
 * The cache holds head_dim values of keys and of values for every position and
 * kv head, quantised by the rule at the top of this header, 32 values along
 * head_dim to a block, after these steps: a value is limited to +-65504 (an
 * infinity counts as that, NaN as 0), so every decoded value is finite and within
 * fp16's range.  It is [pages][kv_heads][2][page_size / 16] granules of 9
 * head_dim bytes ([2]: keys, values), sixteen positions each: 8 head_dim code
 * bytes, then head_dim / 2 fp16 scales.  With blocks = head_dim / 32, position
 * t = 0 .. 15 of the granule and code byte i = 0 .. 15 of a block b:
 *   keys    code byte at t head_dim / 2 + (i / 4 blocks + b) 4 + i % 4
 *           scale     at (t / 4 blocks + b) 4 + t % 4
 *   values  code byte at (b 16 + i) 16 + t
 *           scale     at b 16 + t / 4 4 + {0, 2, 1, 3}[t % 4]
 * (integer divisions).  A byte belongs to one position alone. */

#define Q4_CACHE_GRANULE 16     /* positions; page_size is a multiple of it */
#define Q4_CACHE_MAX_HEAD_DIM 256
#define Q4_CACHE_MAX_SEQS 65536

typedef struct q4_cache {
  void *data;         /* q4_cache_size bytes */
  int64_t pages;      /* 1 .. 2^31 - 1 */
  int64_t page_size;  /* positions per page: a multiple of 16, at most 2^30 */
  int64_t kv_heads;   /* 1 .. 65535 */
  int64_t head_dim;   /* a multiple of 32, at most Q4_CACHE_MAX_HEAD_DIM */
} q4_cache;

/* Some sequences and their rows.  Sequence s has the rows offsets[s] ..
 * offsets[s + 1] - 1 of q, k and v, n of them, and lengths[s] positions, of
 * which its rows are the last: its row i is position lengths[s] - n + i.
 * Position t is in page tables[s][t / page_size].  All arrays are on the device
 * and read when the call runs, 4-byte aligned.
 *   - Rows before offsets[0] and from offsets[seqs] on belong to no sequence:
 *     no call reads them or writes their outputs.
 *   - offsets, which do not fall, are limited to 0 .. tokens, lengths to 0 ..
 *     max_pages page_size.  A row whose position is negative has none.
 *   - A page number outside 0 .. pages - 1 names no page: its positions are not
 *     written, read as 0 and seen by no row.
 *   - Positions that one call writes lie in different places (sequences may
 *     share pages that it reads); a place that two of them name holds either's
 *     bytes or a mixture. */
typedef struct q4_batch {
  int64_t seqs;           /* 1 .. Q4_CACHE_MAX_SEQS */
  int64_t tokens;         /* rows of q, k and v, 1 .. 2^31 - 1 */
  int64_t max_pages;      /* 1 ..; max_pages page_size is at most 2^30 */
  const int32_t *tables;  /* [seqs][max_pages] */
  const int32_t *lengths; /* [seqs] */
  const int32_t *offsets; /* [seqs + 1]; NULL: row s is sequence s's only one (tokens == seqs) */
} q4_batch;

/* Bytes of a cache: pages kv_heads page_size head_dim 36 / 32 (0 for an
 * invalid shape, or one of 2^40 values or more). */
size_t q4_cache_size(int64_t pages, int64_t page_size, int64_t kv_heads, int64_t head_dim);

/* Quantise rows of keys and values into their positions.  k and v are
 * [tokens][kv_heads][head_dim] of `dtype`, row i at k + i k_stride and v + i
 * v_stride elements (at least kv_heads head_dim; whole 16-byte pieces, so that
 * rows of a fused q/k/v product are taken where they are).  Bytes of other
 * positions are not changed. */
q4_status q4_cache_write(const q4_cache *cache, const q4_batch *batch, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, int dtype, q4_stream_t stream);

/* The decoded values (q - 8) d of the rows' positions, rounded once to `dtype`,
 * into k and v, [tokens][kv_heads][head_dim], contiguous.  A row without a
 * position is written as zeros. */
q4_status q4_cache_read(const q4_cache *cache, const q4_batch *batch, void *k, void *v, int dtype,
                        q4_stream_t stream);

/* For a row at position p, head h of `heads` (a multiple of kv_heads, at most
 * 65536; h reads kv head h / (heads / kv_heads)), over the positions t it sees:
 *   s_t = scale q . k_t;  softcap > 0: s_t = softcap tanh(s_t / softcap)
 *   y   = sum_t exp(s_t) v_t / sum_t exp(s_t),  lse = ln sum_t exp(s_t)
 * It sees t < lengths[s], with `causal` t <= p, with window > 0 t > p - window.
 * A row that sees nothing has y = 0, lse = -infinity; any other whose q holds a NaN
 * or an infinity has NaN in both.  q . k and s_t are below 2^126 in magnitude: a
 * larger one may count as an infinity. */
typedef struct q4_attention_options {
  float scale;    /* finite */
  int causal;     /* 0 or 1 */
  int64_t window; /* 0: none */
  float softcap;  /* finite, >= 0; 0: none */
} q4_attention_options;

/* Bytes of workspace q4_attention needs (0 when none or for invalid arguments).
 * `with_offsets`: whether the batch has offsets. */
size_t q4_attention_workspace_size(int64_t seqs, int64_t tokens, int64_t heads, int64_t kv_heads,
                                   int64_t head_dim, int q_dtype, int with_offsets);

/* Softmax attention of q[tokens][heads][head_dim] (row i at q + i q_stride
 * elements, as in q4_cache_write) over the sequences' positions in the cache,
 * into y[tokens][heads][head_dim], contiguous, of any q4_dtype, and, unless
 * NULL, lse[tokens][heads] (fp32).  The rows' own positions are read from the
 * cache too: q4_cache_write comes first.
 *   - fp32 q: fp32 products of the exactly decoded values.
 *   - fp16 and bf16 q on matrix cores, with fp32 sums.  Sequences of few rows
 *     (single tokens, drafts) take the keys' codes as exact integers and their
 *     scales in fp32; sequences of many rows round the decoded keys to fp16
 *     once.  Decoded values and the weights exp(s_t - m) are rounded to fp16
 *     (with fp16 q and up to 16 rows, times heads per kv head, a sequence on
 *     average the weights are kept in two fp16 parts).
 *   - bf16 q are taken as fp16 times a power of two per row and head, as in
 *     q4_linear.
 * Results do not depend on what else runs, but the order of the sums over
 * positions depends on the whole batch's lengths.  Positions that no row sees
 * may hold anything.  `workspace` holds q4_attention_workspace_size bytes (NULL
 * when that is 0), overlaps no other buffer and is shared by no call that may
 * run at the same time. */
q4_status q4_attention(const q4_cache *cache, const q4_batch *batch, const q4_attention_options *options,
                       const void *q, int64_t q_stride, int q_dtype, int64_t heads, void *y, int y_dtype,
                       float *lse, void *workspace, size_t workspace_bytes, q4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBQ4_Q4_H */
