/*
 * indexer_ops.h - the operators around the top-k of a sparse-attention indexer,
 * for NVIDIA GB300 (sm_103a): what makes its scores, and what reads back the
 * rows that it selected. The entry points live in the same library as
 * topk_transform.h and share its status codes (topk_status_t),
 * topk_status_string and topk_last_cuda_error.
 *
 *   indexer_layer_norm   layer norm of the keys, and its gradients
 *   indexer_rotary       rotary positions on queries and keys (and the gradient), with
 *                        one position a token or one on each of several axes
 *   indexer_quantise     rows to e4m3 with one scale for each block of 128 columns
 *   indexer_cache_write  the same, written into a paged cache
 *   indexer_cache_read   cache rows at given slots, back in 16 or 32 bits
 *   indexer_scores       the indexer's scores over a paged cache: products in 8-bit
 *                        floating point, relu, weighted sum over heads
 *   indexer_cache_append rows into a paged cache of heads, with one scale for each block of
 *                        tokens and head
 *   indexer_attention    attention over two such caches (keys, values): whole sequences, or
 *                        the slots that were picked
 *
 * The scores are what topk_transform_* takes, and the positions that
 * topk_transform_paged writes are the slots that indexer_cache_read takes.
 *
 * Memory and ownership, stream order, errors: as in topk_transform.h. Every pointer
 * is device memory owned by the caller; the library never allocates, frees or
 * synchronises; a call enqueues one kernel on `stream` (several where it has 2^30 parts of
 * rows or more) and returns. Every launch
 * allows programmatic dependent launch and waits for the previous kernel of the
 * stream before it touches memory. Host-checkable problems return a status and
 * launch nothing. Values in device memory cannot be checked by the host: a slot or a
 * page id outside the cache is never followed. The access it asks for is skipped, the
 * result is as stated at each entry point, and indexer_guard_hits counts it.
 */
#ifndef INDEXER_OPS_H_
#define INDEXER_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#include "topk_transform.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns that share a scale. */
#define INDEXER_BLOCK 128
/* The head size of indexer_scores: one block. */
#define INDEXER_SCORE_DIM 128
/* The most heads that indexer_scores takes. */
#define INDEXER_MAX_HEADS 128

typedef enum { INDEXER_BF16 = 0, INDEXER_FP16 = 1, INDEXER_FP32 = 2 } indexer_dtype_t;

typedef enum {
  INDEXER_LAYOUT_HALF = 0,       /* pair i: columns start + i and start + rot_dim/2 + i */
  INDEXER_LAYOUT_INTERLEAVED = 1 /* pair i: columns start + 2i and start + 2i + 1 */
} indexer_layout_t;

typedef enum {
  INDEXER_SCALE_FP32 = 0, /* amax / 448, rounded to fp32 */
  INDEXER_SCALE_POW2 = 1  /* the smallest power of two >= amax / 448 */
} indexer_scale_format_t;

/* A paged cache of e4m3 rows. The row at slot s = page * page_size + offset has its
 * codes at codes + page * code_page_stride + offset * code_token_stride (bytes) and
 * its ceil(dim / 128) scales at scales + page * scale_page_stride +
 * offset * scale_token_stride (elements). Rows must not overlap.
 * 0 <= num_pages * page_size <= INT32_MAX; page_size, dim >= 1. */
typedef struct {
  uint8_t* codes;
  float* scales;
  int64_t num_pages;
  int64_t code_page_stride, code_token_stride;
  int64_t scale_page_stride, scale_token_stride;
  int32_t page_size;
  int32_t dim;
} indexer_cache_t;

/* sizeof(indexer_cache_t), for bindings. */
size_t indexer_cache_bytes(void);

/* The widest head of an indexer_block_cache_t. */
#define INDEXER_MAX_HEAD_DIM 256

/* A paged cache of e4m3 rows of several heads, with one scale for each block of `block` tokens
 * (which divides page_size) and head. The row of head h at slot s = page * page_size + offset
 * has its codes at codes + page * code_page_stride + offset * code_token_stride +
 * h * code_head_stride (bytes), its scale at scales + page * scale_page_stride +
 * (offset / block) * scale_block_stride + h * scale_head_stride (elements); the values it
 * stands for are code * scale. codes and its strides are multiples of 16 bytes, dim of 16, at
 * most INDEXER_MAX_HEAD_DIM. Rows and scales must not overlap. Scales are not negative.
 * 0 <= num_pages * page_size <= INT32_MAX; page_size, block, heads >= 1. */
typedef struct {
  uint8_t* codes;
  float* scales;
  int64_t num_pages;
  int64_t code_page_stride, code_token_stride, code_head_stride;
  int64_t scale_page_stride, scale_block_stride, scale_head_stride;
  int32_t page_size, block, heads, dim;
} indexer_block_cache_t;

/* sizeof(indexer_block_cache_t), for bindings. */
size_t indexer_block_cache_bytes(void);

/* Rotary positions. x, out: [tokens, heads, dim] of `dtype`, unit column stride, token
 * and head strides in elements (out's rows must not overlap; out may be x itself, with
 * the same strides, and must otherwise not overlap it; x's strides may be 0).
 * positions [tokens] int32 (any sign), freqs [rot_dim / 2] fp64, finite, in radians
 * per position. With angle = positions[t] * freqs[i], c = scale * cos(angle),
 * s = scale * sin(angle), pair i = (a, b) becomes
 *   (a c - b s, b c + a s)   or, with transpose != 0, the gradient's (a c + b s, b c - a s),
 * computed in fp32 and rounded once. Columns outside [start, start + rot_dim) are copied.
 * Angles keep their precision at any int32 position: freqs become 64-bit fixed-point turns
 * whose product with the position wraps, which leaves them within 2^-31 of a turn (for
 * frequencies of a few radians); sine and cosine are taken in fp32 of an angle that is
 * rounded to 24 bits within an eighth of a turn, 2^-28 of a turn at most.
 * rot_dim even, 2 <= rot_dim, start >= 0, start + rot_dim <= dim <= 65536. */
int indexer_rotary(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                   const int32_t* positions, const double* freqs, int32_t dtype, int64_t tokens,
                   int32_t heads, int32_t dim, int32_t rot_dim, int32_t start, int32_t layout,
                   float scale, int32_t transpose, void* out, int64_t out_token_stride,
                   int64_t out_head_stride, cudaStream_t stream);

/* The same with positions on several axes (time, height and width of images and video):
 * pair i turns by positions[axes[i]][t] * freqs[i]. positions [num_axes, tokens] int32, the
 * axes position_axis_stride elements apart (0: one row for all axes); axes [rot_dim / 2]
 * int32. An axis outside [0, num_axes): its pair turns as at position 0 (it is multiplied by
 * `scale` alone), and is counted. num_axes >= 1. */
int indexer_rotary_axes(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                        const int32_t* positions, int64_t position_axis_stride, int32_t num_axes,
                        const int32_t* axes, const double* freqs, int32_t dtype, int64_t tokens,
                        int32_t heads, int32_t dim, int32_t rot_dim, int32_t start, int32_t layout,
                        float scale, int32_t transpose, void* out, int64_t out_token_stride,
                        int64_t out_head_stride, cudaStream_t stream);

/* Layer norm over the last axis. x [tokens, heads, dim] of `dtype` (unit column stride, token
 * and head strides in elements, 0 allowed), weight and bias (may be NULL) [dim] of
 * `param_dtype`, out [tokens, heads, dim] of `dtype`, contiguous, not overlapping x:
 *   out = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(mean((x - mean)^2) + eps),
 * computed in fp32 (the variance of the differences from the mean) and rounded once. stats
 * (may be NULL) [tokens * heads, 2] fp32, 8-byte aligned, receives mean and rstd for the
 * gradient. A row that holds an infinity or a NaN becomes NaN. 1 <= dim <= 65536, eps >= 0. */
int indexer_layer_norm(const void* x, int64_t x_token_stride, int64_t x_head_stride, int32_t dtype,
                       int64_t tokens, int32_t heads, int32_t dim, const void* weight,
                       const void* bias, int32_t param_dtype, float eps, void* out, float* stats,
                       cudaStream_t stream);

/* Its gradients. grad [tokens, heads, dim] of `dtype` (strides as x's); stats as written
 * above. grad_x [tokens, heads, dim] of `dtype`, contiguous; grad_weight and grad_bias [dim]
 * of `param_dtype`; each may be NULL. With g = grad * weight and n = (x - mean) * rstd:
 *   grad_x = rstd * (g - mean(g) - n * mean(g n)),  grad_weight = sum grad * n,
 *   grad_bias = sum grad,
 * sums in fp32, in an order that depends on the sizes and the device alone. Where grad_weight
 * or grad_bias is wanted, workspace needs indexer_layer_norm_grad_workspace_bytes of the
 * current device (16-byte aligned), and a second kernel adds up what the first one left there. */
int indexer_layer_norm_grad(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                            const void* grad, int64_t grad_token_stride, int64_t grad_head_stride,
                            int32_t dtype, int64_t tokens, int32_t heads, int32_t dim,
                            const void* weight, int32_t param_dtype, const float* stats, void* grad_x,
                            void* grad_weight, void* grad_bias, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream);
size_t indexer_layer_norm_grad_workspace_bytes(int64_t tokens, int32_t heads, int32_t dim);

/* Rows to e4m3. x [tokens, heads, dim] of `dtype` (unit column stride, token and head
 * strides in elements), codes [tokens, heads, dim] and scales [tokens, heads,
 * ceil(dim / 128)], both contiguous. For each block of 128 columns (the last one may be
 * shorter): amax = max(largest |x|, 2^-64); scale by `scale_format`; code = x / scale (the
 * real quotient) rounded to the nearest e4m3 value, ties to even. A block that holds an
 * infinity or a NaN gets the scale NaN and NaN codes throughout.
 * weights (may be NULL; needs dim <= 128): [tokens, heads] fp32; scales then receives
 * weights * scale, what indexer_scores takes as its weights. 1 <= dim <= 65536. */
int indexer_quantise(const void* x, int64_t x_token_stride, int64_t x_head_stride, int32_t dtype,
                     int64_t tokens, int32_t heads, int32_t dim, int32_t scale_format,
                     const float* weights, uint8_t* codes, float* scales, cudaStream_t stream);

/* Rows into a cache: row t of x [tokens, cache->dim] is quantised as above and written at
 * slots[t] (int32). Slot -1: the row is not written. Any other slot outside the cache:
 * not written, and counted. Of rows with one slot, any one is written, code by code and
 * scale by scale: give each row its own. */
int indexer_cache_write(const void* x, int64_t x_token_stride, int32_t dtype, int64_t tokens,
                        const int32_t* slots, int32_t scale_format, const indexer_cache_t* cache,
                        cudaStream_t stream);

/* Rows out of a cache: out [rows, cache->dim] of `dtype` (contiguous) receives
 * code * scale, an fp32 product rounded to `dtype` (past its range: infinity), of the row
 * at slots[i] (int32). Slot -1: zeros. Any other slot outside the cache: zeros, and counted. */
int indexer_cache_read(const indexer_cache_t* cache, const int32_t* slots, int64_t rows,
                       int32_t dtype, void* out, cudaStream_t stream);

/* Scores of queries against a paged cache of keys (cache->dim = 128). q [batch, queries,
 * heads, 128] e4m3 and weights [batch, queries, heads] fp32 (the scale of q's block folded
 * in), contiguous; page_table [batch, page_table_stride] int32, of which the first
 * ceil(row_len / page_size) entries of a row are used; seq_lens [batch, queries] int32;
 * out [batch * queries, row_len] fp32, 4-byte aligned:
 *   out[b*queries + n][j] = scale_j * sum_h weights[b,n,h] * max(q[b,n,h] . k_j, 0)
 * for j < clamp(seq_lens[b,n], 0, row_len), k_j being the row at page
 * page_table[b][j / page_size], offset j % page_size; -inf for the other j. Products are
 * exact, sums are held in fp32. A NaN scale or weight makes its scores NaN (a block with
 * a value that is not finite has one); a NaN code on its own counts as a product of 0.
 * A page id outside [0, num_pages): its positions' scores are -inf, and each is counted
 * at least once. Scores around a wait that ran out are NaN (never, unless there is a bug;
 * it is counted).
 * Needs 1 <= heads <= 128, row_len >= 1, and codes (pointer and strides) and q aligned to
 * 16 bytes. */
int indexer_scores(const uint8_t* q, const float* weights, const indexer_cache_t* cache,
                   const int32_t* page_table, int64_t page_table_stride, const int32_t* seq_lens,
                   int32_t batch, int32_t queries, int32_t heads, int64_t row_len, float* out,
                   cudaStream_t stream);

/* Rows appended to a block-scaled cache. x [tokens, cache->heads, cache->dim] of `dtype` (unit
 * column stride, token and head strides in elements); sequence b's rows are
 * [starts[b], starts[b+1]) of x (starts [batch + 1] int32, from 0 to tokens, not decreasing)
 * and become its last ones: of seq_lens[b] (int32, with the new rows) positions,
 * position j at page page_table[b][j / page_size] (int32 [batch, table_pages], rows
 * page_table_stride apart), offset j % page_size. Rows of x behind the last sequence's are
 * not read.
 * The scale of each block that gets rows, for each head: the smallest power of two >=
 * amax / 448 with amax = max(largest |x| of the new rows, 2^-64), and at least the block's
 * scale so far where the block has positions before the new rows. Codes: x / scale rounded to
 * the nearest e4m3 value, ties to even; where a scale has grown, the block's older codes become
 * code * old / new, rounded so too. New rows with an infinity or a NaN make the block's scale
 * and its codes NaN. Positions of the block behind the last new row are not touched.
 * A sequence whose rows do not lie in x, or whose positions not in [0, table_pages *
 * page_size): nothing is written for it, and it is counted (starts that decrease may also keep
 * other sequences from being written). A page id outside the cache: its rows are not
 * written, and it is counted. Two sequences that append must not share the block they append
 * to, and the pages that one sequence appends to must differ (otherwise one of the rows that
 * meet, or parts of several, are in the cache). tokens <= 2^30, batch <= 2^28. */
int indexer_cache_append(const void* x, int64_t x_token_stride, int64_t x_head_stride, int32_t dtype,
                         int64_t tokens, const int32_t* starts, const int32_t* seq_lens,
                         const int32_t* page_table, int64_t page_table_stride, int64_t table_pages,
                         int32_t batch, const indexer_block_cache_t* cache, cudaStream_t stream);

/* Attention over block-scaled caches of keys and values (as many pages, page_size, heads and
 * dim in both, heads of INDEXER_MAX_HEAD_DIM columns at most: not rows of an indexer_cache_t, with
 * a scale for each 128 columns, nor one latent row that is key and value at once; read such rows
 * back with indexer_cache_read). q [batch, queries, heads, dim] of `dtype` (bf16 or fp16), contiguous, 16-byte
 * aligned, heads a multiple of the caches' (query head h reads their head
 * h / (heads / cache heads)); out like q. For query (b, n) and the set J of positions it sees:
 *   out = sum_J p_j v_j / sum_J p_j,  p_j = exp(softmax_scale * q . k_j)
 * and zeros where J is empty. lse (may be NULL) [batch, queries, heads] fp32 receives
 * log(sum_J p_j), -inf where J is empty.
 * Whole sequences (seq_lens not NULL): index is the page table, int32 [batch, width], rows
 * index_stride apart; J = { j < seq_lens[b][n] } (int32 [batch, queries], clamped to
 * [0, width * page_size]). Picked rows (seq_lens NULL): index [batch * queries, width] int32 has
 * the slots that each query sees, as topk_transform_paged writes them; -1 is none, and a
 * slot that is there twice counts twice. A page id or slot outside the cache: its
 * positions are left out, and it is counted.
 * Values of q count to within 2^-17 of their row's largest one (or of 2^-112, where that is
 * larger); products with codes are exact, sums and the softmax in fp32. For their products with
 * the values' codes the weights p_j (with the values' scales) are rounded to 11 bits, or to 2^-32
 * of the row's largest one where that is coarser; from 65 query rows on a head of the cache on
 * (heads of 80 to 128 columns) some are rounded so twice. A key whose p_j * scale lies below
 * 2^-133 of the row's largest adds to neither sum: values' scales that lie within 2^100 of each
 * other lose none that counts. The split of the work depends on the sizes, the lengths and the
 * device: the same call gives the same bits, another batch around a query may change its last
 * ones.
 * Scales of values are taken as at least 2^-100 (a negative one too), and keys that no query
 * sees may hold anything. For the queries that see the key, a NaN code of a value makes its
 * column NaN, however little the key weighs, and nothing else; a NaN among a key's codes or the
 * key's or value's scales makes the row NaN, and its lse.
 * workspace: indexer_attention_workspace_bytes of the current device, 16-byte aligned; the call
 * enqueues two kernels. */
int indexer_attention(const void* q, int32_t dtype, const indexer_block_cache_t* keys,
                      const indexer_block_cache_t* values, const int32_t* index,
                      int64_t index_stride, int64_t width, const int32_t* seq_lens, int32_t batch,
                      int32_t queries, int32_t heads, float softmax_scale, void* out, float* lse,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream);
size_t indexer_attention_workspace_bytes(int32_t queries, int32_t heads, int32_t cache_heads,
                                         int32_t dim, int32_t picked);

/* Slots and page ids outside the cache, sequences that do not fit (indexer_cache_append) and
 * axes outside the positions, met on the current device since the last reset (each at least
 * once), and kernels' waits that ran out (never, unless there is a bug: the scores or outputs
 * concerned are NaN then). Both wait for all of the device's pending work. */
int indexer_guard_hits(uint64_t* hits);
int indexer_reset_guard_hits(void);

/* For tests (process-wide; returns the previous value): later calls of indexer_scores act as
 * if a wait of every CTA had run out (1) or its shared memory were not aligned (2): scores
 * are NaN, and are counted in indexer_guard_hits. Anything else: 0, no failure. */
int indexer_set_scores_failure(int mode);

/* The same for indexer_attention's kernel of more than 32 query rows on the same keys (rows of
 * 80 to 128 columns), the one that waits: 1, its outputs are NaN, and counted. */
int indexer_set_attention_failure(int mode);

#ifdef __cplusplus
}
#endif

#endif /* INDEXER_OPS_H_ */
