/*
 * fp8lin_serve.h - C ABI of the serving operators of an attention layer
 * (libfp8lin.so, with fp8lin.h): a paged key/value cache in 8 bits, the
 * attention that reads it, and the linear on 4-bit weights.
 *
 * As in fp8lin.h: plain device pointers and sizes, the caller owns all
 * memory, errors are status codes, work goes to the caller's stream of the
 * current device, nothing is allocated and nothing waits. Calls with equal
 * arguments give equal bits.
 *
 * An output is read or written by others of the same launch in no order, so
 * it may share memory with an input only where this is said below, and then
 * has to be that input, row for row: packed rows that overlap otherwise (an
 * output's own, too) are FP8_ERR_INVALID. Views of one tensor with the same
 * strides are told apart element by element, others by whether their tokens
 * lie beside each other.
 */
#ifndef FP8LIN_SERVE_H
#define FP8LIN_SERVE_H

#include "fp8lin.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ---- The paged cache ----
 *
 * Keys and values of `heads` heads of head_dim elements, in E4M3, with a
 * power-of-two scale for each block of 16 consecutive tokens and each head,
 * for keys and for values:
 *   value = code * 2^-bias, scale byte = 127 - bias.
 * A page holds page_tokens tokens (a power of two, 16 .. 4096); head_dim is
 * 64, 128 or 256. Block b of head h of page p is block number
 * n = (p heads + h) page_tokens / 16 + b. It has
 *   k       16 head_dim bytes at k + n 16 head_dim: element d of token t at
 *           1024 (d / 64) + 256 (d % 64 / 16) + 16 t + d % 16;
 *   v       as many at v + n 16 head_dim: element d of token t, with
 *           w = head_dim / 16, at 1024 (d % w / 4) + 256 (t / 4) +
 *           16 (d / w) + 4 (d % 4) + t % 4;
 *   scales  bytes 2 n (keys) and 2 n + 1 (values).
 * All three are 16-B aligned and zero before the first append.
 *
 * A batch: sequence i has lengths[i] tokens, and the call's n_i tokens of it
 * are the last ones, at positions lengths[i] - n_i .. lengths[i] - 1. They
 * are rows starts[i] .. starts[i + 1] - 1 of the call's packed tensors of
 * `tokens` rows (starts: [sequences + 1], not decreasing; NULL: one row a
 * sequence). Rows behind starts[sequences] are neither read nor written.
 * Position p of sequence i lies in page tables[i * ld_tables + p /
 * page_tokens]. A position below 0, past the table's table_pages entries, or
 * whose entry is no page (negative, or pages and above) is not there (a
 * negative length counts as 0):
 * nothing is stored for it, it is read as zeros, and attention does not see
 * it. So a padded sequence is one of length 0.
 * Sequences may share pages that none appends to; those of the call's own
 * tokens are each named once.
 */
typedef struct fp8_cache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* scales;
  int64_t pages;
  int32_t page_tokens, heads, head_dim;
} fp8_cache;

typedef struct fp8_cache_batch {
  const int32_t* tables;
  int64_t ld_tables, table_pages;
  const int32_t* lengths;
  const int32_t* starts; /* or NULL */
  int64_t sequences, tokens;
} fp8_cache_batch;

/* A packed bf16 tensor [tokens, heads, head_dim]: strides in elements, the
 * last one 1; 2-B aligned. */
typedef struct fp8_cache_rows {
  void* p;
  int64_t token_stride, head_stride;
} fp8_cache_rows;

/* Bytes of k (and of v), and of scales. 0 if the sizes are not valid. */
size_t fp8_cache_codes_bytes(int64_t pages, int page_tokens, int heads, int head_dim);
size_t fp8_cache_scales_bytes(int64_t pages, int page_tokens, int heads, int head_dim);

/*
 * Stores the batch's keys and values, and rotates on the way if rot > 0:
 * of the first rot dimensions (a multiple of 16, up to head_dim) of each
 * key and query, pairs (a, b) become
 *   (a cos t - b sin t, b cos t + a sin t), t = position * freqs[j],
 * j < rot / 2: elements (j, j + rot / 2), or (2 j, 2 j + 1) if interleaved.
 * Angles, and keys up to their codes, are computed in 64 bits (sin and cos
 * at far positions; codes are the nearest to the rotated key itself).
 * Queries, if q.p is not NULL, go rotated to q_out (any strides; it may be
 * q itself, and overlap no other input), rounded to bf16, of q_heads heads; with rot = 0 they are copied.
 * Scales: for a block's new tokens, over its finite values,
 *   need = floor(log2(448 / max |x|)), clamped to [-126, 126]; 126 if all
 *          are 0; at most 0 if one is infinite;
 *   bias = need if the block's first token is among them, else the smaller
 *          of need and the bias held,
 *   code = e4m3(clamp(x 2^bias)) to nearest even (NaN stays NaN), clamped to
 *          448, and to 240 for bias -120, the least that a value asks for:
 *          what is held is finite in bf16;
 * where the bias held falls, the codes of the block's earlier tokens are
 * rounded anew, exactly but for those that leave the normal range. Later
 * codes of the block are left as they were.
 */
fp8_status fp8_cache_append(const fp8_cache* cache, const fp8_cache_batch* batch, const fp8_cache_rows* k,
                            const fp8_cache_rows* v, const fp8_cache_rows* q, const fp8_cache_rows* q_out, int q_heads,
                            const float* freqs, int rot, int interleaved, hipStream_t stream);

/* The values of the batch's tokens as the cache holds them, to bf16 (exact
 * within its normal range). k and v may not overlap. */
fp8_status fp8_cache_read(const fp8_cache* cache, const fp8_cache_batch* batch, const fp8_cache_rows* k,
                          const fp8_cache_rows* v, hipStream_t stream);

/*
 * Attention of the batch's queries over the cache, which holds the batch's
 * own tokens already. The query at position p sees positions j <= p, and
 * j > p - window if window > 0. Query head a reads head a / (q_heads /
 * heads) of the cache.
 *   s = scale q . k, |scale| <= 2^64;
 *   if softcap > 0 (2^-64 .. 2^64): s = softcap tanh(s / softcap);
 *   out = sum over the seen of softmax(s) v,  lse = log(sum of exp(s)).
 * Where nothing is seen, or only scores of -inf, out is 0 and lse -inf.
 * Positions from 2^31 - 256 on are not seen. out may be q itself. Keys
 * and values enter the products exactly, sums and the softmax are 32-bit, out
 * is bf16 (any strides), lse fp32 [tokens, q_heads] or NULL. Weights enter as
 * two bf16 each, 2^-17 off, so that out is as far off as its own rounding;
 * in FP8_CACHE_TILES and _ROWS, the forms of batches of many rows, which wait
 * for the products and not for memory, as one, 2^-9 off. The form is the whole
 * batch's, by its mean rows: a decoded token beside a prompt's chunk is
 * computed like the chunk, and much slower over a long context than in a call
 * of its own. lse is the 32-bit weights' in every form. Products beyond the
 * 32-bit range count as infinite. A NaN in a key or value reaches the queries
 * that see it and no others.
 *   ws: fp8_cache_attention_workspace_bytes of the same cache and batch
 *   (their sizes alone count), 16-B aligned; it holds nothing between calls.
 */
size_t fp8_cache_attention_workspace_bytes(const fp8_cache* cache, const fp8_cache_batch* batch, int q_heads);
/* The rows (queries of one key head) that are computed together, and how the
 * work is cut, by the sizes alone. For profiles and tests; 0 and 0 of an empty
 * batch. */
#define FP8_CACHE_SHARES 0 /* equal shares of all tokens a workgroup */
#define FP8_CACHE_TILES 1  /* a tile of rows a workgroup */
#define FP8_CACHE_ROWS 2   /* a tile of rows a wave */
fp8_status fp8_cache_attention_plan(const fp8_cache* cache, const fp8_cache_batch* batch, int q_heads, int* rows, int* form);
fp8_status fp8_cache_attention(const fp8_cache* cache, const fp8_cache_batch* batch, const fp8_cache_rows* q, int q_heads,
                               float scale, float softcap, int window, const fp8_cache_rows* out, float* lse, void* ws,
                               size_t ws_bytes, hipStream_t stream);

/*
 * ---- 4-bit weights ----
 *
 * A weight W [K, N] in E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), with a
 * power-of-two scale for each group of 32 along K:
 *   bias = floor(log2(6 / max |w|)), clamped to [-126, 126]; 0 for a group
 *          that is all zero or holds an infinity,
 *   code = e2m1(clamp(w 2^bias)) to nearest even, value = code * 2^-bias.
 * The codes have no NaN: a group that holds one has scale byte 255 and is
 * NaN as a whole. Codes are stored for the matrix instructions: with N and K rounded up
 * (zero codes) to 16 and 512, for each 16 columns of W and each 128 of K
 * 1024 bytes; byte 256 (k % 128 / 32) + 16 (n % 16) + k % 32 / 2 holds k in
 * its low half for even k. Scale bytes 127 - bias follow the same order:
 * for each 16 columns and each 512 of K 256 bytes, byte
 * 64 (k % 128 / 32) + 4 (n % 16) + k % 512 / 128.
 */
size_t fp4_codes_bytes(int64_t K, int64_t N);
size_t fp4_scales_bytes(int64_t K, int64_t N);
/* The stored form of a bf16 W [K, N], row pitch ldw; codes and scales 16-B aligned. */
fp8_status fp4_quantize(const void* W_bf16, int64_t ldw, int64_t K, int64_t N, uint8_t* codes, uint8_t* scales,
                        hipStream_t stream);
/* Its values in bf16 (exact within its normal range, 2^128 an infinity), row pitch ldw. */
fp8_status fp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t N, void* W_bf16, int64_t ldw,
                          hipStream_t stream);
/* How a product is cut: the kernel, its wave's 16-row and 16-column tiles and
 * the groups of waves that share K. For profiles and tests. */
#define FP4_FUSED 0 /* X quantised by the product's launch */
#define FP4_FEW 1   /* few rows, X quantised before */
#define FP4_MANY 2
#define FP4_EXACT 3 /* many rows, exact products */
fp8_status fp4_linear_plan(int64_t M, int64_t K, int64_t N, int exact, int* form, int* row_tiles, int* col_tiles, int* groups);
/*
 * Y [M, N] (dense) = X [M, K] W on a stored 4-bit W. X is quantised as by
 * fp8_block_quantize (E4M3, a scale for each 128 of a row). exact: products
 * are exact and their sums 32-bit, for a Y that is rounded to 8 bits next.
 * Without it products of more than 32 rows are fp8_block_gemm's, up to twice
 * as fast and 1.5e-5 off, which a bf16 Y does not show; of fewer they are
 * exact all the same. Y does not overlap X. scratch: fp4_linear_bytes (0: none
 * is needed).
 */
size_t fp4_linear_bytes(int64_t M, int64_t K, int64_t N);
fp8_status fp4_linear_fwd_cached(const void* X_bf16, int64_t ldx, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                                 const uint8_t* scales, int exact, void* scratch, size_t scratch_bytes,
                                 void* Y_bf16, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8LIN_SERVE_H */
