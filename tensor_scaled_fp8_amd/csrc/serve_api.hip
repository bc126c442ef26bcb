// C-ABI entry points of the serving operators: argument checks, then kernel
// launches on the caller's stream. No allocation, no host synchronisation.
#include "cache.h"
#include "fp4.h"
#include "serve_overlap.h"

using namespace fp8lin;

namespace {

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline fp8_status hip_status(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_HIP; }

inline bool cache_sizes(int64_t pages, int page_tokens, int heads, int head_dim) {
  return pages >= 0 && pages < ((int64_t)1 << 31) && page_tokens >= kTok && page_tokens <= 4096 &&
         (page_tokens & (page_tokens - 1)) == 0 && heads > 0 && heads <= 1024 &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256);
}
inline bool cache_ok(const fp8_cache* c) {
  return c && cache_sizes(c->pages, c->page_tokens, c->heads, c->head_dim) && aligned(c->k, 16) && aligned(c->v, 16) &&
         aligned(c->scales, 16) && (c->pages == 0 || (c->k && c->v && c->scales));
}
// Rows of one call: fewer than 2^31 of them, and of workgroups that take them
constexpr int64_t kMaxTokens = (int64_t)1 << 26, kMaxSequences = (int64_t)1 << 20;
inline bool batch_ok(const fp8_cache_batch* b) {
  if (!b || b->sequences < 0 || b->tokens < 0 || b->table_pages < 0 || b->ld_tables < 0) return false;
  if (!b->starts && b->tokens != b->sequences) return false;
  return b->sequences == 0 || (b->lengths && aligned(b->lengths, 4) && aligned(b->starts, 4) && aligned(b->tables, 4) &&
                               (b->table_pages == 0 || b->tables));
}
inline bool batch_fits(const fp8_cache_batch* b) {
  return b->tokens <= kMaxTokens && b->sequences <= kMaxSequences && b->table_pages < ((int64_t)1 << 31);
}
inline bool rows_ok(const fp8_cache_rows* r, int64_t tokens) { return r && aligned(r->p, 2) && (tokens == 0 || r->p); }

Cache cache_of(const fp8_cache* c) {
  return {c->k, c->v, c->scales, c->pages, __builtin_ctz((unsigned)c->page_tokens), c->heads};
}
CacheBatch batch_of(const fp8_cache_batch* b) {
  return {b->tables, b->ld_tables, b->table_pages, b->lengths, b->starts, (int)b->sequences, (int)b->tokens};
}
CacheRows rows_of(const fp8_cache_rows* r) { return {(uint16_t*)r->p, r->token_stride, r->head_stride}; }
RowSet set_of(const fp8_cache_rows* r, int64_t tokens, int heads, int head_dim) {
  return {r->p, tokens, heads, head_dim, r->token_stride, r->head_stride};
}
// out is written while in is read: it is in itself or lies apart, and its own rows do
inline bool rows_apart(const RowSet& out, const RowSet& in) {
  return !overlaps_itself(out) && (same_rows(out, in) || !overlap(out, in));
}
inline bool q_heads_ok(int q_heads, int heads) { return q_heads > 0 && q_heads <= 16384 && q_heads % heads == 0; }

CacheAttend attend_of(const fp8_cache* c, const fp8_cache_batch* b, int q_heads) {
  CacheAttend a = {};
  a.c = cache_of(c);
  a.b = batch_of(b);
  a.q_heads = q_heads;
  a.group = q_heads / c->heads;
  return a;
}
// its rows are counted with 31 bits
inline bool attend_fits(const fp8_cache_batch* b, int q_heads) {
  return batch_fits(b) && (b->tokens + 64 * b->sequences) * q_heads < ((int64_t)1 << 31) - 64;
}

inline bool fp4_sizes(int64_t K, int64_t N) { return K >= 0 && N >= 0; }
inline bool fp4_fits(int64_t K, int64_t N) { return K <= (1 << 20) && N <= ((int64_t)1 << 23); }
// X's blocks of 16 rows by 128 are counted with 31 bits
inline bool fp4_rows_fit(int64_t M, int64_t K) {
  return M <= (1 << 22) && (M + 15) / 16 * fp4_xblocks(K) < ((int64_t)1 << 31);
}
// and so are the product's tiles
inline bool fp4_product_fits(int64_t M, int64_t N) { return (M / 64 + 1) * (N / 64 + 1) < ((int64_t)1 << 31); }
struct Fp4Scratch {
  Fp4X x;
  size_t bytes;
  Fp4Scratch(void* p, int64_t M, int64_t K) {
    const size_t codes = fp4_x_codes(M, K);  // a multiple of 2048
    x = {(uint8_t*)p, p ? (uint8_t*)p + codes : nullptr, M, K};
    bytes = codes + fp4_x_scales(M, K);
  }
};

}  // namespace

extern "C" {

size_t fp8_cache_codes_bytes(int64_t pages, int page_tokens, int heads, int head_dim) {
  return cache_sizes(pages, page_tokens, heads, head_dim) ? (size_t)pages * page_tokens * heads * head_dim : 0;
}
size_t fp8_cache_scales_bytes(int64_t pages, int page_tokens, int heads, int head_dim) {
  return cache_sizes(pages, page_tokens, heads, head_dim) ? (size_t)pages * (page_tokens / kTok) * heads * 2 : 0;
}

fp8_status fp8_cache_append(const fp8_cache* cache, const fp8_cache_batch* batch, const fp8_cache_rows* k,
                            const fp8_cache_rows* v, const fp8_cache_rows* q, const fp8_cache_rows* q_out, int q_heads,
                            const float* freqs, int rot, int interleaved, hipStream_t stream) {
  if (!cache_ok(cache) || !batch_ok(batch) || !rows_ok(k, batch->tokens) || !rows_ok(v, batch->tokens))
    return FP8_ERR_INVALID;
  const bool with_q = q && q->p;
  if (with_q && (!rows_ok(q, batch->tokens) || !rows_ok(q_out, batch->tokens) || !q_heads_ok(q_heads, cache->heads)))
    return FP8_ERR_INVALID;
  if (rot < 0 || rot % 16 || rot > cache->head_dim || (rot && (!freqs || !aligned(freqs, 4)))) return FP8_ERR_INVALID;
  if (!batch_fits(batch)) return FP8_ERR_UNSUPPORTED;
  if (with_q) {
    const RowSet out = set_of(q_out, batch->tokens, q_heads, cache->head_dim);
    if (!rows_apart(out, set_of(q, batch->tokens, q_heads, cache->head_dim)) ||
        overlap(out, set_of(k, batch->tokens, cache->heads, cache->head_dim)) ||
        overlap(out, set_of(v, batch->tokens, cache->heads, cache->head_dim)))
      return FP8_ERR_INVALID;
  }
  CacheAppend a = {cache_of(cache), batch_of(batch), rows_of(k), rows_of(v), {nullptr, 0, 0}, {nullptr, 0, 0}, 0, rot,
                   interleaved != 0, freqs};
  if (with_q) {
    a.q = rows_of(q);
    a.qo = rows_of(q_out);
    a.q_heads = q_heads;
  }
  return hip_status(launch_cache_append(a, cache->head_dim, stream));
}

fp8_status fp8_cache_read(const fp8_cache* cache, const fp8_cache_batch* batch, const fp8_cache_rows* k,
                          const fp8_cache_rows* v, hipStream_t stream) {
  if (!cache_ok(cache) || !batch_ok(batch) || !rows_ok(k, batch->tokens) || !rows_ok(v, batch->tokens))
    return FP8_ERR_INVALID;
  if (!batch_fits(batch)) return FP8_ERR_UNSUPPORTED;
  const RowSet rk = set_of(k, batch->tokens, cache->heads, cache->head_dim);
  const RowSet rv = set_of(v, batch->tokens, cache->heads, cache->head_dim);
  if (overlaps_itself(rk) || overlaps_itself(rv) || overlap(rk, rv)) return FP8_ERR_INVALID;
  return hip_status(launch_cache_read(cache_of(cache), batch_of(batch), rows_of(k), rows_of(v), cache->head_dim, stream));
}

size_t fp8_cache_attention_workspace_bytes(const fp8_cache* cache, const fp8_cache_batch* batch, int q_heads) {
  if (!cache || !cache_sizes(cache->pages, cache->page_tokens, cache->heads, cache->head_dim) || !batch ||
      batch->tokens < 0 || batch->sequences < 0 || !q_heads_ok(q_heads, cache->heads) || !attend_fits(batch, q_heads))
    return 0;
  return cache_attention_ws_bytes(attend_of(cache, batch, q_heads), cache->head_dim);
}

fp8_status fp8_cache_attention_plan(const fp8_cache* cache, const fp8_cache_batch* batch, int q_heads, int* rows, int* form) {
  if (!cache || !cache_sizes(cache->pages, cache->page_tokens, cache->heads, cache->head_dim) || !batch ||
      batch->tokens < 0 || batch->sequences < 0 || !q_heads_ok(q_heads, cache->heads) || !rows || !form)
    return FP8_ERR_INVALID;
  if (!attend_fits(batch, q_heads)) return FP8_ERR_UNSUPPORTED;
  cache_attention_plan(attend_of(cache, batch, q_heads), cache->head_dim, rows, form);
  return FP8_OK;
}

fp8_status fp8_cache_attention(const fp8_cache* cache, const fp8_cache_batch* batch, const fp8_cache_rows* q, int q_heads,
                               float scale, float softcap, int window, const fp8_cache_rows* out, float* lse, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
  if (!cache_ok(cache) || !batch_ok(batch) || !rows_ok(q, batch->tokens) || !rows_ok(out, batch->tokens) ||
      !q_heads_ok(q_heads, cache->heads) || !(softcap == 0.0f || (softcap >= 0x1p-64f && softcap <= 0x1p64f)) || window < 0 ||
      !(__builtin_fabsf(scale) <= 0x1p64f) || !aligned(lse, 4) || !aligned(ws, 16))
    return FP8_ERR_INVALID;
  if (!attend_fits(batch, q_heads)) return FP8_ERR_UNSUPPORTED;
  if (!rows_apart(set_of(out, batch->tokens, q_heads, cache->head_dim), set_of(q, batch->tokens, q_heads, cache->head_dim)))
    return FP8_ERR_INVALID;
  CacheAttend a = attend_of(cache, batch, q_heads);
  a.q = rows_of(q);
  a.out = rows_of(out);
  a.lse = lse;
  a.scale = scale;
  a.cap = softcap;
  a.window = window;
  const size_t need = cache_attention_ws_bytes(a, cache->head_dim);
  if (need && (!ws || ws_bytes < need)) return FP8_ERR_INVALID;
  return hip_status(launch_cache_attention(a, cache->head_dim, ws, stream));
}

size_t fp4_codes_bytes(int64_t K, int64_t N) {
  return K <= 0 || N <= 0 || !fp4_fits(K, N) ? 0 : (size_t)((N + 15) / 16) * fp4_kblocks(K) * 1024;
}
size_t fp4_scales_bytes(int64_t K, int64_t N) { return fp4_codes_bytes(K, N) / 16; }

fp8_status fp4_quantize(const void* W, int64_t ldw, int64_t K, int64_t N, uint8_t* codes, uint8_t* scales,
                        hipStream_t stream) {
  if (!fp4_sizes(K, N) || ldw < 0 || !aligned(W, 2) || !aligned(codes, 16) || !aligned(scales, 16)) return FP8_ERR_INVALID;
  if (K && N && (!W || !codes || !scales)) return FP8_ERR_INVALID;
  if (!fp4_fits(K, N)) return FP8_ERR_UNSUPPORTED;
  return hip_status(launch_fp4_quantize((const uint16_t*)W, ldw, {codes, scales, K, N}, stream));
}

fp8_status fp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t N, void* W, int64_t ldw,
                          hipStream_t stream) {
  if (!fp4_sizes(K, N) || (K > 1 && ldw < N) || !aligned(W, 2) || !aligned(codes, 16) || !aligned(scales, 16))
    return FP8_ERR_INVALID;
  if (K && N && (!W || !codes || !scales)) return FP8_ERR_INVALID;
  if (!fp4_fits(K, N)) return FP8_ERR_UNSUPPORTED;
  return hip_status(launch_fp4_dequantize({(uint8_t*)codes, (uint8_t*)scales, K, N}, (uint16_t*)W, ldw, stream));
}

size_t fp4_linear_bytes(int64_t M, int64_t K, int64_t N) {
  if (M <= 0 || K <= 0 || N <= 0 || !fp4_fits(K, N) || !fp4_rows_fit(M, K) || fp4_fused(M, K)) return 0;
  return Fp4Scratch(nullptr, M, K).bytes;
}

fp8_status fp4_linear_plan(int64_t M, int64_t K, int64_t N, int exact, int* form, int* row_tiles, int* col_tiles, int* groups) {
  if (M < 0 || !fp4_sizes(K, N) || !form || !row_tiles || !col_tiles || !groups) return FP8_ERR_INVALID;
  if (!fp4_fits(K, N) || !fp4_rows_fit(M, K) || !fp4_product_fits(M, N)) return FP8_ERR_UNSUPPORTED;
  const Fp4Form f = fp4_form(M, K, N, exact != 0);
  *form = f.kind;
  *row_tiles = f.mf;
  *col_tiles = f.nb;
  *groups = f.groups;
  return FP8_OK;
}

fp8_status fp4_linear_fwd_cached(const void* X, int64_t ldx, int64_t M, int64_t K, int64_t N, const uint8_t* codes,
                                 const uint8_t* scales, int exact, void* scratch, size_t scratch_bytes, void* Y,
                                 hipStream_t stream) {
  if (M < 0 || !fp4_sizes(K, N) || ldx < 0 || !aligned(X, 2) || !aligned(codes, 16) || !aligned(scales, 16) ||
      !aligned(scratch, 16) || !aligned(Y, 2))
    return FP8_ERR_INVALID;
  if ((M && K && !X) || (K && N && (!codes || !scales)) || (M && N && !Y)) return FP8_ERR_INVALID;
  if (!fp4_fits(K, N) || !fp4_rows_fit(M, K) || !fp4_product_fits(M, N)) return FP8_ERR_UNSUPPORTED;
  // X is read until the last workgroup ends
  const RowSet xs(X, M, 1, K, ldx, 0), ys(Y, M, 1, N, N, 0);
  if (!xs.empty() && !ys.empty() && xs.lo() < ys.hi() && ys.lo() < xs.hi()) return FP8_ERR_INVALID;
  const size_t need = fp4_linear_bytes(M, K, N);
  if (need && (!scratch || scratch_bytes < need)) return FP8_ERR_INVALID;
  const Bf16Mat x = {(const uint16_t*)X, ldx, M, K};
  const Fp4Mat w = {(uint8_t*)codes, (uint8_t*)scales, K, N};
  if (K == 0) return hip_status(launch_fp4_zero((uint16_t*)Y, M * N, stream));
  if (fp4_fused(M, K)) return hip_status(launch_fp4_fused(x, w, (uint16_t*)Y, stream));
  const Fp4Scratch s(scratch, M, K);
  const hipError_t e = launch_fp4_x(x, s.x, stream);
  if (e != hipSuccess) return FP8_ERR_HIP;
  return hip_status(launch_fp4_linear(s.x, w, (uint16_t*)Y, exact != 0, stream));
}

}  // extern "C"
