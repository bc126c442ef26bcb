// Shared declarations of the paged 8-bit cache (cache_*.hip).
//
// A block is 16 tokens of one head, with one scale for its keys and one for
// its values. Its codes are laid out as the attention's matrix instructions
// take them, so that a wave's 64 lanes load a block by 16 contiguous bytes
// each and use them as they come:
//   keys    lane 16 q + t of piece p: token t, elements 64 p + 16 q ..+15 (a
//           row of A for two 16x16x32 products, reduced over elements);
//   values  lane 16 q + r of piece p: tokens 4 q ..+3 of each of the elements
//           w r + 4 p ..+3 (w = D / 16): element w r + i is row r of the i-th
//           16-row tile of A, reduced over tokens. The weights come out of
//           the first product with tokens 4 q ..+3 in lane group q.
#pragma once

#include "block_quant.h"
#include "fp8lin_serve.h"

namespace fp8lin {

constexpr int kTok = 16;  // tokens of a block

struct Cache {
  uint8_t *k, *v, *scales;
  int64_t pages;
  int shift, heads;  // a page holds 2^shift tokens
};
struct CacheBatch {
  const int32_t* tables;
  int64_t ld, table_pages;
  const int32_t *lengths, *starts;
  int sequences, tokens;
};
// [tokens, heads, D] bf16, strides in elements
struct CacheRows {
  uint16_t* p;
  int64_t tok, head;
};

// rows of sequence i in the packed tensors: within [0, tokens] whatever starts holds
__device__ inline int start_of(const CacheBatch& b, int i) {
  if (!b.starts) return i;
  const int s = b.starts[i];
  return s < 0 ? 0 : s < b.tokens ? s : b.tokens;
}
struct Seq {
  int row0, n;   // its rows
  int64_t p0;    // the first one's position
};
__device__ inline Seq seq_of(const CacheBatch& b, int i) {
  Seq s;
  s.row0 = start_of(b, i);
  const int e = b.starts ? start_of(b, i + 1) : i + 1;
  s.n = e > s.row0 ? e - s.row0 : 0;
  const int len = b.lengths[i];
  s.p0 = (int64_t)(len > 0 ? len : 0) - s.n;
  return s;
}
// The largest i with first(i) <= v, of a first that does not decrease from first(0) <= v.
template <typename F>
__device__ inline int last_upto(int n, int64_t v, F first) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (first(m) <= v) lo = m;
    else hi = m;
  }
  return lo;
}
// Number of the block of head h at position pos of sequence i (a multiple of 16); -1: not there
__device__ inline int64_t block_at(const Cache& c, const CacheBatch& b, int i, int64_t pos, int h) {
  if (pos < 0) return -1;
  const int64_t t = pos >> c.shift;
  if (t >= b.table_pages) return -1;
  const int64_t page = b.tables[i * b.ld + t];
  if (page < 0 || page >= c.pages) return -1;
  const int in = (int)(pos & ((1 << c.shift) - 1)) >> 4;
  return ((page * c.heads + h) << (c.shift - 4)) + in;
}

struct CacheAppend {
  Cache c;
  CacheBatch b;
  CacheRows k, v, q, qo;
  int q_heads, rot, interleaved;
  const float* freqs;
};
hipError_t launch_cache_append(const CacheAppend& a, int head_dim, hipStream_t st);
hipError_t launch_cache_read(const Cache& c, const CacheBatch& b, const CacheRows& k, const CacheRows& v, int head_dim,
                             hipStream_t st);

struct CacheAttend {
  Cache c;
  CacheBatch b;
  CacheRows q, out;
  float* lse;
  int q_heads, group;  // query heads; of each key head
  float scale, cap;
  int window;
};
size_t cache_attention_ws_bytes(const CacheAttend& a, int head_dim);
void cache_attention_plan(const CacheAttend& a, int head_dim, int* rows, int* form);
hipError_t launch_cache_attention(const CacheAttend& a, int head_dim, void* ws, hipStream_t st);

}  // namespace fp8lin
