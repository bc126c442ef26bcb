// Which calls would write what they still read, on the host: workgroups of one
// launch read and write a packed tensor's rows in no order, so an output may
// share memory with an input only where each row is read and written by the
// same wave: where it is that input.
#pragma once

#include <cstdint>

namespace fp8lin {

// Rows of d elements of 2 bytes: row (i, j) of n x heads at p + i tok + j head
struct RowSet {
  intptr_t p;  // in elements
  int64_t n, heads, d, tok, head;
  RowSet(const void* at, int64_t n_, int64_t heads_, int64_t d_, int64_t tok_, int64_t head_)
      : p((intptr_t)at / 2), n(n_), heads(heads_), d(d_), tok(n_ > 1 ? tok_ : 0), head(heads_ > 1 ? head_ : 0) {}
  bool empty() const { return n <= 0 || heads <= 0 || d <= 0; }
  // first element and one past the last, of a token's rows and of all
  __int128 token_lo() const { return (__int128)p + (head < 0 ? (__int128)(heads - 1) * head : 0); }
  __int128 token_hi() const { return (__int128)p + (head > 0 ? (__int128)(heads - 1) * head : 0) + d; }
  __int128 lo() const { return token_lo() + (tok < 0 ? (__int128)(n - 1) * tok : 0); }
  __int128 hi() const { return token_hi() + (tok > 0 ? (__int128)(n - 1) * tok : 0); }
};

// Whether some x + i step, from <= i <= to, lies within (-d, d)
inline bool comes_near(__int128 x, int64_t step, int64_t from, int64_t to, int64_t d) {
  const auto at = [&](__int128 i) {
    const __int128 v = x + (i < from ? from : i > to ? to : i) * step;
    return v > -d && v < d;
  };
  if (step == 0) return at(0);
  const __int128 i = -x / step;  // the least |v| is next to it
  return at(i - 1) || at(i) || at(i + 1);
}

// Two rows of r share an element
inline bool overlaps_itself(const RowSet& r) {
  if (r.empty()) return false;
  if (r.n > 1 && comes_near(0, r.tok, 1, r.n - 1, r.d)) return true;
  if (r.heads > 1 && comes_near(0, r.head, 1, r.heads - 1, r.d)) return true;
  if (r.n == 1 || r.heads == 1) return false;
  const __int128 t = r.tok < 0 ? -(__int128)r.tok : r.tok, h = r.head < 0 ? -(__int128)r.head : r.head;
  if (t >= (r.heads - 1) * h + r.d || h >= (r.n - 1) * t + r.d) return false;  // one dimension lies within the other
  for (int64_t j = 1; j < r.heads; ++j)
    if (comes_near((__int128)j * r.head, r.tok, 1 - r.n, r.n - 1, r.d)) return true;
  return false;
}

// A row of a and one of b (of the same d) share an element. Exact for rows of the same
// strides, as views of one projection have them; of different strides those
// are told apart whose tokens lie beside each other, or that lie apart as
// wholes, and others are taken to overlap.
inline bool overlap(RowSet a, RowSet b) {
  if (a.empty() || b.empty() || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  if (a.n == 1) a.tok = b.tok;
  if (b.n == 1) b.tok = a.tok;
  if (a.heads == 1) a.head = b.head;
  if (b.heads == 1) b.head = a.head;
  if (a.tok != b.tok) return true;
  if (a.tok) {
    const __int128 t = a.tok < 0 ? -(__int128)a.tok : a.tok;
    const __int128 m = ((b.token_lo() - a.token_lo()) % t + t) % t;
    if (m >= a.token_hi() - a.token_lo() && m + b.token_hi() - b.token_lo() <= t) return false;
  }
  if (a.head != b.head) return true;
  for (int64_t j = 1 - a.heads; j < b.heads; ++j)
    if (comes_near((__int128)b.p - a.p + (__int128)j * a.head, a.tok, 1 - a.n, b.n - 1, a.d)) return true;
  return false;
}

// The same rows at the same places
inline bool same_rows(const RowSet& a, const RowSet& b) {
  return a.p == b.p && a.n == b.n && a.heads == b.heads && a.d == b.d && a.tok == b.tok && a.head == b.head;
}

}  // namespace fp8lin
