// Attention over the paged 8-bit cache.
//
// A workgroup's tile is R = 16 MT rows of one key head, a row being one of
// the head's queries of one token, and a range of the tokens that they see;
// its waves share out the tokens, 32 (two blocks) at a time, each with a
// softmax of its own (running maximum, sum, weighted values), joined over LDS
// at the tile's end.
//   s^T [tokens, rows] = K Q^T and o^T [D, rows] += V^T p^T by 16x16x32 bf16
// products: K and V come as the first operand straight from memory (the
// cache holds them in its order), converted to bf16 by the instruction that
// applies the block's scale, exactly. The weights p^T leave the first product
// in the lanes that the second takes them from: lane group g has tokens
// 4 g ..+3 of both blocks.
//
// The running maximum moves only when a score exceeds it by 2^8: until then
// the weights are scaled by up to 2^8, which costs neither range nor
// precision, and no lane has to know of another's scores.
//
// FINE: a weight goes into the product as two bf16, its rounding and what
// that left (2^-17 of it): the outputs are then bf16's own rounding off and no
// more. It costs a second product of V and a third of the softmax, which a
// call that waits for the cache's bytes does not notice. Otherwise outputs are
// divided by the sum of the rounded weights, and LSE keeps the sum of the
// weights themselves beside it, for the logarithm alone: prompts of 31 to 250
// tokens 1.1e-6 off, by the sum of the rounded ones, 2^-9 off each, 0.0029. A
// call that asks for it pays with its VALU (prompts of 1501 to 6007 tokens:
// 704 us without, 770).
//
// Few rows (a decode batch): the work of all (sequence, tile, head) is one
// line of units of 128 tokens, cut into equal shares, one a workgroup, two or
// three a CU: whatever the lengths, all CUs end together.
// A tile cut by a share's end leaves its parts' sums in the workspace, and a
// second launch joins them. Many rows (prompts): one workgroup a tile; of
// still more, one wave a tile; the last tiles of a sequence, which see most,
// before its others. The host knows a batch's mean rows and no more, so one
// form takes all of it: a decoded token beside a prompt's chunk is one tile,
// walked to its end by one workgroup or wave, with weights in one bf16 (63
// tokens over 100 to 32768 and a chunk of 2048 over 4096, 64 query and 8 key
// heads: 1473 us, apart 150 and 218).
#include "cache.h"

namespace fp8lin {
namespace {

constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;

typedef __bf16 ca_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 ca_bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t ca_u32x4 __attribute__((ext_vector_type(4)));

__device__ inline uint32_t bf16_of2(uint32_t w, float s, bool hi) {
  return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))
            : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
}
// 8 codes, of two words with a scale each
__device__ inline ca_bf16x8 widen(uint32_t a, float sa, uint32_t b, float sb) {
  const ca_u32x4 r = {bf16_of2(a, sa, false), bf16_of2(a, sa, true), bf16_of2(b, sb, false), bf16_of2(b, sb, true)};
  return __builtin_bit_cast(ca_bf16x8, r);
}
// both bf16 of a word added (by way of a function's argument: the compiler
// takes a vector's first element for any that is cast in place)
__device__ inline float add2(uint32_t w, float l) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(ca_bf16x2, w), __builtin_bit_cast(ca_bf16x2, 0x3F803F80u), l, false);
}
__device__ inline bq_f32x4 mma(ca_bf16x8 a, ca_bf16x8 b, bq_f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float nan() { return __uint_as_float(0x7FC00000u); }

__device__ inline uint32_t high_half(uint32_t w) { return w & 0xFFFF0000u; }

__device__ inline float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// over the four lanes that share lane % 16
__device__ inline float quad_max(float a) {
  a = fmaxf(a, __shfl_xor(a, 16));
  return fmaxf(a, __shfl_xor(a, 32));
}
__device__ inline float quad_sum(float a) {
  a += __shfl_xor(a, 16);
  return a + __shfl_xor(a, 32);
}

// tanh by exp(2 x), near 0 by its series (up to x^9: 1e-8 of it at 1/4)
__device__ inline float tanh_(float x) {
  const float t = 1.0f - 2.0f * __builtin_amdgcn_rcpf(exp2_(2.0f * kLog2e * x) + 1.0f), y = x * x;
  const float near = x * (1.0f + y * (-1.0f / 3 + y * (2.0f / 15 + y * (-17.0f / 315 + y * (62.0f / 2835)))));
  return __builtin_fabsf(x) < 0.25f ? near : t;
}

// Bytes of w, as 0xFF, that are codes of NaN; of scale 2^120 also those beyond
// bf16: a block holds none, but for what an earlier use of its page left
// behind the last token.
__device__ inline uint32_t nan_bytes(uint32_t w, float scale) {
  const uint32_t m = (((w & 0x7F7F7F7Fu) + (scale < 0x1p120f ? 0x01010101u : 0x08080808u)) & 0x80808080u) >> 7;
  return m * 0xFFu;
}
__device__ inline float lse_of(float m, float sum) {
  return sum == 0 ? -__builtin_inff() : (m + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

constexpr int kGroup = 32;                // tokens of a wave's step
constexpr int kStep = kGroup * kWaves;    // of a workgroup's
constexpr int kStepLog = 7;
static_assert(kStep == 1 << kStepLog, "a step's tokens");
constexpr int kShares = 512;              // two workgroups a CU
constexpr int64_t kMostTokens = ((int64_t)1 << 31) - 256;

// A value that all lanes have, to scalar registers
__device__ inline int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline int64_t uni(int64_t x) {
  return (int64_t)(uint32_t)uni((int)x) | (int64_t)uni((int)(x >> 32)) << 32;
}
__device__ inline Seq uni(Seq s) { return {uni(s.row0), uni(s.n), uni(s.p0)}; }

// One tile of a sequence
struct Tile {
  int seq, h;
  Seq s;
  int r0;           // its first row of the sequence's n * group
  int first, last;  // positions of the first and the last row's token
};
template <int R>
__device__ inline bool tile_at(const CacheAttend& a, int seq, const Seq& s, int at, int h, Tile& t) {
  t.seq = seq;
  t.h = h;
  t.s = s;
  const int rows = s.n * a.group;
  if (at < 0 || at > (rows - 1) / R || rows == 0) return false;
  t.r0 = at * R;
  const int end = rows - t.r0 > R ? t.r0 + R : rows;
  t.first = uni((int)s.p0 + t.r0 / a.group);
  t.last = uni((int)s.p0 + (end - 1) / a.group);
  return true;
}
// The tokens that rows of positions first .. last see: from a multiple of 32
struct Span {
  int64_t from, to;
};
__device__ inline Span span_of(const CacheAttend& a, int64_t first, int64_t last) {
  int64_t have = a.b.table_pages << a.c.shift;
  if (have > kMostTokens) have = kMostTokens;
  Span s;
  s.to = last + 1 < have ? last + 1 : have;
  s.from = a.window > 0 && first - a.window + 1 > 0 ? (first - a.window + 1) / kGroup * kGroup : 0;
  if (s.to < s.from) s.to = s.from;
  return s;
}

template <int D, int MT>
struct State {
  float m[MT], l[MT];  // of this lane's row of each 16; l over this lane's tokens
  float e[MT];         // LSE: their sum before rounding
  bq_f32x4 o[MT][D / 16];
};
// 32 tokens' codes, of the keys or of the values
template <int D>
struct Codes {
  ca_u32x4 w[2][D / 64];
};

// The blocks of a wave's next 32 steps: lane 2 n + b has block b of step n
struct Blocks {
  uint32_t lo, hi;  // its number; hi < 0: it is not there
  uint32_t scales;  // bytes of K and V
};
__device__ inline Blocks blocks_of(const CacheAttend& a, const Tile& t, int64_t j, int64_t to, int step, int lane) {
  j += (lane >> 1) * step + 16 * (lane & 1);
  const int64_t blk = j < to ? block_at(a.c, a.b, t.seq, j, t.h) : -1;
  Blocks b = {(uint32_t)blk, (uint32_t)(blk >> 32), 127u | 127u << 8};
  if (blk >= 0) b.scales = *(const uint16_t*)(a.c.scales + 2 * blk);
  return b;
}
// Issues the loads of step n's codes. A block that is not there is read as
// zeros, and so is every block if there is no such step: loads that depend on
// no branch can be waited for singly.
template <int D, bool V>
__device__ inline void load_codes(const CacheAttend& a, const Blocks& bl, int n, bool real, int lane, Codes<D>& c) {
  const int off = 16 * lane;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint32_t lo = __builtin_amdgcn_readlane(bl.lo, 2 * n + b), hi = __builtin_amdgcn_readlane(bl.hi, 2 * n + b);
    const bool there = (int)hi >= 0 && real;
    const int64_t blk = there ? (int64_t)((uint64_t)hi << 32 | lo) : 0;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((V ? a.c.v : a.c.k) + blk * (kTok * D), (short)0,
                                                                       there ? kTok * D : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) c.w[b][i] = __builtin_amdgcn_raw_buffer_load_b128(r, off + 1024 * i, 0, 0);
  }
}
// How a product of a query and a key becomes a weight's exponent: times unit,
// after tanh with a cap. A negative scale's sign goes to the queries, and of a
// scale of 0 they are 0 (NaN where they are not finite, as 0 times them is), so
// that unit is above 0 and the largest score is the largest product's.
struct Scores {
  float unit, per_cap, cap_log2, twice;  // twice: 2 log2(e) per_cap, or 0 for a cap above kNearCap
  uint32_t flip;  // of the queries' bits
  bool none;      // scale 0
};
// Up to this cap 1 - 2 / (exp(2 x) + 1) is near enough for tanh near 0 too:
// 3 2^-24 off, of a score 2^-16, a weight's own rounding. It takes 3
// instructions for the 13 of tanh_ (drafted tokens under a window and a cap of
// 50: 29.5 us by that one, 27.2).
constexpr float kNearCap = 64.0f;
__device__ inline Scores scores_of(const CacheAttend& a, bool cap) {
  const float scale = a.scale == 0 ? 1.0f : __builtin_fabsf(a.scale);
  const float per_cap = cap ? __builtin_fminf(scale / a.cap, 0x1p120f) : 0.0f;
  return {cap ? 1.0f : scale * kLog2e, per_cap, cap ? a.cap * kLog2e : 0.0f, a.cap <= kNearCap ? 2.0f * kLog2e * per_cap : 0.0f,
          a.scale < 0 ? 0x80008000u : 0u, a.scale == 0};
}

// Step n's scales
struct Scales {
  float k[2], v[2];
  bool there[2];
};
__device__ inline Scales scales_of(const Blocks& bl, int n) {
  Scales s;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint32_t sc = __builtin_amdgcn_readlane(bl.scales, 2 * n + b);
    s.k[b] = scale_value(sc & 0xFFu);
    s.v[b] = scale_value(sc >> 8);
    s.there[b] = (int)__builtin_amdgcn_readlane(bl.hi, 2 * n + b) >= 0;
  }
  return s;
}

// Queries as the second operand: of few rows in registers, else in LDS
template <int D, int MT>
struct Queries {
  ca_bf16x8 f[D / 32];
  __device__ ca_bf16x8 get(int, int i) const { return f[i]; }
};

// 32 tokens from j0 into a wave's state. hard: some of them are hidden from
// some rows (pos: the positions of the lane's rows; -1: no row). next_k,
// next_v issue the next step's loads, as soon as this one's codes are used.
template <int D, int MT, bool CAP, bool FINE, bool LSE, typename Q, typename NextK, typename NextV>
__device__ inline void attend_group(const CacheAttend& a, const Scores& sc, int j0, bool hard, const int (&pos)[MT], const Q& query,
                                    int g, const Scales& s8, Codes<D>& k, Codes<D>& c, State<D, MT>& st, NextK next_k,
                                    NextV next_v) {
  constexpr int P = D / 64;
  // While two waves share a SIMD, the one at its products goes first and the
  // other's softmax fills the gaps (prompts of 1501 to 6007 tokens: 709 us
  // without, 695).
  if (MT > 1) __builtin_amdgcn_s_setprio(1);
  bq_f32x4 x[MT][2];
#pragma unroll
  for (int r = 0; r < MT; ++r) x[r][0] = x[r][1] = (bq_f32x4){0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 2 * P; ++i) {
    const ca_u32x4 w0 = k.w[0][i / 2], w1 = k.w[1][i / 2];
    const ca_bf16x8 k0 = i & 1 ? widen(w0.z, s8.k[0], w0.w, s8.k[0]) : widen(w0.x, s8.k[0], w0.y, s8.k[0]);
    const ca_bf16x8 k1 = i & 1 ? widen(w1.z, s8.k[1], w1.w, s8.k[1]) : widen(w1.x, s8.k[1], w1.y, s8.k[1]);
#pragma unroll
    for (int r = 0; r < MT; ++r) {
      const ca_bf16x8 q = query.get(r, i);
      x[r][0] = mma(k0, q, x[r][0]);
      x[r][1] = mma(k1, q, x[r][1]);
    }
  }
  if (MT > 1) __builtin_amdgcn_s_setprio(0);
  next_k();
  if constexpr (CAP) {
    if (sc.twice > 0) {
#pragma unroll
      for (int r = 0; r < MT; ++r)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[r][b][i] = __builtin_fmaf(-2.0f * sc.cap_log2, __builtin_amdgcn_rcpf(exp2_(x[r][b][i] * sc.twice) + 1.0f), sc.cap_log2);
    } else {
#pragma unroll
      for (int r = 0; r < MT; ++r)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[r][b][i] = sc.cap_log2 * tanh_(x[r][b][i] * sc.per_cap);
    }
  }
  uint32_t seen[MT];  // bit i: the row sees token i of the lane's 8
  if (hard) {
#pragma unroll
    for (int r = 0; r < MT; ++r) {
      seen[r] = 0;
      int at = pos[r];
      asm volatile("" : "+v"(at));  // computed here: every step would pay for the selects
      const int low = a.window > 0 && at >= a.window ? at - a.window : -1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = j0 + 16 * (i >> 2) + 4 * g + (i & 3);
        const bool is = s8.there[i >> 2] & (j <= at) & (j > low);
        seen[r] |= is ? 1u << i : 0u;
        if (!is) x[r][i >> 2][i & 3] = -__builtin_inff();
      }
    }
  }
  float top[MT];
  bool over = false;
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    // a NaN stays one: its row's sum will be, whatever the maximum
    top[r] = larger(larger(larger(x[r][0][0], x[r][0][1]), larger(x[r][0][2], x[r][0][3])),
                    larger(larger(x[r][1][0], x[r][1][1]), larger(x[r][1][2], x[r][1][3]))) * sc.unit;
    over |= top[r] > st.m[r] + kSlack;
  }
  if (__any(over)) {
#pragma unroll
    for (int r = 0; r < MT; ++r) {
      const float m = fmaxf(quad_max(top[r]), st.m[r]);
      const float f = m == st.m[r] ? 1.0f : exp2_(st.m[r] - m);
      st.m[r] = m;
      st.l[r] *= f;
      if constexpr (LSE) st.e[r] *= f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) st.o[r][i] *= f;
    }
  }
  ca_bf16x8 pf[MT], pl[FINE ? MT : 1];
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    const float base = st.m[r] == -__builtin_inff() ? 0.0f : st.m[r];
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = exp2_(__builtin_fmaf(x[r][i >> 2][i & 3], sc.unit, -base));
    ca_u32x4 w, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
      if constexpr (FINE)
        y[i] = pack_bf16(p[2 * i] - __uint_as_float(w[i] << 16), p[2 * i + 1] - __uint_as_float(high_half(w[i])));
    }
    pf[r] = __builtin_bit_cast(ca_bf16x8, w);
    const auto sum = [&] { return ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7])); };
    if constexpr (FINE) {
      pl[r] = __builtin_bit_cast(ca_bf16x8, y);
      st.l[r] += sum();
    } else {
      if constexpr (LSE) st.e[r] += sum();
      // of the rounded weights, two an instruction
#pragma unroll
      for (int i = 0; i < 4; ++i) st.l[r] = add2(w[i], st.l[r]);
    }
  }
  if (hard) {
    // a hidden token's weight is 0, but a NaN times 0 is one: the NaNs are
    // taken out of the product, and given to the rows that see them
    uint32_t any = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) any |= nan_bytes(c.w[b][i][n], s8.v[b]);
    if (__any(any != 0)) {
      // found anew: 32 registers less than held from the search
#pragma unroll
      for (int i = 0; i < P; ++i) asm volatile("" : "+v"(c.w[0][i]), "+v"(c.w[1][i]));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t n[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          n[b] = nan_bytes(c.w[b][i / 4][i % 4], s8.v[b]);
          c.w[b][i / 4][i % 4] &= ~n[b];
          n[b] &= 0x38383838u;  // 1
        }
        const ca_bf16x8 nf = widen(n[0], 1.0f, n[1], 1.0f);
#pragma unroll
        for (int r = 0; r < MT; ++r) {
          ca_u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = (seen[r] >> (2 * e) & 1u) * 0x3F80u | (seen[r] >> (2 * e + 1) & 1u) * 0x3F800000u;
          const bq_f32x4 y = mma(nf, __builtin_bit_cast(ca_bf16x8, w), (bq_f32x4){0, 0, 0, 0});
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (y[e] > 0) st.o[r][i][e] = nan();
        }
      }
    }
  }
  if (MT > 1) __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const ca_bf16x8 vf = widen(c.w[0][i / 4][i % 4], s8.v[0], c.w[1][i / 4][i % 4], s8.v[1]);
#pragma unroll
    for (int r = 0; r < MT; ++r) {
      st.o[r][i] = mma(vf, pf[r], st.o[r][i]);
      if constexpr (FINE) st.o[r][i] = mma(vf, pl[r], st.o[r][i]);
    }
  }
  next_v();
}

// `steps` times 32 tokens, from j on every `step`, into a wave's state
template <int D, int MT, bool CAP, bool FINE, bool LSE, typename Q>
__device__ inline void walk(const CacheAttend& a, const Scores& sc, const Tile& t, int64_t j, int64_t to, int step, int steps,
                            const int (&pos)[MT], const Q& query, int lane, State<D, MT>& st) {
  Blocks bl = blocks_of(a, t, j, to, step, lane);
  Codes<D> k, v;
  load_codes<D, false>(a, bl, 0, steps > 0, lane, k);
  load_codes<D, true>(a, bl, 0, steps > 0, lane, v);
  for (int n = 0; n < steps; ++n) {
    const int j0 = (int)(j + (int64_t)n * step), next = (n + 1) & 31;
    const bool more = n + 1 < steps;
    const auto next_k = [&] { load_codes<D, false>(a, bl, next, more, lane, k); };
    const auto next_v = [&] { load_codes<D, true>(a, bl, next, more, lane, v); };
    const Scales s8 = scales_of(bl, n & 31);
    if (next == 0 && more) bl = blocks_of(a, t, j + (int64_t)(n + 1) * step, to, step, lane);
    // hidden from somebody: the rows' positions are first .. last
    const bool hard = uni((int)(!s8.there[0] || !s8.there[1] || j0 + 31 > t.first || (a.window > 0 && t.last >= a.window && j0 <= t.last - a.window)));
    attend_group<D, MT, CAP, FINE, LSE>(a, sc, j0, hard, pos, query, lane >> 4, s8, k, v, st, next_k, next_v);
  }
}

// Where a tile's part goes: parts[slot][row][D] and the row's maximum and sum
struct Space {
  float* parts;
  float* sums;  // [slot][row][2]
  int4* heads;  // [share]: parts of the tile that starts in it and ends in a later one, sequence, head, first row
};

template <int D, int MT, bool LSE = false>
struct Shared {
  float acc[kWaves][4][D / 16 < 8 ? D / 16 : 8][64];
  float ml[kWaves][LSE ? 3 : 2][16 * MT];
  ca_u32x4 q[MT > 1 ? MT : 1][MT > 1 ? D / 32 : 1][MT > 1 ? 64 : 1];
};
template <int D>
struct LdsQueries {
  const ca_u32x4* q;  // [16 rows][D / 32][lane]
  int lane;
  __device__ ca_bf16x8 get(int r, int i) const { return __builtin_bit_cast(ca_bf16x8, q[(r * (D / 32) + i) * 64 + lane]); }
};

// 0 times two bf16
__device__ inline uint32_t times_zero(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0x7FC0u : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0x7FC00000u : 0u);
}
template <int D>
__device__ inline ca_u32x4 query_at(const CacheAttend& a, const Scores& sc, const Tile& t, int row, int i, int g) {
  if (row >= t.s.n * a.group) return (ca_u32x4){0, 0, 0, 0};
  const int tok = row / a.group, head = t.h * a.group + row % a.group;
  const ca_u32x4 w = *(const bq_u32x4_a2*)(a.q.p + (int64_t)(t.s.row0 + tok) * a.q.tok + head * a.q.head + 64 * (i / 2) +
                                           16 * g + 8 * (i % 2));
  if (sc.none) return (ca_u32x4){times_zero(w.x), times_zero(w.y), times_zero(w.z), times_zero(w.w)};
  return w ^ sc.flip;
}

// The waves' sums (their maxima and sums are in sh.ml already) joined and written
template <int D, int MT, bool LSE>
__device__ inline void finish(const CacheAttend& a, const Tile& t, const Space& ws, int slot, Shared<D, MT, LSE>& sh,
                              const State<D, MT>& st, int lane, int wave) {
  constexpr int R = 16 * MT, W = D / 16, C = W < 8 ? W : 8;
  const int lo16 = lane & 15, g = lane >> 4, rows = t.s.n * a.group;
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    const int row = 16 * r + lo16;
    float m = sh.ml[0][0][row], sum = 0, before = 0, f[kWaves];  // before rounding
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sh.ml[w][0][row]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = sh.ml[w][0][row];
      f[w] = mw == m ? 1.0f : exp2_(mw - m);
      sum += sh.ml[w][1][row] * f[w];
      if constexpr (LSE) before += sh.ml[w][2][row] * f[w];
    }
    const bool have = t.r0 + row < rows;
    const int tok = (t.r0 + row) / a.group, head = t.h * a.group + (t.r0 + row) % a.group;
    const int64_t tr = t.s.row0 + tok;
    const float inv = sum == 0 ? 0.0f : 1.0f / sum;
    const int d = W * (4 * g + wave);  // this lane's D / 16 elements
    uint16_t* out = a.out.p + tr * a.out.tok + head * a.out.head + d;
    float* part = ws.parts + ((int64_t)slot * R + row) * D + d;
#pragma unroll
    for (int c = 0; c < W; c += C) {
      if (r || c) __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < C; ++i) sh.acc[wave][k][i][lane] = st.o[r][c + i][k];
      __syncthreads();
      float o[C];
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] += sh.acc[w][wave][i][lane] * f[w];
      if (!have) continue;
      if (slot >= 0) {
#pragma unroll
        for (int i = 0; i < C; i += 4) *(bq_f32x4*)(part + c + i) = (bq_f32x4){o[i], o[i + 1], o[i + 2], o[i + 3]};
      } else {
#pragma unroll
        for (int i = 0; i < C; i += 4)
          *(bq_u32x2_a2*)(out + c + i) =
              (bq_u32x2){pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv)};
      }
    }
    if (have && wave == 0 && g == 0) {
      if (slot >= 0) {
        ws.sums[((int64_t)slot * R + row) * 2] = m;
        ws.sums[((int64_t)slot * R + row) * 2 + 1] = sum;
      } else if (a.lse) {
        a.lse[tr * a.q_heads + head] = lse_of(m, LSE ? before : sum);
      }
    }
  }
  __syncthreads();
}

// The tile's tokens from .. to (from a multiple of 32): its output, or with
// slot >= 0 a part of it.
template <int D, int MT, bool CAP, bool FINE, bool LSE>
__device__ inline void run_tile(const CacheAttend& a, const Tile& t, int64_t from, int64_t to, const Space& ws, int slot,
                                Shared<D, MT, LSE>& sh) {
  constexpr int W = D / 16;
  const Scores sc = scores_of(a, CAP);
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // nothing is held from tile to tile
  const int wave = uni((int)(threadIdx.x >> 6));
  const int lo16 = lane & 15, g = lane >> 4;
  const int rows = t.s.n * a.group;
  from = uni(from);
  to = uni(to);
  const int64_t j = from + wave * kGroup;
  const int steps = j < to ? (int)((to - j + kStep - 1) / kStep) : 0;
  int pos[MT];
  State<D, MT> st;
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    const int row = t.r0 + 16 * r + lo16;
    pos[r] = row < rows ? (int)t.s.p0 + row / a.group : -1;
    st.m[r] = -__builtin_inff();
    st.l[r] = st.e[r] = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) st.o[r][i] = (bq_f32x4){0, 0, 0, 0};
  }
  Queries<D, MT> mine;
  if constexpr (MT == 1) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) mine.f[i] = __builtin_bit_cast(ca_bf16x8, query_at<D>(a, sc, t, t.r0 + lo16, i, g));
  } else {
    for (int n = wave; n < MT * (D / 32); n += kWaves)
      sh.q[n / (D / 32)][n % (D / 32)][lane] = query_at<D>(a, sc, t, t.r0 + 16 * (n / (D / 32)) + lo16, n % (D / 32), g);
    __syncthreads();
  }
  if constexpr (MT == 1) walk<D, MT, CAP, FINE, LSE>(a, sc, t, j, to, kStep, steps, pos, mine, lane, st);
  else walk<D, MT, CAP, FINE, LSE>(a, sc, t, j, to, kStep, steps, pos, LdsQueries<D>{&sh.q[0][0][0], lane}, lane, st);
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    const float l = quad_sum(st.l[r]);
    if (lane < 16) {
      sh.ml[wave][0][16 * r + lane] = st.m[r];
      sh.ml[wave][1][16 * r + lane] = l;
    }
    if constexpr (LSE) {
      const float e = quad_sum(st.e[r]);
      if (lane < 16) sh.ml[wave][2][16 * r + lane] = e;
    }
  }
  __syncthreads();
  // what follows is computed here, and not held in registers through the loop
  int lane_ = lane;
  asm volatile("" : "+v"(lane_));
  finish(a, t, ws, slot, sh, st, lane_, wave);
}

// A share is counted in units of 128 2^shift tokens (so that all of a call's
// are fewer than 2^31). A tile costs those that its sequence's rows see, and
// kBegin more: its lookups and first loads, which nothing overlaps, and its
// join over LDS take as long as two units (a layer's decode step of 32
// sequences of 50 to 8192 tokens, 32 heads: 203 us counted as 0, 149 as 1, 141
// as 2, 144 as 4).
constexpr int kBegin = 2;
struct Units {
  int tiles, units;
  int64_t from;  // the first one's first token
};
template <int R>
__device__ inline Units units_of(const CacheAttend& a, const Seq& s, int shift) {
  const Span p = span_of(a, s.p0, s.p0 + s.n - 1);
  return {(s.n * a.group + R - 1) / R, (int)((p.to - p.from + (kStep << shift) - 1) >> (kStepLog + shift)) + kBegin, p.from};
}

// Sum over the lanes up to this one, of values up to kMostUnits and no more
// than that: all that a batch can have, so that whatever starts holds
// (decreasing ones count rows twice) no place is outside of it.
constexpr int kMostUnits = 1 << 30;
__device__ inline int least(int a, int b) { return a < b ? a : b; }
__device__ inline int scan(int x) {
  const auto add = [](int a, int b) {
    const uint32_t s = (uint32_t)a + (uint32_t)b;
    return (int)(s < (uint32_t)kMostUnits ? s : (uint32_t)kMostUnits);
  };
  x = add(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true));   // row_shr:1
  x = add(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true));
  x = add(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true));
  x = add(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true));
  x = add(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));  // row_bcast:15 into rows 1 and 3
  x = add(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));  // row_bcast:31 into rows 2 and 3
  return x;
}

template <int D, int MT, bool CAP>
__global__ __launch_bounds__(64 * kWaves, 2) void cache_attention_shares_kernel(CacheAttend a, Space ws, int shift) {
  constexpr int R = 16 * MT;
  __shared__ Shared<D, MT> sh;
  const int lane = threadIdx.x & 63;
  // units before each lane's sequences; every wave finds its workgroup's place by itself
  const int per = (a.b.sequences + 63) / 64;
  int mine = 0;
  Seq s = {0, 0, 0};
  for (int i = lane * per; i < (lane + 1) * per && i < a.b.sequences; ++i) {
    s = seq_of(a.b, i);
    const Units n = units_of<R>(a, s, shift);
    mine = least(mine + n.tiles * a.c.heads * n.units, kMostUnits);
  }
  const int upto = scan(mine), total = __builtin_amdgcn_readlane(upto, 63);
  const int share = (total + (int)gridDim.x - 1) / (int)gridDim.x;
  int u = blockIdx.x * share;
  const int end = total - u < share ? total : u + share;
  int4 open = {0, 0, 0, 0};
  if (share > 0 && u < end) {
    const int at_lane = 63 - __builtin_clzll(__ballot(upto - mine <= u));
    int rem = u - __builtin_amdgcn_readlane(upto - mine, at_lane), seq = at_lane * per;
    s = {__builtin_amdgcn_readlane(s.row0, at_lane), __builtin_amdgcn_readlane(s.n, at_lane),
         (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)s.p0, at_lane) |
             (int64_t)__builtin_amdgcn_readlane((int)(s.p0 >> 32), at_lane) << 32};
    bool known = per == 1, found = false;  // s is seq's; and the place in its tiles
    Units n = {0, 0, 0};
    int k0 = 0, at = 0, h = 0;
    while (u < end && seq < a.b.sequences) {
      if (!found) {
        if (!known) s = uni(seq_of(a.b, seq));
        known = false;
        n = units_of<R>(a, s, shift);
        n = {uni(n.tiles), uni(n.units), uni(n.from)};
        if (rem >= n.tiles * a.c.heads * n.units) {
          rem -= n.tiles * a.c.heads * n.units;
          ++seq;
          continue;
        }
        const int item = uni((int)((uint32_t)rem / (uint32_t)n.units));
        k0 = rem - item * n.units;
        h = uni((int)((uint32_t)item / (uint32_t)n.tiles));
        at = item - h * n.tiles;
        found = true;
      }
      const int k1 = end - u < n.units - k0 ? k0 + (end - u) : n.units;
      if (k1 > kBegin) {
        Tile t;
        tile_at<R>(a, seq, s, at, h, t);
        const Span own = span_of(a, t.first, t.last);
        const bool first = k0 <= kBegin, whole = first && k1 == n.units;
        const int64_t lo = n.from + ((int64_t)(first ? 0 : k0 - kBegin) * kStep << shift);
        const int64_t hi = n.from + ((int64_t)(k1 - kBegin) * kStep << shift);
        const int64_t from = lo > own.from ? lo : own.from, to = hi < own.to ? hi : own.to;
        run_tile<D, MT, CAP, true, false>(a, t, from, to, ws, whole ? -1 : 2 * (int)blockIdx.x + first, sh);
        if (first && !whole)
          open = make_int4(1 + (u + (n.units - k0) - 1) / share - (int)blockIdx.x, seq, t.h, t.r0);
      } else if (n.units == kBegin) {
        // it sees nothing
        Tile t;
        tile_at<R>(a, seq, s, at, h, t);
        if (k1 == n.units) run_tile<D, MT, CAP, true, false>(a, t, 0, 0, ws, -1, sh);
      }
      u += k1 - k0;
      k0 = 0;
      if (u < end && ++at == n.tiles) {
        at = 0;
        if (++h == a.c.heads) {
          h = 0;
          rem = 0;
          ++seq;
          found = false;
        }
      }
    }
  }
  if (threadIdx.x == 0) ws.heads[blockIdx.x] = open;
}

// Joins the parts of the tile that starts in share blockIdx.x: 256 elements
// of its rows by 64 lanes, the parts over the waves.
template <int D, int MT>
__global__ __launch_bounds__(64 * kWaves) void cache_attention_join_kernel(CacheAttend a, Space ws) {
  constexpr int R = 16 * MT;
  __shared__ bq_f32x4 acc[kWaves][64];
  __shared__ float ml[kWaves][2][64];
  const int4 open = ws.heads[blockIdx.x];
  if (open.x == 0) return;
  const int parts = open.x < (int)(gridDim.x - blockIdx.x) ? open.x : (int)(gridDim.x - blockIdx.x);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Seq s = seq_of(a.b, open.y);
  const int row = (blockIdx.y * 256 + 4 * lane) / D, d = (blockIdx.y * 256 + 4 * lane) % D;
  const int at = open.w + row;
  const bool have = at < s.n * a.group;
  if (open.w + (int)(blockIdx.y * 256) / D >= s.n * a.group) return;
  float m = -__builtin_inff(), l = 0;
  bq_f32x4 o = {0, 0, 0, 0};
  // wave w: parts w, w + 4, ..; each part's sum, scaled to the running maximum
  if (have)
    for (int p = wave; p < parts; p += kWaves) {
      const int64_t slot = p == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + p);
      const float mp = ws.sums[(slot * R + row) * 2], lp = ws.sums[(slot * R + row) * 2 + 1];
      const bq_f32x4 x = *(const bq_f32x4*)(ws.parts + (slot * R + row) * D + d);
      const float top = fmaxf(m, mp), f = m == top ? 1.0f : exp2_(m - top), fp = mp == top ? 1.0f : exp2_(mp - top);
      m = top;
      l = l * f + lp * fp;
      o = o * f + x * fp;
    }
  acc[wave][lane] = o;
  ml[wave][0][lane] = m;
  ml[wave][1][lane] = l;
  __syncthreads();
  if (wave || !have) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, ml[w][0][lane]);
  l = 0;
  o = (bq_f32x4){0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float mw = ml[w][0][lane], f = mw == m ? 1.0f : exp2_(mw - m);
    l += ml[w][1][lane] * f;
    o += acc[w][lane] * f;
  }
  const float inv = l == 0 ? 0.0f : 1.0f / l;
  const int64_t tr = s.row0 + at / a.group;
  const int head = open.z * a.group + at % a.group;
  *(bq_u32x2_a2*)(a.out.p + tr * a.out.tok + head * a.out.head + d) =
      (bq_u32x2){pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv)};
  if (a.lse && d == 0) a.lse[tr * a.q_heads + head] = lse_of(m, l);
}

// The tile that virtual tile v is, of key head h: sequence i's are numbered
// from starts[i] group / R + i on
template <int R>
__device__ inline bool tile_of(const CacheAttend& a, int64_t v, int h, Tile& t) {
  const auto first = [&](int j) { return (int64_t)start_of(a.b, j) * a.group / R + j; };
  const int seq = uni(last_upto(a.b.sequences, v, first));
  return tile_at<R>(a, seq, uni(seq_of(a.b, seq)), uni((int)(v - first(seq))), h, t);
}

// More rows: a workgroup takes a tile, its waves sharing out the tokens; a
// sequence's last tiles, which see most of it, go first.
template <int D, int MT, bool CAP, bool LSE>
__global__ __launch_bounds__(64 * kWaves, 2) void cache_attention_tiles_kernel(CacheAttend a) {
  __shared__ Shared<D, MT, LSE> sh;
  const int64_t v = (gridDim.x - 1 - blockIdx.x) / a.c.heads;
  Tile t;
  if (!tile_of<16 * MT>(a, v, (int)((gridDim.x - 1 - blockIdx.x) % a.c.heads), t)) return;
  const Span s = span_of(a, t.first, t.last);
  run_tile<D, MT, CAP, false, LSE>(a, t, s.from, s.to, Space{}, -1, sh);
}

// Many rows: a wave takes a tile with all its tokens, without a word to the
// others, which have the rows beside its own, so that what one loads the
// others find in the CU's cache. Prompts of 1501 to 6007 tokens, 64 query and
// 8 key heads (8600 tiles): 708 us, by the kernel above 811; one of 4096, 32
// heads each with its own keys (2080 tiles, a single round here): 190 and 175.
// Its state does not quite fit 256 registers: the compiler spills 23 of heads
// of 128 elements (29 with a cap), 38 to 41 of heads of 256, none of 64.
template <int D, int MT, bool CAP, bool LSE>
__global__ __launch_bounds__(64 * kWaves, 2) void cache_attention_rows_kernel(CacheAttend a) {
  constexpr int R = 16 * MT, W = D / 16;
  __shared__ ca_u32x4 queries[kWaves][MT * (D / 32) * 64];
  const int lane = threadIdx.x & 63, wave = uni((int)(threadIdx.x >> 6));
  const int lo16 = lane & 15, g = lane >> 4;
  const int64_t v = (int64_t)((gridDim.x - 1 - blockIdx.x) / a.c.heads) * kWaves + wave;
  const int h = (int)((gridDim.x - 1 - blockIdx.x) % a.c.heads);
  Tile t;
  if (!tile_of<R>(a, v, h, t)) return;
  const Scores sc = scores_of(a, CAP);
  const Span s = span_of(a, t.first, t.last);
  const int64_t from = uni(s.from), to = uni(s.to);
  const int rows = t.s.n * a.group;
#pragma unroll
  for (int n = 0; n < MT * (D / 32); ++n)
    queries[wave][n * 64 + lane] = query_at<D>(a, sc, t, t.r0 + 16 * (n / (D / 32)) + lo16, n % (D / 32), g);
  int pos[MT];
  State<D, MT> st;
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    const int row = t.r0 + 16 * r + lo16;
    pos[r] = row < rows ? (int)t.s.p0 + row / a.group : -1;
    st.m[r] = -__builtin_inff();
    st.l[r] = st.e[r] = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) st.o[r][i] = (bq_f32x4){0, 0, 0, 0};
  }
  // the wave's own lanes read them: LDS serves a wave in order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  walk<D, MT, CAP, false, LSE>(a, sc, t, from, to, kGroup, (int)((to - from + kGroup - 1) / kGroup), pos,
                          LdsQueries<D>{queries[wave], lane}, lane, st);
  int lane_ = lane;
  asm volatile("" : "+v"(lane_));  // computed here, and not held in registers through the loop
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    const float sum = quad_sum(st.l[r]), inv = sum == 0 ? 0.0f : 1.0f / sum;
    float before = 0;
    if constexpr (LSE) before = quad_sum(st.e[r]);
    const int row = t.r0 + 16 * r + (lane_ & 15);
    if (row >= rows) continue;
    const int head = t.h * a.group + row % a.group;
    const int64_t tr = t.s.row0 + row / a.group;
    uint16_t* out = a.out.p + tr * a.out.tok + head * a.out.head + 4 * W * (lane_ >> 4);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < W; i += 4)
        *(bq_u32x2_a2*)(out + W * k + i) = (bq_u32x2){pack_bf16(st.o[r][i][k] * inv, st.o[r][i + 1][k] * inv),
                                                      pack_bf16(st.o[r][i + 2][k] * inv, st.o[r][i + 3][k] * inv)};
    if constexpr (LSE)
      if (lane_ < 16) a.lse[tr * a.q_heads + head] = lse_of(st.m[r], before);
  }
}

// Rows of a tile and whether a workgroup takes whole tiles: by the mean rows
// of a sequence and key head, all that the host knows of the lengths.
struct Form {
  int mt;
  bool tiles;
  int64_t count;  // of tiles, at most
  int shift;      // of a unit
  int most;       // workgroups that share the work
  int shares;     // no more of them than there can be units
};
// Workgroups that share the work: two a CU, by their registers, and three of
// tiles of 16 rows of up to 128 elements if every CU has a tile. With fewer, of
// long sequences, the third only cuts them up further (us of one decoded token
// with two and three a CU, by sequences, lengths, query and key heads: 100 of
// 10 to 3000, 10 and 10 of 128 elements 38.8 and 35.7, of 64 30.9 and 26.2; 64
// of 100 to 16000, 32 and 4 of 128 47.1 and 44.6, of 64 31.2 and 30.0; 8 of
// 100 to 3000, 64 and 8 of 128 13.9 and 15.2).
int most_shares(int head_dim, int mt, int64_t tiles) { return mt == 1 && head_dim <= 128 && tiles >= 256 ? kShares * 3 / 2 : kShares; }
constexpr int most_rows(int head_dim) { return head_dim == 256 ? 2 : 4; }  // 16-row tiles, by a wave's registers
Form form_of(const CacheAttend& a, int head_dim) {
  const int64_t rows = a.b.starts ? ((int64_t)a.b.tokens * a.group + a.b.sequences - 1) / a.b.sequences : a.group;
  Form f;
  f.mt = rows <= 16 ? 1 : rows <= 32 ? 2 : most_rows(head_dim);
  f.count = ((int64_t)a.b.tokens * a.group / (16 * f.mt) + a.b.sequences) * a.c.heads;
  int64_t most = a.b.table_pages << a.c.shift;
  most = most < kMostTokens ? most : kMostTokens;
  f.shift = 0;
  const auto units = [&] { return f.count * ((most + kStep) / ((int64_t)kStep << f.shift) + 1 + kBegin); };
  while (units() >= kMostUnits && f.shift < 23) ++f.shift;
  f.most = most_shares(head_dim, f.mt, f.count);
  f.shares = units() < f.most ? (int)units() : f.most;
  f.tiles = a.b.starts && rows > 32 && f.count >= 2 * kShares;
  return f;
}
constexpr int64_t kRowsTiles = 5 * kShares;  // of waves that take whole tiles: more than a round of them

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
Space space_of(void* ws, const Form& f, int head_dim, size_t* bytes) {
  const size_t rows = (size_t)2 * f.most * 16 * f.mt;
  uint8_t* p = (uint8_t*)ws;
  const size_t parts = round256(rows * head_dim * 4), sums = round256(rows * 8);
  *bytes = parts + sums + f.most * sizeof(int4);
  return {(float*)p, (float*)(p + parts), (int4*)(p + parts + sums)};
}

template <int D, int MT, bool CAP, bool LSE>
hipError_t run_tiles(const CacheAttend& a, const Form& f, hipStream_t st) {
  const dim3 block(64 * kWaves);
  if (f.count >= kRowsTiles) {
    const unsigned grid = (unsigned)((f.count / a.c.heads + kWaves - 1) / kWaves * a.c.heads);
    cache_attention_rows_kernel<D, MT, CAP, LSE><<<grid, block, 0, st>>>(a);
  } else {
    cache_attention_tiles_kernel<D, MT, CAP, LSE><<<(unsigned)f.count, block, 0, st>>>(a);
  }
  return hipGetLastError();
}

template <int D, int MT>
hipError_t run(const CacheAttend& a, const Form& f, const Space& ws, hipStream_t st) {
  const dim3 block(64 * kWaves);
  if constexpr (MT == most_rows(D)) {
    if (f.tiles && a.cap > 0) return a.lse ? run_tiles<D, MT, true, true>(a, f, st) : run_tiles<D, MT, true, false>(a, f, st);
    if (f.tiles) return a.lse ? run_tiles<D, MT, false, true>(a, f, st) : run_tiles<D, MT, false, false>(a, f, st);
  }
  if (a.cap > 0) cache_attention_shares_kernel<D, MT, true><<<f.shares, block, 0, st>>>(a, ws, f.shift);
  else cache_attention_shares_kernel<D, MT, false><<<f.shares, block, 0, st>>>(a, ws, f.shift);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int rows = !a.b.starts && a.group < 16 * MT ? a.group : 16 * MT;
  cache_attention_join_kernel<D, MT><<<dim3(f.shares, (rows * D + 255) / 256), block, 0, st>>>(a, ws);
  return hipGetLastError();
}

}  // namespace

size_t cache_attention_ws_bytes(const CacheAttend& a, int head_dim) {
  if (!a.b.tokens || !a.b.sequences) return 0;
  const Form f = form_of(a, head_dim);
  size_t n = 0;
  if (!f.tiles) space_of(nullptr, f, head_dim, &n);
  return n;
}

void cache_attention_plan(const CacheAttend& a, int head_dim, int* rows, int* form) {
  if (!a.b.tokens || !a.b.sequences) {
    *rows = *form = 0;
    return;
  }
  const Form f = form_of(a, head_dim);
  *rows = 16 * f.mt;
  *form = !f.tiles ? FP8_CACHE_SHARES : f.count < kRowsTiles ? FP8_CACHE_TILES : FP8_CACHE_ROWS;
}

hipError_t launch_cache_attention(const CacheAttend& a, int head_dim, void* ws, hipStream_t st) {
  if (!a.b.tokens || !a.b.sequences) return hipSuccess;
  const Form f = form_of(a, head_dim);
  size_t n;
  const Space s = space_of(ws, f, head_dim, &n);
  if (f.mt == 1)
    return head_dim == 64 ? run<64, 1>(a, f, s, st) : head_dim == 128 ? run<128, 1>(a, f, s, st) : run<256, 1>(a, f, s, st);
  if (f.mt == 2)
    return head_dim == 64 ? run<64, 2>(a, f, s, st) : head_dim == 128 ? run<128, 2>(a, f, s, st) : run<256, 2>(a, f, s, st);
  return head_dim == 64 ? run<64, 4>(a, f, s, st) : run<128, 4>(a, f, s, st);
}

}  // namespace fp8lin
