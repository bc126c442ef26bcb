// Appending to the paged cache, with the rotation on the way, and reading
// back. One workgroup takes the rows of a batch that lie in one block of 16
// positions; its waves share out the heads: an item is the keys or the
// values of a head, or a query head, and a wave owns an item's block alone,
// so the scale that its tokens share needs no atomics.
//
// Blocks are numbered without reading the batch on the host: sequence i's
// start at starts[i] / 16 + 2 i, since n rows touch at most n / 16 + 2 blocks
// wherever they begin.
//
// Angles are position * freq in 64 bits, their sines and cosines are computed
// once a workgroup, and keys are rotated and rounded to 8 bits from 64-bit
// values: a 32-bit rotation would put one in a million keys on the wrong side
// of a rounding border. The step between goes by 32 bits rounded to odd,
// which keeps a value on its side of any border of the 8-bit format.
#include "cache.h"

namespace fp8lin {
namespace {

constexpr int kWaves = 4;

// v to 32 bits, to odd: cut, with the last bit set if anything was cut off
__device__ inline float to_odd(double v) {
  const float f = (float)v;
  const double d = (double)f;
  uint32_t u = __float_as_uint(f);
  if (d == v || v != v || __builtin_isinf(v)) return f;
  if (__builtin_fabs(d) > __builtin_fabs(v)) --u;
  return __uint_as_float(u | 1u);
}

__device__ inline uint32_t wave_max(uint32_t m) {
  m = row16_max(m);
  const auto mx = [](uint32_t a, uint32_t b) { return umax(a, b); };
  m = swap16_max(m, m, mx);
  return swap32_max(m, m, mx);
}

// What a block's new values ask of its scale: the scale byte by their finite
// magnitudes (bits; 0: none), 1 for none; at least 127 with an infinity.
__device__ inline uint32_t need_byte(uint32_t mag, bool inf) {
  uint32_t s = mag ? scale_byte<FP8_E4M3>(mag) : 1u;
  return inf ? umax(s, 127u) : s;
}
// Clamped to the format's largest value; of scale 2^120, the largest there is,
// to 240: what is held is finite in bf16, so that a hidden token's weight of 0
// leaves 0 of it.
constexpr float kTopScale = 0x1p120f;
__device__ inline float clamped(float f, float scale) {
  const float m = scale < kTopScale ? 448.0f * scale : 240.0f * kTopScale;
  return f != f ? f : fminf(fmaxf(f, -m), m);
}
// codes of four values; beyond the largest only if an infinity is among them or of the largest scale
__device__ inline uint32_t codes_of(float a, float b, float c, float d, float s, bool inf) {
  if (inf || s >= kTopScale) return code4<FP8_E4M3>(clamped(a, s), clamped(b, s), clamped(c, s), clamped(d, s), s);
  return code4<FP8_E4M3>(a, b, c, d, s);
}
// codes of scale s0 rounded anew to scale s1
__device__ inline uint32_t recode(uint32_t w, float s0, float s1) {
  const bq_f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s0, false);
  const bq_f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s0, true);
  return code4<FP8_E4M3>(lo.x, lo.y, hi.x, hi.y, s1);
}

// The rows of one block of positions
struct Part {
  int seq, row0;    // packed row of slot 0 (of those in [from, to))
  int from, to;     // slots of the batch's rows
  int64_t pos;      // position of slot 0
};
__device__ inline bool part_of(const CacheBatch& b, int v, Part& p) {
  int i, at;
  if (b.starts) {
    const auto first = [&](int j) { return (int64_t)(start_of(b, j) / kTok) + 2 * j; };
    i = last_upto(b.sequences, v, first);
    at = v - (int)first(i);
  } else {
    i = v;
    at = 0;
  }
  const Seq s = seq_of(b, i);
  p.seq = i;
  p.pos = ((s.p0 >> 4) + at) * kTok;  // the shift rounds down, below 0 too
  const int64_t from = s.p0 - p.pos, to = s.p0 + s.n - p.pos;
  p.from = from > 0 ? (int)from : 0;
  p.to = to < kTok ? (int)to : kTok;
  p.row0 = s.row0 - (int)from;
  return p.from < p.to;
}
inline unsigned parts_of(const CacheBatch& b) {
  return b.starts ? (unsigned)(b.tokens / kTok + 2 * (int64_t)b.sequences) : (unsigned)b.sequences;
}

// Angles of a slot, one more than there are: lanes of 16 slots read the same
// angle at a time, which 64 apart lay in one bank (of an append of 8200 tokens
// and 40 heads two thirds of all cycles: 150 us, 134 without)
__host__ __device__ inline int angles_pitch(int rot) { return rot / 2 + 1; }

// How 8 elements from d (a multiple of 8) of a row turn: with those from
// `other`, by the angles from `angle` on
struct Turn {
  int other, angle;
  bool turns, low;
};
__device__ inline Turn turn_of(int d, int rot, int inter) {
  const int half = rot / 2;
  Turn t;
  t.turns = d < rot;
  t.low = d < half;
  t.other = !t.turns || inter ? d : t.low ? d + half : d - half;
  t.angle = !t.turns ? 0 : inter ? d / 2 : t.low ? d : d - half;
  return t;
}
// T: the precision; cs: the angles' cos and sin in it
template <typename T, typename T2>
__device__ inline void rotate8(bq_u32x4 own, bq_u32x4 other, const Turn& t, int inter, const T2* cs, T y[8]) {
  float x[8];
  widen8(own, x);
  if (inter) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const T2 v = cs[t.angle + j];
      const T p = x[2 * j], q = x[2 * j + 1];
      y[2 * j] = t.turns ? p * v.x - q * v.y : p;
      y[2 * j + 1] = t.turns ? q * v.x + p * v.y : q;
    }
  } else {
    float o[8];
    widen8(other, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const T2 v = cs[t.angle + j];
      const T p = x[j], q = t.low ? -o[j] : o[j];
      y[j] = t.turns ? p * v.x + q * v.y : p;
    }
  }
}
__device__ inline bq_u32x4 row8(const uint16_t* p) { return *(const bq_u32x4_a2*)p; }

__device__ inline void add_mag(float f, uint32_t& mag, bool& inf) {
  const uint32_t m = __float_as_uint(f) & 0x7FFFFFFFu;
  if (m < 0x7F800000u) mag = umax(mag, m);
  inf |= m == 0x7F800000u;
}

// Scale of the block's new values against the one held: the byte, and whether
// the codes before slot `from` have to be rounded anew.
struct Scales {
  float now, held;
  bool again;
};
__device__ inline Scales settle(uint8_t* at, uint32_t mag, bool inf, int from, int lane) {
  uint32_t byte = need_byte(wave_max(mag), inf);
  Scales s;
  s.again = false;
  s.held = 1.0f;
  if (from > 0) {
    const uint32_t was = *at;
    s.held = scale_value(was);
    s.again = byte > was;
    byte = umax(byte, was);
  }
  if (lane == 0) *at = (uint8_t)byte;
  s.now = scale_value(byte);
  return s;
}

// All of an item's loads are issued at once, of rows that exist; what they
// bring for slots of no row is left out afterwards.
template <int D>
__device__ inline void append_keys(const CacheAppend& a, const Part& p, int64_t blk, int h, const double2* cs, int lane) {
  constexpr int P = D / 64;
  const int t = lane & 15, q = lane >> 4;
  const bool mine = t >= p.from && t < p.to;
  const uint16_t* row = a.k.p + (int64_t)(p.row0 + (mine ? t : p.from)) * a.k.tok + h * a.k.head;
  bq_u32x4 own[P][2], other[P][2];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = 64 * i + 16 * q + 8 * e;
      own[i][e] = row8(row + d);
      other[i][e] = row8(row + turn_of(d, a.rot, a.interleaved).other);
    }
  float f[P][16];
  uint32_t mag = 0;
  bool inf = false;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (a.rot) {
        double y[8];
        rotate8<double>(own[i][e], other[i][e], turn_of(64 * i + 16 * q + 8 * e, a.rot, a.interleaved), a.interleaved,
                        cs + t * angles_pitch(a.rot), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][8 * e + j] = to_odd(y[j]);
      } else {
        widen8(own[i][e], &f[i][8 * e]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) add_mag(f[i][8 * e + j], mag, inf);
    }
  const bool any_inf = __any(inf && mine);
  const Scales s = settle(a.c.scales + 2 * blk, mine ? mag : 0, any_inf, p.from, lane);
  uint8_t* at = a.c.k + blk * (kTok * D) + 16 * lane;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    bq_u32x4* const w = (bq_u32x4*)(at + 1024 * i);
    if (mine) {
      bq_u32x4 c;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = codes_of(f[i][4 * j], f[i][4 * j + 1], f[i][4 * j + 2], f[i][4 * j + 3], s.now, any_inf);
      *w = c;
    } else if (s.again && t < p.from) {
      bq_u32x4 c = *w;
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = recode(c[j], s.held, s.now);
      *w = c;
    }
  }
}

template <int D>
__device__ inline void append_values(const CacheAppend& a, const Part& p, int64_t blk, int h, int lane) {
  constexpr int W = D / 16;
  const int r = lane & 15, t0 = 4 * (lane >> 4);
  bq_u32x2 x[4][W / 4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int slot = t0 + t < p.from ? p.from : t0 + t < p.to ? t0 + t : p.to - 1;
    const uint16_t* row = a.v.p + (int64_t)(p.row0 + slot) * a.v.tok + h * a.v.head + W * r;
    if constexpr (W == 4) {
      x[t][0] = *(const bq_u32x2_a2*)row;
    } else {
#pragma unroll
      for (int j = 0; j < W / 8; ++j) {
        const bq_u32x4 v = row8(row + 8 * j);
        x[t][2 * j] = (bq_u32x2){v.x, v.y};
        x[t][2 * j + 1] = (bq_u32x2){v.z, v.w};
      }
    }
  }
  float f[4][W];
  uint32_t mag = 0, fresh = 0, before = 0;  // bytes of the slots of the batch, and of those before
  bool inf = false;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const bool mine = t0 + t >= p.from && t0 + t < p.to;
    fresh |= mine ? 0xFFu << (8 * t) : 0u;
    before |= t0 + t < p.from ? 0xFFu << (8 * t) : 0u;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t w = x[t][j / 4][j / 2 & 1];
      f[t][j] = mine ? __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16) : 0.0f;
      add_mag(f[t][j], mag, inf);
    }
  }
  const bool any_inf = __any(inf);
  const Scales s = settle(a.c.scales + 2 * blk + 1, mag, any_inf, p.from, lane);
  if (!fresh && !(s.again && before)) return;
  uint8_t* at = a.c.v + blk * (kTok * D) + 16 * lane;
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    bq_u32x4* const w = (bq_u32x4*)(at + 1024 * i);
    bq_u32x4 old = {0, 0, 0, 0}, c;
    if (fresh != 0xFFFFFFFFu) old = *w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * i + j;
      uint32_t keep = old[j];
      if (s.again) keep = (keep & ~before) | (recode(keep, s.held, s.now) & before);
      c[j] = (codes_of(f[0][e], f[1][e], f[2][e], f[3][e], s.now, any_inf) & fresh) | (keep & ~fresh);
    }
    *w = c;
  }
}

template <int D>
__device__ inline void rotate_queries(const CacheAppend& a, const Part& p, int h, const float2* cs, int lane) {
  constexpr int L = D / 8, N = kTok * L / 64;  // lanes a row; turns of 64 / L rows
  const int d = 8 * (lane % L);
  const Turn turn = turn_of(d, a.rot, a.interleaved);
  bq_u32x4 own[N], other[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = i * (64 / L) + lane / L, slot = t < p.from ? p.from : t < p.to ? t : p.to - 1;
    const uint16_t* row = a.q.p + (int64_t)(p.row0 + slot) * a.q.tok + h * a.q.head;
    own[i] = row8(row + d);
    other[i] = row8(row + turn.other);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = i * (64 / L) + lane / L;
    if (t < p.from || t >= p.to) continue;
    bq_u32x4 w = own[i];
    if (a.rot) {
      float y[8];
      rotate8<float>(own[i], other[i], turn, a.interleaved, cs + t * angles_pitch(a.rot), y);
      // what does not turn is copied as it is, a NaN with its bits
      const bq_u32x4 r = pack8(y);
      w = turn.turns ? r : w;
    }
    *(bq_u32x4_a2*)(a.qo.p + (int64_t)(p.row0 + t) * a.qo.tok + h * a.qo.head + d) = w;
  }
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void cache_append_kernel(CacheAppend a, int items) {
  extern __shared__ double2 cs[];  // cos, sin of [16 slots][rot / 2 + 1], then the same in 32 bits
  float2* const cs32 = (float2*)(cs + kTok * angles_pitch(a.rot));
  Part p;
  if (!part_of(a.b, blockIdx.x, p)) return;
  const int half = a.rot / 2;
  if (half) {
    for (int i = p.from * half + threadIdx.x; i < p.to * half; i += 64 * kWaves) {
      const int t = i / half, j = i - t * half;
      double s, c;
      sincos((double)(p.pos + t) * (double)a.freqs[j], &s, &c);
      cs[t * angles_pitch(a.rot) + j] = make_double2(c, s);
      cs32[t * angles_pitch(a.rot) + j] = make_float2((float)c, (float)s);
    }
    __syncthreads();
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int total = 2 * a.c.heads + a.q_heads;
  const int64_t first = block_at(a.c, a.b, p.seq, p.pos, 0);  // head 0's block; a page's heads follow each other
  for (int i = blockIdx.y * items + wave; i < (int)(blockIdx.y + 1) * items && i < total; i += kWaves) {
    if (i >= 2 * a.c.heads) {
      rotate_queries<D>(a, p, i - 2 * a.c.heads, cs32, lane);
      continue;
    }
    if (first < 0) continue;
    const int64_t blk = first + ((int64_t)(i >> 1) << (a.c.shift - 4));
    if (i & 1) append_values<D>(a, p, blk, i >> 1, lane);
    else append_keys<D>(a, p, blk, i >> 1, cs, lane);
  }
}

// ---- one token a sequence (a decode step) ----
//
// Nothing here waits for more than it must: a wave is alone (no barrier), its
// rows, its page and its angles are under way at once, and a lane has its own
// head, so that a wave stores the keys of 16 heads, the values of 4, or turns
// the queries of 64 / (D / 8). 173 sequences of 8 key and 64 query heads by
// the kernel above: 15.0 us, here 5.9.

struct One {
  int64_t pos, page;  // block number of head 0, or -1
  int slot;
};

// The earlier codes of a block to a new scale, by a whole wave; of values, only
// of the groups of 4 tokens before the new one's
template <int D>
__device__ inline void recode_block(uint8_t* at, int upto, float held, float now, bool values, int lane) {
  const bool mine = values ? (lane >> 4) < (upto >> 2) : (lane & 15) < upto;
  if (!mine) return;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    bq_u32x4* const w = (bq_u32x4*)(at + 1024 * i + 16 * lane);
    bq_u32x4 c = *w;
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = recode(c[j], held, now);
    *w = c;
  }
}
// for each head of a wave whose scale moved; lane l of `first`: a head's own lane
template <int D>
__device__ inline void recode_blocks(uint64_t moved, uint8_t* base, int64_t blk, int upto, const Scales& s, bool values,
                                     int lane) {
  while (moved) {
    const int l = __builtin_ctzll(moved);
    moved &= moved - 1;
    const int64_t b = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)blk, l) |
                      (int64_t)__builtin_amdgcn_readlane((int)(blk >> 32), l) << 32;
    recode_block<D>(base + b * (kTok * D), upto, __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s.held), l)),
                    __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s.now), l)), values, lane);
  }
}
__device__ inline Scales settle_one(uint32_t mag, bool inf, int slot, uint32_t was) {
  uint32_t byte = need_byte(mag, inf);
  Scales s;
  s.held = slot ? scale_value(was) : 1.0f;
  s.again = slot && byte > was;
  if (slot) byte = umax(byte, was);
  s.now = scale_value(byte);
  return s;
}
__device__ inline uint8_t byte_of(float scale) { return (uint8_t)(__float_as_uint(scale) >> 23); }

template <int D>
__device__ inline void append_key_one(const CacheAppend& a, const One& o, const bq_u32x4 (&own)[D / 64][2],
                                      const bq_u32x4 (&other)[D / 64][2], int64_t blk, bool have, uint32_t was,
                                      const double2* cs, int lane) {
  constexpr int P = D / 64;
  const int q = lane >> 4;
  float f[P][16];
  uint32_t mag = 0;
  bool inf = false;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (a.rot) {
        double y[8];
        rotate8<double>(own[i][e], other[i][e], turn_of(64 * i + 16 * q + 8 * e, a.rot, a.interleaved), a.interleaved, cs, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][8 * e + j] = to_odd(y[j]);
      } else {
        widen8(own[i][e], &f[i][8 * e]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) add_mag(f[i][8 * e + j], mag, inf);
    }
  const auto mx = [](uint32_t x, uint32_t y) { return umax(x, y); };
  mag = swap16_max(mag, mag, mx);
  mag = swap32_max(mag, mag, mx);
  uint32_t odd = inf;
  if (__any(inf)) {
    odd = swap16_max(odd, odd, mx);
    odd = swap32_max(odd, odd, mx);
  }
  const Scales s = settle_one(mag, odd, o.slot, was);
  if (have) {
    uint8_t* at = a.c.k + blk * (kTok * D) + 16 * (16 * q + o.slot);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      bq_u32x4 c;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = codes_of(f[i][4 * j], f[i][4 * j + 1], f[i][4 * j + 2], f[i][4 * j + 3], s.now, odd);
      *(bq_u32x4*)(at + 1024 * i) = c;
    }
    if (q == 0) a.c.scales[2 * blk] = byte_of(s.now);
  }
  recode_blocks<D>(__ballot(have && q == 0 && s.again), a.c.k, blk, o.slot, s, false, lane);
}

template <int D>
__device__ inline void append_value_one(const CacheAppend& a, const One& o, const bq_u32x2 (&x)[D / 64], int64_t blk,
                                        bool have, uint32_t was, int lane) {
  constexpr int W = D / 16;
  const int r = lane & 15;
  float f[W];
  uint32_t mag = 0;
  bool inf = false;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const uint32_t w = x[j / 4][j / 2 & 1];
    f[j] = __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
    add_mag(f[j], mag, inf);
  }
  mag = row16_max(mag);
  uint32_t odd = inf;
  if (__any(inf)) odd = row16_max(odd);
  const Scales s = settle_one(mag, odd, o.slot, was);
  if (have) {
    uint8_t* at = a.c.v + blk * (kTok * D) + 16 * (16 * (o.slot >> 2) + r);
    const int sh = 8 * (o.slot & 3);
    const uint32_t mine = 0xFFu << sh, early = (1u << sh) - 1u;  // bytes of the token and of those before
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      bq_u32x4* const w = (bq_u32x4*)(at + 1024 * i);
      bq_u32x4 c = *w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t code = codes_of(f[4 * i + j], 0, 0, 0, s.now, odd) & 0xFFu;
        uint32_t keep = c[j];
        if (s.again) keep = (keep & ~early) | (recode(keep, s.held, s.now) & early);
        c[j] = (keep & ~mine) | code << sh;
      }
      *w = c;
    }
    if (r == 0) a.c.scales[2 * blk + 1] = byte_of(s.now);
  }
  recode_blocks<D>(__ballot(have && r == 0 && s.again), a.c.v, blk, o.slot, s, true, lane);
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void cache_append_one_kernel(CacheAppend a) {
  constexpr int P = D / 64, L = D / 8;
  // each wave its own: cos, sin, then the same in 32 bits
  __shared__ double2 cs_all[kWaves][128];
  __shared__ float2 cs32_all[kWaves][128];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int keys = (a.c.heads + 15) / 16, values = (a.c.heads + 3) / 4;
  const int queries = (a.q_heads + 64 / L - 1) / (64 / L);
  const int item = blockIdx.y * kWaves + wave, seq = blockIdx.x, half = a.rot / 2;
  if (item >= keys + values + queries) return;
  const bool is_key = item < keys, is_value = !is_key && item < keys + values;
  One o;
  const int len = a.b.lengths[seq];
  o.pos = (int64_t)(len > 0 ? len : 0) - 1;
  o.slot = (int)(o.pos & 15);
  // rows first: they wait for nothing
  bq_u32x4 own[P][2], other[P][2];
  bq_u32x2 x[P];
  int h = 0;
  if (is_key) {
    h = 16 * item + (lane & 15);
    const uint16_t* row = a.k.p + seq * a.k.tok + (h < a.c.heads ? h : a.c.heads - 1) * a.k.head;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = 64 * i + 16 * (lane >> 4) + 8 * e;
        own[i][e] = row8(row + d);
        other[i][e] = row8(row + turn_of(d, a.rot, a.interleaved).other);
      }
  } else if (is_value) {
    h = 4 * (item - keys) + (lane >> 4);
    const uint16_t* row = a.v.p + seq * a.v.tok + (h < a.c.heads ? h : a.c.heads - 1) * a.v.head + D / 16 * (lane & 15);
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = *(const bq_u32x2_a2*)(row + 4 * i);
  } else {
    h = 64 / L * (item - keys - values) + lane / L;
    const uint16_t* row = a.q.p + seq * a.q.tok + (h < a.q_heads ? h : a.q_heads - 1) * a.q.head;
    const int d = 8 * (lane % L);
    own[0][0] = row8(row + d);
    other[0][0] = row8(row + turn_of(d, a.rot, a.interleaved).other);
  }
  const bool stores = is_key || is_value;
  const int64_t first = stores ? block_at(a.c, a.b, seq, o.pos - o.slot, 0) : -1;
  const bool have = first >= 0 && h < a.c.heads;
  const int64_t blk = have ? first + ((int64_t)h << (a.c.shift - 4)) : 0;
  const uint32_t was = have && o.slot ? a.c.scales[2 * blk + is_value] : 0u;
  double2* const cs = cs_all[wave];
  float2* const cs32 = cs32_all[wave];
  if (!is_value)
    for (int j = lane; j < half; j += 64) {
      double s, c;
      sincos((double)o.pos * (double)a.freqs[j], &s, &c);
      cs[j] = make_double2(c, s);
      cs32[j] = make_float2((float)c, (float)s);
    }
  // the wave's own lanes read them: LDS serves a wave in order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  if (is_key) append_key_one<D>(a, o, own, other, blk, have, was, cs, lane);
  else if (is_value) append_value_one<D>(a, o, x, blk, have, was, lane);
  else if (h < a.q_heads) {
    const int d = 8 * (lane % L);
    const Turn turn = turn_of(d, a.rot, a.interleaved);
    bq_u32x4 w = own[0][0];
    if (a.rot) {
      float y[8];
      rotate8<float>(own[0][0], other[0][0], turn, a.interleaved, cs32, y);
      const bq_u32x4 r = pack8(y);
      w = turn.turns ? r : w;
    }
    *(bq_u32x4_a2*)(a.qo.p + seq * a.qo.tok + h * a.qo.head + d) = w;
  }
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void cache_read_kernel(Cache c, CacheBatch b, CacheRows k, CacheRows v,
                                                                 int items) {
  Part p;
  if (!part_of(b, blockIdx.x, p)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lo = lane & 15, hi = lane >> 4;
  const int64_t first = block_at(c, b, p.seq, p.pos, 0);
  for (int i = blockIdx.y * items + wave; i < (int)(blockIdx.y + 1) * items && i < 2 * c.heads; i += kWaves) {
    const int h = i >> 1;
    const int64_t blk = first < 0 ? -1 : first + ((int64_t)h << (c.shift - 4));
    const float s = blk < 0 ? 1.0f : scale_value(c.scales[2 * blk + (i & 1)]);
    const uint8_t* at = (i & 1 ? c.v : c.k) + blk * (kTok * D) + 16 * lane;
    bq_u32x4 w[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) w[j] = blk < 0 ? (bq_u32x4){0, 0, 0, 0} : *(const bq_u32x4*)(at + 1024 * j);
    if (i & 1) {
      // four tokens of D / 16 elements: tokens' bytes apart, then widened
      constexpr int W = D / 16;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int slot = 4 * hi + t;
        if (slot < p.from || slot >= p.to) continue;
        uint16_t* o = v.p + (int64_t)(p.row0 + slot) * v.tok + h * v.head + W * lo;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t e = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) e |= (w[j][x] >> (8 * t) & 0xFFu) << (8 * x);
          const bq_u32x4 y = uncode8_bf16<FP8_E4M3>(make_uint2(e, 0), s);
          *(bq_u32x2_a2*)(o + 4 * j) = (bq_u32x2){y.x, y.y};
        }
      }
    } else if (lo >= p.from && lo < p.to) {
      uint16_t* o = k.p + (int64_t)(p.row0 + lo) * k.tok + h * k.head + 16 * hi;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        *(bq_u32x4_a2*)(o + 64 * j) = uncode8_bf16<FP8_E4M3>(make_uint2(w[j].x, w[j].y), s);
        *(bq_u32x4_a2*)(o + 64 * j + 8) = uncode8_bf16<FP8_E4M3>(make_uint2(w[j].z, w[j].w), s);
      }
    }
  }
}

// Items a workgroup takes of its block's: all of them where there are blocks
// enough for the chip, as few as one a wave where there are not.
inline int items_of(unsigned parts, int total, unsigned most) {
  const unsigned groups = parts >= most ? 1 : (most + parts - 1) / parts;
  const int n = (int)((total + groups - 1) / groups);
  return n < kWaves ? kWaves : n;
}

// Workgroups that an append (whose angles each of a block's computes anew) and
// a read are spread over: 8200 tokens, 40 heads: 134, 126 and 138 us with 1024,
// 2048 and 4096 of an append; 69, 57 and 52 us of a read.
constexpr unsigned kAppendGroups = 2048, kReadGroups = 4096;

}  // namespace

hipError_t launch_cache_append(const CacheAppend& a, int head_dim, hipStream_t st) {
  const unsigned parts = parts_of(a.b);
  if (!parts || !a.b.tokens || !a.b.sequences) return hipSuccess;
  if (!a.b.starts) {
    const int row = head_dim / 8, items = (a.c.heads + 15) / 16 + (a.c.heads + 3) / 4 + (a.q_heads + 64 / row - 1) / (64 / row);
    const dim3 grid(parts, (items + kWaves - 1) / kWaves);
    if (head_dim == 64) cache_append_one_kernel<64><<<grid, 64 * kWaves, 0, st>>>(a);
    else if (head_dim == 128) cache_append_one_kernel<128><<<grid, 64 * kWaves, 0, st>>>(a);
    else cache_append_one_kernel<256><<<grid, 64 * kWaves, 0, st>>>(a);
    return hipGetLastError();
  }
  const int total = 2 * a.c.heads + a.q_heads, items = items_of(parts, total, kAppendGroups);
  const dim3 grid(parts, (total + items - 1) / items);
  const size_t lds = (size_t)kTok * angles_pitch(a.rot) * (sizeof(double2) + sizeof(float2));
  if (head_dim == 64) cache_append_kernel<64><<<grid, 64 * kWaves, lds, st>>>(a, items);
  else if (head_dim == 128) cache_append_kernel<128><<<grid, 64 * kWaves, lds, st>>>(a, items);
  else cache_append_kernel<256><<<grid, 64 * kWaves, lds, st>>>(a, items);
  return hipGetLastError();
}

hipError_t launch_cache_read(const Cache& c, const CacheBatch& b, const CacheRows& k, const CacheRows& v, int head_dim,
                             hipStream_t st) {
  const unsigned parts = parts_of(b);
  if (!parts || !b.tokens || !b.sequences) return hipSuccess;
  const int items = items_of(parts, 2 * c.heads, kReadGroups);
  const dim3 grid(parts, (2 * c.heads + items - 1) / items);
  if (head_dim == 64) cache_read_kernel<64><<<grid, 64 * kWaves, 0, st>>>(c, b, k, v, items);
  else if (head_dim == 128) cache_read_kernel<128><<<grid, 64 * kWaves, 0, st>>>(c, b, k, v, items);
  else cache_read_kernel<256><<<grid, 64 * kWaves, 0, st>>>(c, b, k, v, items);
  return hipGetLastError();
}

}  // namespace fp8lin
