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
__device__ inline float clamp448(float f, float scale) {
  const float m = 448.0f * scale;
  return f != f ? f : fminf(fmaxf(f, -m), m);
}
// codes of four values; beyond the format's largest only if an infinity is among them
__device__ inline uint32_t codes_of(float a, float b, float c, float d, float s, bool inf) {
  if (inf) return code4<FP8_E4M3>(clamp448(a, s), clamp448(b, s), clamp448(c, s), clamp448(d, s), s);
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

__device__ inline void load8(const uint16_t* p, float f[8]) { widen8(*(const bq_u32x4_a2*)p, f); }

// 8 elements from d (a multiple of 8) of a row, rotated. T: the precision.
template <typename T>
__device__ inline void rotated8(const uint16_t* row, int d, int rot, int inter, const double2* cs, T y[8]) {
  float x[8];
  load8(row + d, x);
  if (d >= rot) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j];
  } else if (inter) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double2 t = cs[d / 2 + j];
      const T c = (T)t.x, s = (T)t.y, a = x[2 * j], b = x[2 * j + 1];
      y[2 * j] = a * c - b * s;
      y[2 * j + 1] = b * c + a * s;
    }
  } else {
    const int half = rot / 2;
    const bool low = d < half;
    const int j0 = low ? d : d - half;
    float o[8];
    load8(row + (low ? d + half : j0), o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double2 t = cs[j0 + j];
      const T c = (T)t.x, s = low ? -(T)t.y : (T)t.y;
      y[j] = (T)x[j] * c + (T)o[j] * s;
    }
  }
}

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

template <int D>
__device__ inline void append_keys(const CacheAppend& a, const Part& p, int64_t blk, int h, const double2* cs, int lane) {
  constexpr int P = D / 64;
  const int t = lane & 15, q = lane >> 4;
  const bool mine = t >= p.from && t < p.to;
  float f[P][16];
  uint32_t mag = 0;
  bool inf = false;
  if (mine) {
    const uint16_t* row = a.k.p + (int64_t)(p.row0 + t) * a.k.tok + h * a.k.head;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        double y[8];
        rotated8<double>(row, 64 * i + 16 * q + 8 * e, a.rot, a.interleaved, cs + t * (a.rot / 2), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[i][8 * e + j] = to_odd(y[j]);
          add_mag(f[i][8 * e + j], mag, inf);
        }
      }
  }
  const bool any_inf = __any(inf);
  const Scales s = settle(a.c.scales + 2 * blk, mag, any_inf, p.from, lane);
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
  float f[4][W];
  uint32_t mag = 0, fresh = 0;  // fresh: bytes of the slots of the batch
  bool inf = false;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int j = 0; j < W; ++j) f[t][j] = 0.0f;
    if (t0 + t >= p.from && t0 + t < p.to) {
      fresh |= 0xFFu << (8 * t);
      const uint16_t* row = a.v.p + (int64_t)(p.row0 + t0 + t) * a.v.tok + h * a.v.head + W * r;
      if constexpr (W == 4) {
        const bq_u32x2 w = *(const bq_u32x2_a2*)row;
        f[t][0] = __uint_as_float(w.x << 16);
        f[t][1] = __uint_as_float(w.x & 0xFFFF0000u);
        f[t][2] = __uint_as_float(w.y << 16);
        f[t][3] = __uint_as_float(w.y & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int j = 0; j < W; j += 8) load8(row + j, &f[t][j]);
      }
#pragma unroll
      for (int j = 0; j < W; ++j) add_mag(f[t][j], mag, inf);
    }
  }
  const bool any_inf = __any(inf);
  const Scales s = settle(a.c.scales + 2 * blk + 1, mag, any_inf, p.from, lane);
  uint32_t before = 0;  // bytes of the slots before the batch's
#pragma unroll
  for (int t = 0; t < 4; ++t) before |= t0 + t < p.from ? 0xFFu << (8 * t) : 0u;
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
__device__ inline void rotate_queries(const CacheAppend& a, const Part& p, int h, const double2* cs, int lane) {
  constexpr int L = D / 8;  // lanes a row
  const int d = 8 * (lane % L);
  for (int t = p.from + lane / L; t < p.to; t += 64 / L) {
    const int64_t row = p.row0 + t;
    float y[8];
    rotated8<float>(a.q.p + row * a.q.tok + h * a.q.head, d, a.rot, a.interleaved, cs + t * (a.rot / 2), y);
    *(bq_u32x4_a2*)(a.qo.p + row * a.qo.tok + h * a.qo.head + d) = pack8(y);
  }
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void cache_append_kernel(CacheAppend a, int items) {
  extern __shared__ double2 cs[];  // cos, sin of [16 slots][rot / 2]
  Part p;
  if (!part_of(a.b, blockIdx.x, p)) return;
  const int half = a.rot / 2;
  if (half) {
    for (int i = p.from * half + threadIdx.x; i < p.to * half; i += 64 * kWaves) {
      const int t = i / half;
      double s, c;
      sincos((double)(p.pos + t) * (double)a.freqs[i - t * half], &s, &c);
      cs[i] = make_double2(c, s);
    }
    __syncthreads();
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int total = 2 * a.c.heads + a.q_heads;
  for (int i = blockIdx.y * items + wave; i < (int)(blockIdx.y + 1) * items && i < total; i += kWaves) {
    if (i >= 2 * a.c.heads) {
      rotate_queries<D>(a, p, i - 2 * a.c.heads, cs, lane);
      continue;
    }
    const int64_t blk = block_at(a.c, a.b, p.seq, p.pos, i >> 1);
    if (blk < 0) continue;
    if (i & 1) append_values<D>(a, p, blk, i >> 1, lane);
    else append_keys<D>(a, p, blk, i >> 1, cs, lane);
  }
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void cache_read_kernel(Cache c, CacheBatch b, CacheRows k, CacheRows v,
                                                                 int items) {
  Part p;
  if (!part_of(b, blockIdx.x, p)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lo = lane & 15, hi = lane >> 4;
  for (int i = blockIdx.y * items + wave; i < (int)(blockIdx.y + 1) * items && i < 2 * c.heads; i += kWaves) {
    const int h = i >> 1;
    const int64_t blk = block_at(c, b, p.seq, p.pos, h);
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
inline int items_of(unsigned parts, int total) {
  const unsigned groups = parts >= 1024 ? 1 : (1024 + parts - 1) / parts;
  const int n = (int)((total + groups - 1) / groups);
  return n < kWaves ? kWaves : n;
}

}  // namespace

hipError_t launch_cache_append(const CacheAppend& a, int head_dim, hipStream_t st) {
  const unsigned parts = parts_of(a.b);
  if (!parts || !a.b.tokens) return hipSuccess;
  const int total = 2 * a.c.heads + a.q_heads, items = items_of(parts, total);
  const dim3 grid(parts, (total + items - 1) / items);
  const size_t lds = (size_t)kTok * (a.rot / 2) * sizeof(double2);
  if (head_dim == 64) cache_append_kernel<64><<<grid, 64 * kWaves, lds, st>>>(a, items);
  else if (head_dim == 128) cache_append_kernel<128><<<grid, 64 * kWaves, lds, st>>>(a, items);
  else cache_append_kernel<256><<<grid, 64 * kWaves, lds, st>>>(a, items);
  return hipGetLastError();
}

hipError_t launch_cache_read(const Cache& c, const CacheBatch& b, const CacheRows& k, const CacheRows& v, int head_dim,
                             hipStream_t st) {
  const unsigned parts = parts_of(b);
  if (!parts || !b.tokens) return hipSuccess;
  const int items = items_of(parts, 2 * c.heads);
  const dim3 grid(parts, (2 * c.heads + items - 1) / items);
  if (head_dim == 64) cache_read_kernel<64><<<grid, 64 * kWaves, 0, st>>>(c, b, k, v, items);
  else if (head_dim == 128) cache_read_kernel<128><<<grid, 64 * kWaves, 0, st>>>(c, b, k, v, items);
  else cache_read_kernel<256><<<grid, 64 * kWaves, 0, st>>>(c, b, k, v, items);
  return hipGetLastError();
}

}  // namespace fp8lin
