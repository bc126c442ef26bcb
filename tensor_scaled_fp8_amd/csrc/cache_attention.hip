// Attention over the paged 8-bit cache.
//
// A workgroup takes R = 16 rows of one key head, a row being one of the
// head's queries of one token, and the tokens they see; its waves share out
// the tokens, 32 (two blocks) at a time, each with a softmax of its own
// (running maximum, sum, weighted values), joined over LDS at the end.
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
#include "cache.h"

namespace fp8lin {
namespace {

constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;

typedef __bf16 ca_bf16x8 __attribute__((ext_vector_type(8)));
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
__device__ inline bq_f32x4 mma(ca_bf16x8 a, ca_bf16x8 b, bq_f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float nan() { return __uint_as_float(0x7FC00000u); }

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

// bytes of w that are codes of NaN, as 0xFF
__device__ inline uint32_t nan_bytes(uint32_t w) {
  const uint32_t m = (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
  return m * 0xFFu;
}

template <int D>
struct State {
  float m, l;  // of this lane's row; l over this lane's tokens
  bq_f32x4 o[D / 16];
};

// One row's tile of a sequence
struct Tile {
  int seq, h;
  Seq s;
  int r0;          // its first row of the sequence's n * group
  int first, last; // positions of the first and the last row's token (last < first: no rows)
};

// 32 tokens from j0 into a wave's state. HARD: the mask hides some of them
// from some rows; pos is the lane's row's position (-1: no row).
template <int D, bool CAP>
__device__ inline void attend_group(const CacheAttend& a, const Tile& t, int64_t j0, int hi, int pos,
                                    const ca_bf16x8 (&qf)[D / 32], State<D>& st, int lane) {
  constexpr int P = D / 64;
  const int lo16 = lane & 15, g = lane >> 4;
  ca_u32x4 kc[2][P], vc[2][P];
  float ks[2], vs[2];
  bool there[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t blk = j0 + 16 * b < hi ? block_at(a.c, a.b, t.seq, j0 + 16 * b, t.h) : -1;
    there[b] = blk >= 0;
    ks[b] = vs[b] = 1.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) kc[b][i] = vc[b][i] = (ca_u32x4){0, 0, 0, 0};
    if (there[b]) {
      const uint32_t sc = *(const uint16_t*)(a.c.scales + 2 * blk);
      ks[b] = scale_value(sc & 0xFFu);
      vs[b] = scale_value(sc >> 8);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        kc[b][i] = *(const ca_u32x4*)(a.c.k + blk * (kTok * D) + 1024 * i + 16 * lane);
        vc[b][i] = *(const ca_u32x4*)(a.c.v + blk * (kTok * D) + 1024 * i + 16 * lane);
      }
    }
  }
  float s[8];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    bq_f32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c = mma(widen(kc[b][i].x, ks[b], kc[b][i].y, ks[b]), qf[2 * i], c);
      c = mma(widen(kc[b][i].z, ks[b], kc[b][i].w, ks[b]), qf[2 * i + 1], c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[4 * b + i] = c[i] * a.scale;
      if constexpr (CAP) s[4 * b + i] = a.cap * tanh_(s[4 * b + i] / a.cap);
      s[4 * b + i] *= kLog2e;
    }
  }
  // hidden from somebody: the rows' positions are first .. last
  const bool hard = !there[0] || !there[1] || j0 + 31 > t.first || (a.window > 0 && j0 <= (int64_t)t.last - a.window);
  bool seen[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) seen[i] = true;
  if (hard) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t j = j0 + 16 * (i >> 2) + 4 * g + (i & 3);
      seen[i] = there[i >> 2] && j <= pos && (a.window <= 0 || j > (int64_t)pos - a.window);
      if (!seen[i]) s[i] = -__builtin_inff();
    }
  }
  float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
  if (__any(top > st.m + kSlack)) {
    const float m = fmaxf(quad_max(top), st.m);
    const float f = m == st.m ? 1.0f : exp2_(st.m - m);
    st.m = m;
    st.l *= f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i] *= f;
  }
  const float base = st.m == -__builtin_inff() ? 0.0f : st.m;
  ca_u32x4 pw;
  float p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = exp2_(s[i] - base);
    st.l += p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) pw[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
  const ca_bf16x8 pf = __builtin_bit_cast(ca_bf16x8, pw);
  if (hard) {
    // a hidden token's weight is 0, but a NaN times 0 is one: the NaNs are
    // taken out of the product, and given to the rows that see them
    uint32_t any = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) any |= nan_bytes(vc[b][i][k]);
    if (__any(any != 0)) {
      ca_u32x4 sw;
#pragma unroll
      for (int i = 0; i < 4; ++i) sw[i] = (seen[2 * i] ? 0x3F80u : 0u) | (seen[2 * i + 1] ? 0x3F800000u : 0u);
      const ca_bf16x8 sf = __builtin_bit_cast(ca_bf16x8, sw);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t n[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          n[b] = nan_bytes(vc[b][i / 4][i % 4]);
          vc[b][i / 4][i % 4] &= ~n[b];
          n[b] &= 0x38383838u;  // 1
        }
        const bq_f32x4 c = mma(widen(n[0], 1.0f, n[1], 1.0f), sf, (bq_f32x4){0, 0, 0, 0});
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c[k] > 0) st.o[i][k] = nan();
      }
    }
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    st.o[i] = mma(widen(vc[0][i / 4][i % 4], vs[0], vc[1][i / 4][i % 4], vs[1]), pf, st.o[i]);
}

// The tile that virtual tile v is: sequence i's tiles of R rows start at
// starts[i] group / R + i
template <int R>
__device__ inline bool tile_of(const CacheAttend& a, int64_t v, int h, Tile& t) {
  int64_t at;
  if (a.b.starts) {
    const auto first = [&](int j) { return (int64_t)start_of(a.b, j) * a.group / R + j; };
    t.seq = last_upto(a.b.sequences, v, first);
    at = v - first(t.seq);
  } else {
    const int per = (a.group + R - 1) / R;
    t.seq = (int)(v / per);
    at = v - (int64_t)t.seq * per;
  }
  t.h = h;
  t.s = seq_of(a.b, t.seq);
  const int64_t rows = (int64_t)t.s.n * a.group;
  if (at < 0 || at * R >= rows) return false;
  t.r0 = (int)(at * R);
  const int64_t end = at * R + R < rows ? at * R + R : rows;
  t.first = (int)(t.s.p0 + t.r0 / a.group);
  t.last = (int)(t.s.p0 + (end - 1) / a.group);
  return true;
}

template <int D, bool CAP>
__global__ __launch_bounds__(64 * kWaves) void cache_attention_kernel(CacheAttend a) {
  constexpr int R = 16, W = D / 16;
  constexpr int C = W < 8 ? W : 8;  // joined at a time
  __shared__ float acc[kWaves][4][C][64];
  __shared__ float ml[kWaves][2][R];
  Tile t;
  if (!tile_of<R>(a, blockIdx.x / a.c.heads, blockIdx.x % a.c.heads, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lo16 = lane & 15, g = lane >> 4;
  const int64_t row = t.r0 + lo16;
  const bool mine = row < (int64_t)t.s.n * a.group;
  const int tok = (int)(row / a.group), head = t.h * a.group + (int)(row % a.group);
  const int pos = mine ? (int)(t.s.p0 + tok) : -1;
  const int64_t have = a.b.table_pages << a.c.shift;
  const int hi = (int)(t.last + 1 < have ? t.last + 1 : have);
  const int64_t from = a.window > 0 && (int64_t)t.first - a.window + 1 > 0 ? (int64_t)t.first - a.window + 1 : 0;
  ca_bf16x8 qf[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    ca_u32x4 w = {0, 0, 0, 0};
    if (mine)
      w = *(const bq_u32x4_a2*)(a.q.p + (int64_t)(t.s.row0 + tok) * a.q.tok + head * a.q.head + 64 * (i / 2) + 16 * g +
                                8 * (i % 2));
    qf[i] = __builtin_bit_cast(ca_bf16x8, w);
  }
  State<D> st;
  st.m = -__builtin_inff();
  st.l = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) st.o[i] = (bq_f32x4){0, 0, 0, 0};
  for (int64_t j0 = (from / 32 + wave) * 32; j0 < hi; j0 += 32 * kWaves)
    attend_group<D, CAP>(a, t, j0, hi, pos, qf, st, lane);
  const float l = quad_sum(st.l);
  if (lane < R) {
    ml[wave][0][lane] = st.m;
    ml[wave][1][lane] = l;
  }
  __syncthreads();
  float m = ml[0][0][lo16], sum = 0, f[kWaves];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, ml[w][0][lo16]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float mw = ml[w][0][lo16];
    f[w] = mw == m ? 1.0f : exp2_(mw - m);
    sum += ml[w][1][lo16] * f[w];
  }
  const int64_t tr = t.s.row0 + tok;
  const float inv = sum == 0 ? 0.0f : 1.0f / sum;
  uint16_t* out = a.out.p + tr * a.out.tok + head * a.out.head + W * (4 * g + wave);
#pragma unroll
  for (int c = 0; c < W; c += C) {
    if (c) __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < C; ++i) acc[wave][k][i][lane] = st.o[c + i][k];
    __syncthreads();
    float o[C];
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] += acc[w][wave][i][lane] * f[w];
    if (mine)
#pragma unroll
      for (int i = 0; i < C; i += 4)
        *(bq_u32x2_a2*)(out + c + i) =
            (bq_u32x2){pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv)};
  }
  if (mine && a.lse && wave == 0 && g == 0)
    a.lse[tr * a.q_heads + head] = sum == 0 ? -__builtin_inff() : (m + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

template <int D>
hipError_t run(const CacheAttend& a, hipStream_t st) {
  const int64_t tiles = a.b.starts ? (int64_t)a.b.tokens * a.group / 16 + a.b.sequences
                                   : (int64_t)a.b.sequences * ((a.group + 15) / 16);
  const unsigned grid = (unsigned)(tiles * a.c.heads);
  if (a.cap > 0) cache_attention_kernel<D, true><<<grid, 64 * kWaves, 0, st>>>(a);
  else cache_attention_kernel<D, false><<<grid, 64 * kWaves, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t cache_attention_ws_bytes(const CacheAttend&, int) { return 0; }

hipError_t launch_cache_attention(const CacheAttend& a, int head_dim, void*, hipStream_t st) {
  if (!a.b.tokens || !a.b.sequences) return hipSuccess;
  return head_dim == 64 ? run<64>(a, st) : head_dim == 128 ? run<128>(a, st) : run<256>(a, st);
}

}  // namespace fp8lin
