// Device pieces shared by the block-scaled quantise and SwiGLU kernels.
//
// Codes come straight from v_cvt_scalef32_pk_{fp8,bf8}_{bf16,f32}, which
// divides by the scale and rounds once to nearest even: 2 elements an
// instruction, no multiply, and bf16 inputs are never widened. Checked
// against a multiply and the plain conversion: the same codes for every
// bf16 value and scale. Maxima of bf16 are taken two at a time on their
// magnitude bits. These kernels run each instruction once a workgroup, so
// their code is kept small: an 18 KB body of branches cost 11 us a launch,
// whatever the matrix, in instruction fetches alone.
#pragma once

#include "block.h"

namespace fp8lin {

typedef unsigned int bq_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int bq_u32x2 __attribute__((ext_vector_type(2)));
typedef bq_u32x4 bq_u32x4_a2 __attribute__((aligned(2)));  // a row of an odd pitch starts at any 2 bytes
typedef bq_u32x2 bq_u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t bq_u32_a2 __attribute__((aligned(2)));
typedef float bq_f32x2 __attribute__((ext_vector_type(2)));
typedef float bq_f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bq_bf16x2 __attribute__((ext_vector_type(2)));
typedef short bq_s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short bq_u16x2 __attribute__((ext_vector_type(2)));

__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ inline uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(bq_u16x2, a),
                                                                __builtin_bit_cast(bq_u16x2, b)));
}
__device__ inline uint32_t pk_min(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(bq_u16x2, a),
                                                                __builtin_bit_cast(bq_u16x2, b)));
}
// |a| or |b|, the larger; a NaN if either is one (v_maximum3_f32)
__device__ inline float nan_max(float a, float b) {
  return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}

// max over the 16 lanes that share t / 16 (one DPP row)
__device__ inline uint32_t row16_max(uint32_t m) {
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));   // lanes ^ 1
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));   // lanes ^ 2
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, true));  // half-row mirror
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, true));  // row mirror
  return m;
}

// Scale byte 127 - bias from the bits of a block's max |x| in 32 bits. The
// sum carries into the exponent exactly if the significand is above 1.75;
// an amax below the normal range gives the largest bias, 126 (byte 1), by
// itself. 0, infinity and NaN: bias 0.
template <int FMT>
__device__ inline uint32_t scale_byte(uint32_t mag) {
  constexpr int kTop = FMT == FP8_E4M3 ? kTopExpE4M3 : kTopExpE5M2;
  const int e = (int)((mag + 0x1FFFFFu) >> 23) - kTop;
  return mag - 1u < 0x7F7FFFFFu ? (uint32_t)(e > 1 ? e : 1) : 127u;
}
// 2^(byte - 127); bytes are 1 .. 253
__device__ inline float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

template <int FMT, bool HI>
__device__ inline uint32_t code2(uint32_t old, uint32_t pair, float scale) {  // two bf16
  const bq_s16x2 o = __builtin_bit_cast(bq_s16x2, old);
  const bq_bf16x2 v = __builtin_bit_cast(bq_bf16x2, pair);
  if constexpr (FMT == FP8_E4M3)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, scale, HI));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(o, v, scale, HI));
}
template <int FMT, bool HI>
__device__ inline uint32_t code2(uint32_t old, float a, float b, float scale) {
  const bq_s16x2 o = __builtin_bit_cast(bq_s16x2, old);
  if constexpr (FMT == FP8_E4M3)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, HI));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(o, a, b, scale, HI));
}
template <int FMT>
__device__ inline uint32_t code4(uint32_t p0, uint32_t p1, float s) {
  return code2<FMT, true>(code2<FMT, false>(0, p0, s), p1, s);
}
template <int FMT>
__device__ inline uint32_t code4(float a, float b, float c, float d, float s) {
  return code2<FMT, true>(code2<FMT, false>(0, a, b, s), c, d, s);
}

// A block with an infinity or a NaN has scale 1: its values are clamped to
// the format's largest, a NaN stays one. Such blocks are rare: callers
// branch round this for a whole wave.
template <int FMT>
__device__ inline uint32_t clamp_pair(uint32_t pair, bool odd) {
  constexpr uint32_t kMax = FMT == FP8_E4M3 ? 0x43E0u : 0x4760u;  // 448, 57344 in bf16
  const uint32_t m = pair & 0x7FFF7FFFu;
  uint32_t r = pk_min(m, kMax | kMax << 16);
  if ((m & 0xFFFFu) > 0x7F80u) r |= 0x7FFFu;
  if ((m >> 16) > 0x7F80u) r |= 0x7FFF0000u;
  return odd ? r | (pair & 0x80008000u) : pair;
}
template <int FMT>
__device__ inline float clamp_one(float f, bool odd) {
  constexpr float kMax = FMT == FP8_E4M3 ? 448.0f : 57344.0f;
  return !odd || f != f ? f : fminf(fmaxf(f, -kMax), kMax);
}

// 8 bf16 (four dwords) to 32 bits
__device__ inline void widen8(bq_u32x4 w, float f[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// Rows r, r + STEP, ... (N of them), columns cx .. cx + 7, of a matrix;
// zeros past its ends; in-bounds for any pitch. `inside` (the same for the
// whole workgroup): all of it exists. Otherwise each load is of the nearest
// 8 columns and row that do exist, shifted and masked after all are issued;
// matrices of fewer than 8 columns are gathered. ONCE: nobody else reads it.
template <int N, int STEP, bool ONCE = true>
__device__ inline void load_rows(const Bf16Mat& x, int64_t r, int64_t cx, bool inside, bq_u32x4 (&w)[N]) {
  if (inside) {
    const uint16_t* p = x.p + r * x.ld + cx;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bq_u32x4_a2* q = (const bq_u32x4_a2*)(p + i * STEP * x.ld);
      if constexpr (ONCE) w[i] = __builtin_nontemporal_load(q);
      else w[i] = *q;
    }
    return;
  }
  if (x.cols < 8) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = (bq_u32x4){0, 0, 0, 0};
#pragma clang loop unroll(disable)
    for (int k = 0; k < x.cols; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (r + i * STEP < x.rows && cx == 0) {
          const uint32_t e = (uint32_t)x.p[(r + i * STEP) * x.ld + k] << (16 * (k & 1));
          w[i].x |= k >> 1 == 0 ? e : 0;
          w[i].y |= k >> 1 == 1 ? e : 0;
          w[i].z |= k >> 1 == 2 ? e : 0;
          w[i].w |= k >> 1 == 3 ? e : 0;
        }
    return;
  }
  const int64_t c = cx + 8 <= x.cols ? cx : x.cols - 8;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t q = r + i * STEP < x.rows ? r + i * STEP : x.rows - 1;
    w[i] = *(const bq_u32x4_a2*)(x.p + q * x.ld + c);
  }
  const int sh = 16 * (int)(cx - c);  // bits of 128 that belong to earlier columns
  const bool far = sh >= 64;
  const int s = sh & 63;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool none = r + i * STEP >= x.rows || sh >= 128;
    const uint64_t lo = (uint64_t)w[i].y << 32 | w[i].x, hi = (uint64_t)w[i].w << 32 | w[i].z;
    const uint64_t l = far ? hi >> s : lo >> s | (hi << 1) << (63 - s), h = far ? 0 : hi >> s;
    w[i] = (bq_u32x4){(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
    if (none) w[i] = (bq_u32x4){0, 0, 0, 0};
  }
}

__device__ inline uint32_t pack_bf16(float a, float b) {  // round to nearest even
  const bq_f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bq_bf16x2));
}

__device__ inline void store8(uint16_t* row, int64_t cx, int64_t cols, bq_u32x4 w) {
  if (cx + 8 <= cols) {
    __builtin_nontemporal_store(w, (bq_u32x4_a2*)(row + cx));
    return;
  }
  const int n = (int)(cols - cx);  // below 8, or none
  uint16_t* p = row + cx;
  if (n <= 0) return;
  if (n & 4) {
    *(bq_u32x2_a2*)p = (bq_u32x2){w.x, w.y};
    p += 4;
    w.x = w.z;
    w.y = w.w;
  }
  if (n & 2) {
    *(bq_u32_a2*)p = w.x;
    p += 2;
    w.x = w.y;
  }
  if (n & 1) *p = (uint16_t)w.x;
}
__device__ inline bq_u32x4 pack8(const float f[8]) {
  return (bq_u32x4){pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}

// bits of the largest |x| of a row's block from 16 lanes' 8 values each
__device__ inline uint32_t row_mag(const float f[8]) {
  const float m = nan_max(nan_max(nan_max(f[0], f[1]), nan_max(f[2], f[3])),
                          nan_max(nan_max(f[4], f[5]), nan_max(f[6], f[7])));
  return row16_max(__float_as_uint(m) & 0x7FFFFFFFu);
}
__device__ inline uint32_t row_mag(bq_u32x4 w) {
  const bq_u32x4 a = w & 0x7FFF7FFFu;
  const uint32_t m = pk_max(pk_max(a.x, a.y), pk_max(a.z, a.w));
  return row16_max(umax(m & 0xFFFFu, m >> 16)) << 16;
}
// one lane's 8 values of a row, 16 lanes to a block
struct Row8 {
  float f[8];
};
template <int FMT>
__device__ inline uint2 row_code(const Row8& v, float s) {
  return make_uint2(code4<FMT>(v.f[0], v.f[1], v.f[2], v.f[3], s), code4<FMT>(v.f[4], v.f[5], v.f[6], v.f[7], s));
}
template <int FMT>
__device__ inline uint2 row_code(bq_u32x4 w, float s) {
  return make_uint2(code4<FMT>(w.x, w.y, s), code4<FMT>(w.z, w.w, s));
}
template <int FMT>
__device__ inline Row8 clamp_row(Row8 v, bool odd) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v.f[k] = clamp_one<FMT>(v.f[k], odd);
  return v;
}
template <int FMT>
__device__ inline bq_u32x4 clamp_row(bq_u32x4 w, bool odd) {
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = clamp_pair<FMT>(w[k], odd);
  return w;
}
__device__ inline uint32_t row_mag(const Row8& v) { return row_mag(v.f); }

// codes and scale bytes of N rows; one branch for all of them, so that
// their reductions over lanes overlap
template <int FMT, int N, typename V>
__device__ inline void rows_codes(const V (&v)[N], uint2 (&q)[N], uint32_t (&byte)[N]) {
  uint32_t m[N], all = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m[i] = row_mag(v[i]);
    all = umax(all, m[i]);
    byte[i] = scale_byte<FMT>(m[i]);
    q[i] = row_code<FMT>(v[i], scale_value(byte[i]));
  }
  if (__builtin_expect(__any(all >= 0x7F800000u), 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      q[i] = row_code<FMT>(clamp_row<FMT>(v[i], m[i] >= 0x7F800000u), scale_value(byte[i]));
  }
}

// Stores of rows that may not exist: through a buffer resource that ends
// with the matrix's last row within the tile, so that a row past it is
// dropped without a branch.
__device__ inline __amdgpu_buffer_rsrc_t tile_rsrc(const BlockMat& o, int64_t r0, int rows) {
  const int64_t n = o.rows - r0 < rows ? o.rows - r0 : rows;
  return __builtin_amdgcn_make_buffer_rsrc(o.codes + r0 * o.pitch, (short)0, (int)(n * o.pitch), 0x00020000);
}
__device__ inline void put_codes(__amdgpu_buffer_rsrc_t r, uint2 q, int off) {
  __builtin_amdgcn_raw_buffer_store_b64((bq_u32x2){q.x, q.y}, r, off, 0, 0);
}
// a row's scale byte (column cx: any of the block's)
__device__ inline void put_byte(const BlockMat& o, int64_t row, int64_t cx, uint32_t byte) {
  if ((threadIdx.x & 15) == 0 && row < o.rows) o.scales[cx / kBlk * o.srows + scale_pos(row)] = (uint8_t)byte;
}

// codes of a row's 8 columns to 32 bits: code * scale, exactly
template <int FMT>
__device__ inline void uncode8(uint2 q, float s, float f[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w = k ? q.y : q.x;
    bq_f32x2 lo, hi;
    if constexpr (FMT == FP8_E4M3) {
      lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true);
    } else {
      lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, s, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, s, true);
    }
    f[4 * k] = lo.x;
    f[4 * k + 1] = lo.y;
    f[4 * k + 2] = hi.x;
    f[4 * k + 3] = hi.y;
  }
}
// the same rounded to bf16 (exact but for values below its normal range)
template <int FMT>
__device__ inline bq_u32x4 uncode8_bf16(uint2 q, float s) {
  bq_u32x4 r;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w = k ? q.y : q.x;
    if constexpr (FMT == FP8_E4M3) {
      r[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
      r[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true));
    } else {
      r[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, false));
      r[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, true));
    }
  }
  return r;
}

__device__ inline uint2 row_codes_at(const BlockMat& q, int64_t row, int64_t cx) {
  return *(const uint2*)(q.codes + row * q.pitch + cx);
}
__device__ inline float row_scale_at(const BlockMat& q, int64_t row, int64_t cx) {
  return scale_value(q.scales[cx / kBlk * q.srows + scale_pos(row)]);
}

// ---- the transposing part ------------------------------------------------
// A 128 x 128 tile's codes in LDS, 128 bytes a column of the source. A write
// is a few rows of columns 8 cc + j for 16 cc, a read whole columns: odd
// groups of 8 columns swap the two halves of each 256-byte bank line, and
// 16-byte chunks are swizzled by pairs of groups, so that neither conflicts.
__device__ inline int lds_chunk(int c, int chunk) { return (c ^ ((c >> 3) & 1)) * 8 + (chunk ^ ((c >> 4) & 7)); }

// the tile to memory: row trow0 + c of o gets LDS column c, c < cols
template <int THREADS>
__device__ inline void put_tile(const uint4* tile, const BlockMat& o, int64_t trow0, int64_t cols, int64_t r0) {
  const int n = (int)(cols < kBlk ? cols : kBlk);
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc(o.codes + trow0 * o.pitch + r0, (short)0, (int)(n * o.pitch - r0), 0x00020000);
#pragma unroll
  for (int k = 0; k < 1024 / THREADS; ++k) {
    const int q = threadIdx.x + THREADS * k;
    const int c = q >> 3, part = q & 7;
    const uint4 v = tile[lds_chunk(c, part)];
    __builtin_amdgcn_raw_buffer_store_b128((bq_u32x4){v.x, v.y, v.z, v.w}, r, c * (int)o.pitch + 16 * part, 0, 0);
  }
}

// Two values' maxima over pairs of lanes 32 (16) apart at once: the result
// holds a's in the lower half (even rows of 16) and b's in the upper (odd).
template <typename Max>
__device__ inline uint32_t swap32_max(uint32_t a, uint32_t b, Max mx) {
  const bq_u32x2 r = __builtin_bit_cast(bq_u32x2, __builtin_amdgcn_permlane32_swap(a, b, false, false));
  return mx(r.x, r.y);
}
template <typename Max>
__device__ inline uint32_t swap16_max(uint32_t a, uint32_t b, Max mx) {
  const bq_u32x2 r = __builtin_bit_cast(bq_u32x2, __builtin_amdgcn_permlane16_swap(a, b, false, false));
  return mx(r.x, r.y);
}

}  // namespace fp8lin
