// Device pieces shared by the block-scaled quantise and SwiGLU kernels.
//
// A 256-thread block holds a 128 x 128 tile as 8 x 8 patches in 32 bits:
// thread t has rows 8 (t / 16) .. + 7, columns 8 (t % 16) .. + 7. A row's
// block of 128 then lies in 16 neighbouring lanes, a column's in 16 lane
// groups of all four waves.
#pragma once

#include "block.h"

namespace fp8lin {

typedef unsigned int bq_u32x4 __attribute__((ext_vector_type(4)));
typedef bq_u32x4 bq_u32x4_a2 __attribute__((aligned(2)));  // a row of an odd pitch starts at any 2 bytes
typedef float bq_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bq_bf16x2 __attribute__((ext_vector_type(2)));

__device__ inline uint32_t mag_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }
__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// max over the 16 lanes that share t / 16 (one DPP row)
__device__ inline uint32_t row16_max(uint32_t m) {
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));   // lanes ^ 1
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));   // lanes ^ 2
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, true));  // half-row mirror
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, true));  // row mirror
  return m;
}

// four values at a scale to four codes; `odd`: the block holds an infinity
// or a NaN (its scale is then 1), so values are clamped; a NaN stays one.
// Elsewhere the scale keeps every value within the format's largest.
template <int FMT>
__device__ inline uint32_t code4(float f0, float f1, float f2, float f3, float scale, bool odd) {
  f0 *= scale;
  f1 *= scale;
  f2 *= scale;
  f3 *= scale;
  if (odd) {
    constexpr float kMax = FMT == FP8_E4M3 ? 448.0f : 57344.0f;
    f0 = f0 != f0 ? f0 : fminf(fmaxf(f0, -kMax), kMax);
    f1 = f1 != f1 ? f1 : fminf(fmaxf(f1, -kMax), kMax);
    f2 = f2 != f2 ? f2 : fminf(fmaxf(f2, -kMax), kMax);
    f3 = f3 != f3 ? f3 : fminf(fmaxf(f3, -kMax), kMax);
  }
  int r;
  if constexpr (FMT == FP8_E4M3) {
    r = __builtin_amdgcn_cvt_pk_fp8_f32(f0, f1, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(f2, f3, r, true);
  } else {
    r = __builtin_amdgcn_cvt_pk_bf8_f32(f0, f1, 0, false);
    r = __builtin_amdgcn_cvt_pk_bf8_f32(f2, f3, r, true);
  }
  return (uint32_t)r;
}

// 8 bf16 (four dwords) to 32 bits
__device__ inline void widen8(bq_u32x4 w, float f[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// columns cx .. cx + 7 of a row, zeros past cols; in-bounds for any pitch
__device__ inline bq_u32x4 load8(const uint16_t* row, int64_t cx, int64_t cols) {
  if (cx + 8 <= cols) return __builtin_nontemporal_load((const bq_u32x4_a2*)(row + cx));
  bq_u32x4 w = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (cx + k < cols) w[k >> 1] |= (uint32_t)row[cx + k] << (16 * (k & 1));
  return w;
}

__device__ inline uint32_t pack_bf16(float a, float b) {  // round to nearest even
  const bq_f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bq_bf16x2));
}

__device__ inline void store8(uint16_t* row, int64_t cx, int64_t cols, const float f[8]) {
  const bq_u32x4 w = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  if (cx + 8 <= cols) {
    __builtin_nontemporal_store(w, (bq_u32x4_a2*)(row + cx));
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (cx + k < cols) row[cx + k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}

// one row's 8 values in each of 16 lanes -> codes and scale byte of that
// row's block (column cx = this lane's first; a whole block is written, so
// columns past cols hold zero codes). All 16 lanes call it.
template <int FMT>
__device__ inline void quant_row8(const float f[8], const BlockMat& o, int64_t row, int64_t cx) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = umax(m, mag_bits(f[k]));
  m = row16_max(m);
  const int32_t b = bias_from_amax_bits(m, FMT, 0, 0, nullptr);
  const float s = pow2f(b);
  const bool odd = m >= 0x7F800000u;
  const uint2 q = make_uint2(code4<FMT>(f[0], f[1], f[2], f[3], s, odd), code4<FMT>(f[4], f[5], f[6], f[7], s, odd));
  if (row < o.rows) {
    *(uint2*)(o.codes + row * o.pitch + cx) = q;
    if ((threadIdx.x & 15) == 0) o.scales[cx / kBlk * o.srows + scale_pos(row)] = (uint8_t)(127 - b);
  }
}

// codes of a row's 8 columns to 32 bits
template <int FMT>
__device__ inline void uncode8(uint2 q, float s, float f[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int w = (int)(k ? q.y : q.x);
    bq_f32x2 lo, hi;
    if constexpr (FMT == FP8_E4M3) {
      lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
      hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_f32_bf8(w, false);
      hi = __builtin_amdgcn_cvt_pk_f32_bf8(w, true);
    }
    f[4 * k] = lo.x * s;
    f[4 * k + 1] = lo.y * s;
    f[4 * k + 2] = hi.x * s;
    f[4 * k + 3] = hi.y * s;
  }
}

// 2^(byte - 127); bytes are 1 .. 253
__device__ inline float scale_value(uint8_t byte) { return __uint_as_float((uint32_t)byte << 23); }

template <int FMT>
__device__ inline void load_row8(const BlockMat& q, int64_t row, int64_t cx, float f[8]) {
  const uint2 w = *(const uint2*)(q.codes + row * q.pitch + cx);
  uncode8<FMT>(w, scale_value(q.scales[cx / kBlk * q.srows + scale_pos(row)]), f);
}

// LDS of the transposing part: the tile's codes and the column maxima of each wave
struct QuantLds {
  uint4 tile[kBlk * kBlk / 16];
  uint32_t cmax[4][kBlk];
};

// A tile in patches -> the transposed form: row trow0 + c0 + j of o holds
// column c0 + j, its columns r0 .. r0 + 127 (o.rows: how many columns the
// source has from c0 = 0 on; rows past the source's are zeros in v). The
// whole workgroup calls it; a barrier at entry lets it follow itself.
template <int FMT>
__device__ inline void quant_cols(const float v[8][8], const BlockMat& o, int64_t trow0, int64_t r0, int64_t c0,
                                  QuantLds& lds) {
  const int t = threadIdx.x, rg = t >> 4, cc = t & 15;
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m[j] = umax(m[j], mag_bits(v[i][j]));
    m[j] = umax(m[j], (uint32_t)__shfl_xor((int)m[j], 16, 64));
    m[j] = umax(m[j], (uint32_t)__shfl_xor((int)m[j], 32, 64));
  }
  __syncthreads();  // the tile and maxima of an earlier call are read
  if ((t & 63) < 16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) lds.cmax[t >> 6][8 * cc + j] = m[j];
  }
  __syncthreads();
  uint8_t* const l8 = (uint8_t*)lds.tile;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = 8 * cc + j;
    const uint32_t mm = umax(umax(lds.cmax[0][c], lds.cmax[1][c]), umax(lds.cmax[2][c], lds.cmax[3][c]));
    const int32_t b = bias_from_amax_bits(mm, FMT, 0, 0, nullptr);
    const float s = pow2f(b);
    const bool odd = mm >= 0x7F800000u;
    // 16-byte chunks of an LDS row are swizzled by (row / 8), which spreads
    // the 8-byte writes over the banks
    *(uint2*)(l8 + c * kBlk + ((((rg >> 1) ^ (cc & 7))) << 4) + 8 * (rg & 1)) =
        make_uint2(code4<FMT>(v[0][j], v[1][j], v[2][j], v[3][j], s, odd),
                   code4<FMT>(v[4][j], v[5][j], v[6][j], v[7][j], s, odd));
    if (rg == 0 && c0 + c < o.rows)
      o.scales[r0 / kBlk * o.srows + scale_pos(trow0 + c0 + c)] = (uint8_t)(127 - b);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int q = t + 256 * k;
    const int c = q >> 3, part = q & 7;
    if (c0 + c < o.rows)
      *(uint4*)(o.codes + (trow0 + c0 + c) * o.pitch + r0 + 16 * part) = lds.tile[c * 8 + (part ^ ((c >> 3) & 7))];
  }
}

}  // namespace fp8lin
