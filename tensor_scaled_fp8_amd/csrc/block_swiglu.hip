// SwiGLU with 8-bit checkpoints. Forward, from the bf16 gate g and up u:
//   h = g s u,  s = 1 / (1 + exp(-g)),
// and the E4M3 block-scaled forms g', u' that the backward reads in place
// of g and u (half their bytes). Backward, at g', u':
//   dg = dh u' s' (1 + g' (1 - s')),  du = dh g' s',  h' = g' s' u'.
// Everything is computed in 32 bits and rounded once, to bf16 or to a
// block-scaled code. Bound by HBM: every input read once, every output
// written once, the maxima of a block taken in registers. 4096 x 28672:
// forward 147 us and backward 145, 6.4 TB/s; the gradients of 2048 x 10240
// straight to their stored forms 56 us, 3.4 TB/s (two waves a SIMD).
#include <type_traits>

#include "block_quant.h"

namespace fp8lin {
namespace {

// s = 1 / (1 + e^-g), as s r^2. The exponential's argument is rounded in 32
// bits, so s is off by about |g| 2^-23 relative, below the outputs' 8 bits
// wherever s is not 0. Far below 0 the plain expression leaves 32 bits (1 / e^-g
// is below 2^-126 from g = -87.4 on, e^-g above 2^128 from -88.8) where g s u is
// still an ordinary number for a large u: there (FAR) s is taken at -80 and
// the rest of e^g is the square of r, multiplied in last. Beyond g = -400 every
// finite product is 0; the bound on g keeps the products before r finite.
constexpr float kFar = -80.0f, kGone = -400.0f;
struct Sigmoid {
  float g, s, r;
};
template <bool FAR>
__device__ inline Sigmoid sigmoid(float g) {
  if constexpr (!FAR) return {g, __builtin_amdgcn_rcpf(1.0f + __expf(-g)), 1.0f};
  const float c = g < kGone && g > -__builtin_inff() ? kGone : g;
  return {c, __builtin_amdgcn_rcpf(1.0f + __expf(-fmaxf(c, kFar))),
          __builtin_amdgcn_exp2f(fminf(c - kFar, 0.0f) * 0.72134752f)};  // log2(e) / 2
}
// f(far) for a row's 8 gates of each lane: far is whether any of the wave's is
// below kFar, which is rare, so that the usual case pays for one branch
template <typename F>
__device__ inline void near_or_far(const float g[8], F&& f) {
  const float lo = fminf(fminf(fminf(g[0], g[1]), fminf(g[2], g[3])), fminf(fminf(g[4], g[5]), fminf(g[6], g[7])));
  if (__builtin_expect(__any(lo < kFar), 0)) f(std::true_type{});
  else f(std::false_type{});
}

template <bool FAR>
__device__ inline float gated(float g, float u) {
  const Sigmoid q = sigmoid<FAR>(g);
  const float h = q.g * q.s * u;
  return FAR ? h * q.r * q.r : h;
}
struct Grads {
  float dg, du, h;
};
template <bool FAR>
__device__ inline Grads grads(float g, float u, float dh) {
  const Sigmoid q = sigmoid<FAR>(g);
  const float gs = q.g * q.s;
  Grads x = {dh * u * __builtin_fmaf(gs, 1.0f - q.s, q.s), dh * gs, gs * u};
  if constexpr (FAR) x = {x.dg * q.r * q.r, x.du * q.r * q.r, x.h * q.r * q.r};
  return x;
}

template <int RPT>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(Bf16Mat gate, Bf16Mat up, uint16_t* __restrict__ h, int64_t ldh,
                                                         BlockMat hq, BlockMat gq, BlockMat uq, int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
  bq_u32x4 wg[RPT], wu[RPT];
  const bool inside = r0 + 16 * RPT <= gate.rows && c0 + kBlk <= gate.cols;
  load_rows<RPT, 16>(gate, rr, cx, inside, wg);
  load_rows<RPT, 16>(up, rr, cx, inside, wu);
  Row8 y[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    float g[8], u[8];
    widen8(wg[i], g);
    widen8(wu[i], u);
    near_or_far(g, [&](auto far) {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[i].f[k] = gated<decltype(far)::value>(g[k], u[k]);
    });
    if (h && rr + 16 * i < gate.rows) store8(h + (rr + 16 * i) * ldh, cx, gate.cols, pack8(y[i].f));
  }
  auto put = [&](const BlockMat& o, const auto& v) {
    uint2 q[RPT];
    uint32_t byte[RPT];
    rows_codes<FP8_E4M3>(v, q, byte);
    const __amdgpu_buffer_rsrc_t r = tile_rsrc(o, r0, 16 * RPT);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      put_codes(r, q[i], ((t >> 4) + 16 * i) * (int)o.pitch + (int)cx);
      put_byte(o, rr + 16 * i, cx, byte[i]);
    }
  };
  if (hq.codes) put(hq, y);
  if (gq.codes) {
    put(gq, wg);
    put(uq, wu);
  }
}

template <int RPT>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(Bf16Mat dh, BlockMat gq, BlockMat uq,
                                                         uint16_t* __restrict__ dg, int64_t lddg,
                                                         uint16_t* __restrict__ du, int64_t lddu, int tiles_c) {
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * (16 * RPT), c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x;
  const int64_t rr = r0 + (t >> 4), cx = c0 + 8 * (t & 15);
  bq_u32x4 wd[RPT];
  uint2 wg[RPT], wu[RPT];
  float sg[RPT], su[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = rr + 16 * i;
    wg[i] = wu[i] = make_uint2(0, 0);
    sg[i] = su[i] = 1.0f;
    if (r < dh.rows) {
      wg[i] = row_codes_at(gq, r, cx);
      wu[i] = row_codes_at(uq, r, cx);
      sg[i] = row_scale_at(gq, r, cx);
      su[i] = row_scale_at(uq, r, cx);
    }
  }
  load_rows<RPT, 16>(dh, rr, cx, r0 + 16 * RPT <= dh.rows && c0 + kBlk <= dh.cols, wd);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t r = rr + 16 * i;
    if (r >= dh.rows) continue;
    float g[8], u[8], d[8], a[8], b[8];
    widen8(wd[i], d);
    uncode8<FP8_E4M3>(wg[i], sg[i], g);
    uncode8<FP8_E4M3>(wu[i], su[i], u);
    near_or_far(g, [&](auto far) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const Grads x = grads<decltype(far)::value>(g[k], u[k], d[k]);
        a[k] = x.dg;
        b[k] = x.du;
      }
    });
    if (dg) store8(dg + r * lddg, cx, dh.cols, pack8(a));
    if (du) store8(du + r * lddu, cx, dh.cols, pack8(b));
  }
}

// One 128 x 128 tile: the E5M2 row and transposed forms of dg and du and
// the E4M3 transposed form of h', all from one evaluation: a thread of 512
// holds the three at 4 rows x 8 columns in 32 bits (96 of 144 registers, two
// waves a SIMD; held to 128 registers it spilled, 57 -> 108 us) until the
// columns' maxima are known. dh.p null: h' only.
__device__ inline uint32_t bits_max(uint32_t a, uint32_t b) {
  return __float_as_uint(nan_max(__uint_as_float(a), __uint_as_float(b)));
}
__global__ __launch_bounds__(512) void swiglu_bwd_quant_kernel(Bf16Mat dh, BlockMat gq, BlockMat uq, BlockMat dgq,
                                                                  BlockMat duq, BlockMat dgut, BlockMat ht,
                                                                  int tiles_c) {
  __shared__ uint4 tile[3][kBlk * kBlk / 16];  // h', dg, du
  __shared__ float cmax[3][8][kBlk];           // of each wave
  __shared__ float cscale[3][kBlk];
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * kBlk, c0 = (int64_t)(blockIdx.x % tiles_c) * kBlk;
  const int t = threadIdx.x, rg = t >> 4, cc = t & 15, wave = t >> 6;
  const int64_t rr = r0 + 4 * rg, cx = c0 + 8 * cc;
  const int64_t f = dh.cols;
  bq_u32x4 wd[4];
  uint2 wg[4], wu[4];
  float sg[4], su[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = rr + i;
    wd[i] = (bq_u32x4){0, 0, 0, 0};
    wg[i] = wu[i] = make_uint2(0, 0);
    sg[i] = su[i] = 1.0f;
    if (r < dh.rows) {
      wg[i] = row_codes_at(gq, r, cx);
      wu[i] = row_codes_at(uq, r, cx);
      sg[i] = row_scale_at(gq, r, cx);
      su[i] = row_scale_at(uq, r, cx);
    }
  }
  if (dh.p) load_rows<4, 1>(dh, rr, cx, r0 + kBlk <= dh.rows && c0 + kBlk <= f, wd);
  Row8 v[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float d[8], g[8], u[8];
    widen8(wd[i], d);
    uncode8<FP8_E4M3>(wg[i], sg[i], g);
    uncode8<FP8_E4M3>(wu[i], su[i], u);
    near_or_far(g, [&](auto far) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const Grads x = grads<decltype(far)::value>(g[k], u[k], d[k]);
        v[0][i].f[k] = x.h;
        v[1][i].f[k] = x.dg;
        v[2][i].f[k] = x.du;
      }
    });
  }
  if (dgq.codes) {
    auto put = [&](const BlockMat& o, const Row8 (&x)[4]) {
      uint2 q[4];
      uint32_t byte[4];
      rows_codes<FP8_E5M2>(x, q, byte);
      const __amdgpu_buffer_rsrc_t r = tile_rsrc(o, r0, kBlk);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        put_codes(r, q[i], (4 * rg + i) * (int)o.pitch + (int)cx);
        put_byte(o, rr + i, cx, byte[i]);
      }
    };
    put(dgq, v[1]);
    put(duq, v[2]);
  }
  if (!dgut.codes && !ht.codes) return;
  // columns 2 R, 2 R + 1 of the eight in the R-th 16 lanes
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      m[j] = __float_as_uint(nan_max(nan_max(v[a][0].f[j], v[a][1].f[j]), nan_max(v[a][2].f[j], v[a][3].f[j])));
    float2 q;
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = swap32_max(m[j], m[j + 4], bits_max);
    q.x = __uint_as_float(swap16_max(p[0], p[2], bits_max));
    q.y = __uint_as_float(swap16_max(p[1], p[3], bits_max));
    *(float2*)&cmax[a][wave][8 * cc + 2 * (rg & 3)] = q;
  }
  __syncthreads();
  if (t < 3 * kBlk) {
    const int a = t >> 7, c = t & 127;
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = nan_max(m, cmax[a][k][c]);
    const uint32_t mag = __float_as_uint(m) & 0x7FFFFFFFu;
    const uint32_t byte = a == 0 ? scale_byte<FP8_E4M3>(mag) : scale_byte<FP8_E5M2>(mag);
    cscale[a][c] = mag < 0x7F800000u ? scale_value(byte) : -1.0f;
    const BlockMat& o = a == 0 ? ht : dgut;
    // dg's rows of the transposed gradient are 0 .. f - 1, du's f .. 2 f - 1
    if (o.codes && c0 + c < f) o.scales[r0 / kBlk * o.srows + scale_pos((a == 2 ? f : 0) + c0 + c)] = (uint8_t)byte;
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    uint8_t* const l8 = (uint8_t*)tile[a];
    float s[8];  // negative: an infinity or a NaN in the column
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[j] = cscale[a][8 * cc + j];
      odd |= s[j] < 0;
    }
    odd = __builtin_expect(__any(odd), 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x[4] = {v[a][0].f[j], v[a][1].f[j], v[a][2].f[j], v[a][3].f[j]};
      if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = a == 0 ? clamp_one<FP8_E4M3>(x[i], s[j] < 0) : clamp_one<FP8_E5M2>(x[i], s[j] < 0);
        s[j] = __builtin_fabsf(s[j]);
      }
      const uint32_t q = a == 0 ? code4<FP8_E4M3>(x[0], x[1], x[2], x[3], s[j])
                                : code4<FP8_E5M2>(x[0], x[1], x[2], x[3], s[j]);
      *(uint32_t*)(l8 + 16 * lds_chunk(8 * cc + j, rg >> 2) + 4 * (rg & 3)) = q;
    }
  }
  __syncthreads();
  if (ht.codes) put_tile<512>(tile[0], ht, c0, f - c0, r0);
  if (dgut.codes) {
    put_tile<512>(tile[1], dgut, c0, f - c0, r0);
    put_tile<512>(tile[2], dgut, f + c0, f - c0, r0);
  }
}

inline bool few_rows(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 127) / 128) < 1024; }

}  // namespace

hipError_t launch_swiglu_fwd(const Bf16Mat& gate, const Bf16Mat& up, uint16_t* h, int64_t ldh, const BlockMat& hq,
                             const BlockMat& gq, const BlockMat& uq, hipStream_t st) {
  if (gate.rows == 0 || gate.cols == 0) return hipSuccess;
  const int64_t tc = (gate.cols + kBlk - 1) / kBlk;
  if (few_rows(gate.rows, gate.cols))
    swiglu_fwd_kernel<1><<<dim3((unsigned)((gate.rows + 15) / 16 * tc)), 256, 0, st>>>(gate, up, h, ldh, hq, gq, uq,
                                                                                      (int)tc);
  else
    swiglu_fwd_kernel<4><<<dim3((unsigned)((gate.rows + 63) / 64 * tc)), 256, 0, st>>>(gate, up, h, ldh, hq, gq, uq,
                                                                                      (int)tc);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const Bf16Mat& dh, const BlockMat& gq, const BlockMat& uq, uint16_t* dg, int64_t lddg,
                             uint16_t* du, int64_t lddu, hipStream_t st) {
  if (dh.rows == 0 || dh.cols == 0) return hipSuccess;
  const int64_t tc = (dh.cols + kBlk - 1) / kBlk;
  if (few_rows(dh.rows, dh.cols))
    swiglu_bwd_kernel<1><<<dim3((unsigned)((dh.rows + 15) / 16 * tc)), 256, 0, st>>>(dh, gq, uq, dg, lddg, du, lddu,
                                                                                    (int)tc);
  else
    swiglu_bwd_kernel<4><<<dim3((unsigned)((dh.rows + 63) / 64 * tc)), 256, 0, st>>>(dh, gq, uq, dg, lddg, du, lddu,
                                                                                    (int)tc);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd_quant(const Bf16Mat& dh, const BlockMat& gq, const BlockMat& uq, const BlockMat& dgq,
                                   const BlockMat& duq, const BlockMat& dgut, const BlockMat& ht, hipStream_t st) {
  if (dh.rows == 0 || dh.cols == 0) return hipSuccess;
  const int64_t tc = (dh.cols + kBlk - 1) / kBlk;
  swiglu_bwd_quant_kernel<<<dim3((unsigned)((dh.rows + kBlk - 1) / kBlk * tc)), 512, 0, st>>>(dh, gq, uq, dgq, duq,
                                                                                            dgut, ht, (int)tc);
  return hipGetLastError();
}

}  // namespace fp8lin
