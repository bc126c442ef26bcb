// The linear on a stored 4-bit weight, of few rows: Y [M, N] = X [M, K] W.
// Bound by the one read of W, which wants every CU's loads in flight:
//   - a workgroup makes 16 NB columns of Y; its waves share out the blocks of
//     128 of K and add their FP32 sums over LDS in wave order (the same bits
//     always);
//   - a wave loads its share of W to registers, U blocks at a time: a lane's
//     16 bytes are 32 elements of one column;
//   - both operands become bf16, exactly (4-bit and 8-bit values times powers
//     of two), two elements an instruction, the group's scale with them, and
//     are multiplied by 16x16x32 bf16 products. The 8-bit instructions would
//     take the codes as they are, but drop bits below 2^-13 of a product's
//     neighbours, which a later 8-bit rounding (of a key, of the next
//     linear's input) turns into whole steps: a layer's output was 0.0028
//     off where its own rounding is 0.0017;
//   - of one or a few rows (FUSED) every workgroup quantises X itself, into
//     LDS while its first loads of W fly: one launch, no workspace.
#include <type_traits>

#include "fp4.h"

namespace fp8lin {
namespace {

typedef __bf16 f4_bf16x8 __attribute__((ext_vector_type(8)));

template <int N, int I = 0, typename F>
__device__ inline void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}
// a barrier that orders LDS only: global loads stay in flight
__device__ inline void lds_barrier() {
  __builtin_amdgcn_s_waitcnt((63 & 15) | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 8 elements (a word of codes) to bf16
__device__ inline f4_bf16x8 widen4(uint32_t w, float s) {
  const bq_u32x4 r = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
  return __builtin_bit_cast(f4_bf16x8, r);
}
__device__ inline f4_bf16x8 widen8(uint32_t a, uint32_t b, float s) {
  return __builtin_bit_cast(f4_bf16x8, uncode8_bf16<FP8_E4M3>(make_uint2(a, b), s));
}

__device__ inline int64_t w_at(const Fp4Mat& w, int64_t n, int G) {
  return (n >> 4) * fp4_kblocks(w.K) * 1024 + 256 * G + 16 * (n & 15);
}

// 64 KB of LDS hold the sums of 8 waves, of up to 8 tiles each
constexpr int kept_waves(int tiles, int waves) { return tiles * waves > 64 ? waves / 2 : waves; }

// MF: 16-row fragments of X. FUSED: X comes as bf16 x; otherwise quantised, as xq.
template <bool FUSED, int MF, int NB, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void fp4_few_kernel(Bf16Mat x, Fp4X xq, Fp4Mat w, uint16_t* __restrict__ y, int cols) {
  // partial sums; FUSED: before them X's values in bf16, rows of `pitch` bytes
  extern __shared__ uint4 lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, G = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * cols;
  const int64_t n1 = n0 + cols < w.N ? n0 + cols : w.N;
  const int nk = (int)fp4_xblocks(w.K);
  const int k0 = wave * nk / WAVES, k1 = (wave + 1) * nk / WAVES;
  const int rows = (int)(FUSED ? x.rows : xq.M);
  const int pitch = nk * 256 + 16;
  const uint8_t* wrow[NB];
  const uint8_t* wscale[NB];
  bool have[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t n = n0 + 16 * b + r16;
    have[b] = n < n1;
    wrow[b] = w.codes + w_at(w, n, G);
    wscale[b] = w.scales + (n >> 4) * (fp4_kblocks(w.K) / 4) * 256 + 64 * G + 4 * (n & 15);
  }
  bq_u32x4 wc[U][NB];
  uint32_t ws[U][NB];
  bq_f32x4 acc[MF][NB];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[f][b] = (bq_f32x4){0, 0, 0, 0};
  auto load_w = [&](int kb, int u) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      wc[u][b] = (bq_u32x4){0, 0, 0, 0};
      ws[u][b] = 127;
      if (have[b]) {
        wc[u][b] = __builtin_nontemporal_load((const bq_u32x4*)(wrow[b] + (int64_t)kb * 1024));
        ws[u][b] = wscale[b][(int64_t)(kb >> 2) * 256 + (kb & 3)];
      }
    }
  };
  uint8_t* const l8 = (uint8_t*)lds;
  if constexpr (FUSED) {
    // 16 lanes a block of 128, four turns of 4 WAVES blocks at a time; the
    // first loads are issued before those of W
    const int blocks = rows * nk, c8 = 8 * (int)(threadIdx.x & 15);
    constexpr int kTurn = 4 * WAVES;
    const bool whole = x.cols % kBlk == 0;
    bq_u32x4 v[4];
    const int at0 = threadIdx.x >> 4;
    for (int at = at0; at - at0 < blocks; at += 4 * kTurn) {
      static_for<4>([&](auto I_) {
        constexpr int i = decltype(I_)::value;
        v[i] = (bq_u32x4){0, 0, 0, 0};
        if (at + kTurn * i < blocks) {
          const int r = (at + kTurn * i) / nk, c = (at + kTurn * i - r * nk) * kBlk;
          bq_u32x4 e[1];
          load_rows<1, 1, false>(x, r, c + c8, whole, e);
          v[i] = e[0];
        }
      });
      if (at == at0)
        static_for<U>([&](auto U_) {
          if (k0 + decltype(U_)::value < k1) load_w(k0 + decltype(U_)::value, decltype(U_)::value);
        });
      uint2 q[4];
      uint32_t byte[4];
      rows_codes<FP8_E4M3>(v, q, byte);
      static_for<4>([&](auto I_) {
        constexpr int i = decltype(I_)::value;
        const int b = at + kTurn * i;
        if (b < blocks) {
          const int r = b / nk;
          *(bq_u32x4*)(l8 + r * pitch + (b - r * nk) * 256 + 2 * c8) = uncode8_bf16<FP8_E4M3>(q[i], scale_value(byte[i]));
        }
      });
    }
    lds_barrier();
  }
  // this lane's 32 elements 32 G .. of a row's block: the second half of a
  // piece's lanes hold them in two rows of 16 bytes
  const int64_t xb = fp4_xblocks(w.K);
  const uint8_t* xc = FUSED ? nullptr : xq.codes + (G >> 1) * 1024 + (32 * (G & 1) + r16) * 16;
  const uint8_t* xs = FUSED ? nullptr : xq.scales + 4 * r16;
  for (int kb = k0; kb < k1; kb += U) {
    static_for<U>([&](auto U_) {
      constexpr int u = decltype(U_)::value;
      if (kb + u < k1 && (!FUSED || kb != k0)) load_w(kb + u, u);
    });
    static_for<U>([&](auto U_) {
      constexpr int u = decltype(U_)::value;
      if (kb + u < k1) {
        f4_bf16x8 wf[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) wf[b][j] = widen4(wc[u][b][j], __uint_as_float(ws[u][b] == 255u ? 0x7FC00000u : ws[u][b] << 23));
        static_for<MF>([&](auto F_) {
          constexpr int f = decltype(F_)::value;
          f4_bf16x8 xf[4];
          if constexpr (FUSED) {
            bq_u32x4 e[4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
            if (r16 < rows) {
              const uint8_t* p = l8 + r16 * pitch + (kb + u) * 256 + 64 * G;
#pragma unroll
              for (int j = 0; j < 4; ++j) e[j] = *(const bq_u32x4*)(p + 16 * j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[j] = __builtin_bit_cast(f4_bf16x8, e[j]);
          } else {
            bq_u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
            uint32_t sx = 127;
            if (16 * f + r16 < rows) {
              const uint8_t* p = xc + (f * xb + kb + u) * 2048;
              lo = *(const bq_u32x4*)p;
              hi = *(const bq_u32x4*)(p + 256);
              sx = xs[(f * ((xb + 3) / 4) + ((kb + u) >> 2)) * 64 + ((kb + u) & 3)];
            }
            const float s = scale_value(sx);
            xf[0] = widen8(lo.x, lo.y, s);
            xf[1] = widen8(lo.z, lo.w, s);
            xf[2] = widen8(hi.x, hi.y, s);
            xf[3] = widen8(hi.z, hi.w, s);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[f][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[b][j], xf[j], acc[f][b], 0, 0, 0);
        });
      }
    });
  }
  if constexpr (FUSED) lds_barrier();  // X's values are read
  bq_f32x4* const part = (bq_f32x4*)lds;
  constexpr int S = kept_waves(MF * NB, WAVES);  // waves whose sums LDS holds at once
  if constexpr (S < WAVES) {
    // the upper half's sums first, into the lower half's
    if (wave >= S) {
#pragma unroll
      for (int f = 0; f < MF; ++f)
#pragma unroll
        for (int b = 0; b < NB; ++b) part[((wave - S) * MF * NB + f * NB + b) * 64 + lane] = acc[f][b];
    }
    lds_barrier();
    if (wave < S) {
#pragma unroll
      for (int f = 0; f < MF; ++f)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[f][b] += part[(wave * MF * NB + f * NB + b) * 64 + lane];
    }
    lds_barrier();
  }
  if (wave < S) {
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int b = 0; b < NB; ++b) part[(wave * MF * NB + f * NB + b) * 64 + lane] = acc[f][b];
  }
  lds_barrier();
  for (int i = wave; i < MF * NB; i += WAVES) {
    const int row = 16 * (i / NB) + r16;
    bq_f32x4 s = part[i * 64 + lane];
#pragma unroll
    for (int k = 1; k < S; ++k) s += part[(k * MF * NB + i) * 64 + lane];
    // this lane: columns 4 G .. 4 G + 3 of column block i % NB
    const int64_t n = n0 + 16 * (i % NB) + 4 * G;
    if (row >= rows) continue;
    uint16_t* d = y + row * w.N + n;
    const bq_u32x2 v = {pack_bf16(s.x, s.y), pack_bf16(s.z, s.w)};
    if (n + 4 <= n1) *(bq_u32x2_a2*)d = v;
    else
      for (int k = 0; k < 4 && n + k < n1; ++k) d[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
  }
}

template <bool FUSED, int MF, int NB, int U>
hipError_t run(const Bf16Mat& x, const Fp4X& xq, const Fp4Mat& w, uint16_t* y, int cols, hipStream_t st) {
  constexpr int kWaves = 8;
  size_t lds = 1024 * kept_waves(MF * NB, kWaves) * MF * NB;
  if (FUSED) {
    const size_t values = (size_t)x.rows * (fp4_xblocks(w.K) * 256 + 16);
    if (values > lds) lds = values;
  }
  fp4_few_kernel<FUSED, MF, NB, kWaves, U>
      <<<dim3((unsigned)((w.N + cols - 1) / cols)), 64 * kWaves, lds, st>>>(x, xq, w, y, cols);
  return hipGetLastError();
}

// Columns of Y a workgroup makes: all 256 CUs get one workgroup (or C) of
// equal work, since a CU streams from HBM at no more than its share, 20 GB/s.
// At most `most`, what the accumulators of a wave are laid out for.
inline int part_cols(int64_t N, int most) {
  const int64_t c = (N + 256 * most - 1) / (256 * most);
  return (int)((N + 256 * c - 1) / (256 * c));
}

// Of more rows: a workgroup's tile is 16 MF rows by 64 NB columns. Four waves
// have 16 NB columns each, whose codes go from memory to registers in the
// instruction's order; X's tile goes over LDS, a block of 128 of K at a time
// in turn with the one before. The scaled instruction takes 4-bit and 8-bit
// codes as they are. KG groups of four waves take every KG-th block of K each
// and add their sums at the end: where a CU has no other workgroup, its SIMDs
// then have two waves (222 rows by 7040 x 1664, 104 workgroups: 19.1 us with
// one group, 14.0 with two; 512 by 12288 x 16384, 512 of them: 96 and 113).
//
// EXACT: bf16 products instead, of both codes widened in registers, at half
// the rate (333 rows by 5120 x 15360: 57 us, 34 of the codes): for a Y that is
// rounded to 8 bits next. A lane then has elements
// 32 G ..+31 of X too (of the 8-bit instruction 16 G ..+15 of both halves).
typedef int f4_v8i __attribute__((ext_vector_type(8)));

template <int MF, int NB, int KG, bool EXACT>
__global__ __launch_bounds__(256 * KG, EXACT ? 2 : 1) void fp4_many_kernel(Fp4X x, Fp4Mat w, uint16_t* __restrict__ y, int tiles_n) {
  constexpr int kPieces = 2 * MF, kTurns = (kPieces + 3) / 4;  // of 1024 bytes; each wave's
  __shared__ bq_u32x4 xl[KG][2][kPieces][64];
  const int lane = threadIdx.x & 63;
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = all & 3, kg = all >> 2;
  const int r16 = lane & 15, G = lane >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * MF;  // in 16 rows
  const int64_t p0 = ((int64_t)(blockIdx.x % tiles_n) * 4 + wave) * NB;
  const int64_t panels = (w.N + 15) / 16, mtiles = (x.M + 15) / 16;
  const int nk = (int)fp4_xblocks(x.K);
  const int64_t kb4 = fp4_kblocks(w.K), xk4 = (nk + 3) / 4;
  const uint8_t *wc[NB], *ws[NB], *xs[MF], *xc[kTurns];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t p = p0 + b < panels ? p0 + b : panels - 1;  // a column past the last is computed and not stored
    wc[b] = w.codes + p * kb4 * 1024 + 16 * lane;
    ws[b] = w.scales + p * (kb4 / 4) * 256 + 4 * lane;
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int64_t m = m0 + f < mtiles ? m0 + f : mtiles - 1;
    xs[f] = x.scales + m * xk4 * 64 + 4 * r16;
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int c = wave + 4 * i < kPieces ? wave + 4 * i : kPieces - 1;
    const int64_t m = m0 + c / 2 < mtiles ? m0 + c / 2 : mtiles - 1;
    xc[i] = x.codes + m * nk * 2048 + (c & 1) * 1024 + 16 * lane;
  }
  bq_f32x4 acc[MF][NB];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[f][b] = (bq_f32x4){0, 0, 0, 0};
  // step n of this group is block n KG + kg of K; loads past the last repeat it
  bq_u32x4 xv[2][kTurns], wv[4][NB];
  uint32_t wsv[NB], xsv[MF], wsn[NB], xsn[MF];  // scales of four blocks of K, and of the next four
  const auto load_x = [&](int n, bq_u32x4 (&v)[kTurns]) {
    const int k = n * KG + kg < nk ? n * KG + kg : nk - 1;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) v[i] = *(const bq_u32x4*)(xc[i] + (int64_t)k * 2048);
  };
  const auto store_x = [&](int buf, const bq_u32x4 (&v)[kTurns]) {
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
      if (wave + 4 * i < kPieces) xl[kg][buf][wave + 4 * i][lane] = v[i];
  };
  const auto load_w = [&](int n, bq_u32x4 (&v)[NB]) {
    const int k = n * KG + kg < nk ? n * KG + kg : nk - 1;
#pragma unroll
    for (int b = 0; b < NB; ++b) v[b] = *(const bq_u32x4*)(wc[b] + (int64_t)k * 1024);
  };
  const auto load_scales = [&](int k4) {
    const int64_t at = k4 < xk4 ? k4 : xk4 - 1;
#pragma unroll
    for (int b = 0; b < NB; ++b) wsn[b] = *(const uint32_t*)(ws[b] + at * 256);
#pragma unroll
    for (int f = 0; f < MF; ++f) xsn[f] = *(const uint32_t*)(xs[f] + at * 64);
  };
  load_scales(0);
  load_x(0, xv[0]);
  load_w(0, wv[0]);
  load_x(1, xv[1]);
  load_w(1, wv[1]);
  load_w(2, wv[2]);
  store_x(0, xv[0]);
  load_x(2, xv[0]);
  lds_barrier();
  const int steps = (nk + KG - 1) / KG;
  for (int n4 = 0; n4 < steps; n4 += 4) {
    static_for<4>([&](auto I_) {
      constexpr int i = decltype(I_)::value;
      const int n = n4 + i, kb = n * KG + kg;
      if (n < steps) {
        if constexpr (i * KG % 4 == 0) {
          // this group's first block lowest
#pragma unroll
          for (int b = 0; b < NB; ++b) wsv[b] = wsn[b] >> (8 * kg);
#pragma unroll
          for (int f = 0; f < MF; ++f) xsv[f] = xsn[f] >> (8 * kg);
          load_scales(kb / 4 + 1);
        }
        constexpr int sel = i * KG % 4;
        f4_bf16x8 wf[EXACT ? NB : 1][4];
        if constexpr (EXACT) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t s = wsv[b] >> (8 * sel) & 0xFFu;
#pragma unroll
            for (int j = 0; j < 4; ++j) wf[b][j] = widen4(wv[i][b][j], s == 255u ? __uint_as_float(0x7FC00000u) : scale_value(s));
          }
        }
        load_w(n + 3, wv[(i + 3) & 3]);
        if (kb < nk) {
          // a fragment is read while the one before is multiplied
          constexpr int second = EXACT ? 16 : 64;
          const bq_u32x4* const tile = &xl[kg][i & 1][0][0] + (EXACT ? 64 * (G >> 1) + 32 * (G & 1) + r16 : lane);
          bq_u32x4 p[2], q[2];
          p[0] = tile[0];
          q[0] = tile[second];
          static_for<MF>([&](auto F_) {
            constexpr int f = decltype(F_)::value, at = f & 1;
            if constexpr (f + 1 < MF) {
              p[at ^ 1] = tile[128 * (f + 1)];
              q[at ^ 1] = tile[128 * (f + 1) + second];
            }
            if constexpr (EXACT) {
              const float s = scale_value(xsv[f] >> (8 * sel) & 0xFFu);
              const f4_bf16x8 xf[4] = {widen8(p[at].x, p[at].y, s), widen8(p[at].z, p[at].w, s), widen8(q[at].x, q[at].y, s),
                                       widen8(q[at].z, q[at].w, s)};
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[f][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[b][j], xf[j], acc[f][b], 0, 0, 0);
              __builtin_amdgcn_sched_barrier(0);
              return;
            }
            const f4_v8i e = {(int)p[at].x, (int)p[at].y, (int)p[at].z, (int)p[at].w,
                              (int)q[at].x, (int)q[at].y, (int)q[at].z, (int)q[at].w};
            static_for<NB>([&](auto B_) {
              constexpr int b = decltype(B_)::value;
              const bq_u32x4 c = wv[i][b];
              const f4_v8i a = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
              acc[f][b] =
                  __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, e, acc[f][b], 4, 0, sel, (int)wsv[b], sel, (int)xsv[f]);
            });
            __builtin_amdgcn_sched_barrier(0);
          });
        }
        store_x((i + 1) & 1, xv[(i + 1) & 1]);
        load_x(n + 3, xv[(i + 1) & 1]);
        lds_barrier();
      }
    });
  }
  if constexpr (KG > 1) {
    // the second group's sums over LDS, as many fragments at a time as fit
    static_assert(KG == 2, "two groups are joined");
    constexpr int kAtOnce = KG * 2 * kPieces / (4 * NB) < MF ? KG * 2 * kPieces / (4 * NB) : MF;
    bq_f32x4* const part = (bq_f32x4*)&xl[0][0][0][0];
#pragma unroll
    for (int f0 = 0; f0 < MF; f0 += kAtOnce) {
      if (f0) lds_barrier();
      if (kg == 1) {
#pragma unroll
        for (int f = f0; f < MF && f < f0 + kAtOnce; ++f)
#pragma unroll
          for (int b = 0; b < NB; ++b) part[(((f - f0) * 4 + wave) * NB + b) * 64 + lane] = acc[f][b];
      }
      lds_barrier();
      if (kg == 0) {
#pragma unroll
        for (int f = f0; f < MF && f < f0 + kAtOnce; ++f)
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[f][b] += part[(((f - f0) * 4 + wave) * NB + b) * 64 + lane];
      }
    }
    if (kg) return;
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int64_t row = (m0 + f) * 16 + r16;
    if (row >= x.M) continue;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int64_t n = (p0 + b) * 16 + 4 * G;
      uint16_t* d = y + row * w.N + n;
      const bq_u32x2 v = {pack_bf16(acc[f][b].x, acc[f][b].y), pack_bf16(acc[f][b].z, acc[f][b].w)};
      if (n + 4 <= w.N) *(bq_u32x2_a2*)d = v;
      else
        for (int k = 0; k < 4 && n + k < w.N; ++k) d[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
    }
  }
}

// 16-row fragments of a tile, at most: exact ones hold W's block in bf16 too
constexpr int most_mf(int nb, bool exact) { return exact && nb == 3 ? 5 : 8; }

template <int MF, int NB, bool EXACT>
hipError_t run_many(const Fp4X& x, const Fp4Mat& w, const Fp4Form& f, uint16_t* y, hipStream_t st) {
  const int64_t tm = ((x.M + 15) / 16 + MF - 1) / MF, tn = (w.N + 64 * NB - 1) / (64 * NB);
  if (NB == 1 || f.groups == 2) fp4_many_kernel<MF, NB, 2, EXACT><<<(unsigned)(tm * tn), 512, 0, st>>>(x, w, y, (int)tn);
  else if constexpr (NB > 1) fp4_many_kernel<MF, NB, 1, EXACT><<<(unsigned)(tm * tn), 256, 0, st>>>(x, w, y, (int)tn);
  return hipGetLastError();
}
template <int MF, bool EXACT>
hipError_t run_rows(const Fp4X& x, const Fp4Mat& w, const Fp4Form& f, uint16_t* y, hipStream_t st) {
  if constexpr (MF < 8)
    if (f.nb == 1) return run_many<MF, 1, EXACT>(x, w, f, y, st);
  if constexpr (MF <= most_mf(3, EXACT))
    if (f.nb == 3) return run_many<MF, 3, EXACT>(x, w, f, y, st);
  return run_many<MF, 2, EXACT>(x, w, f, y, st);
}
template <bool EXACT>
hipError_t run_tiles(const Fp4X& x, const Fp4Mat& w, const Fp4Form& f, uint16_t* y, hipStream_t st) {
  switch (f.mf) {
    case 4: return run_rows<4, EXACT>(x, w, f, y, st);
    case 5: return run_rows<5, EXACT>(x, w, f, y, st);
    case 6: return run_rows<6, EXACT>(x, w, f, y, st);
    case 7: return run_rows<7, EXACT>(x, w, f, y, st);
    default: return run_rows<8, EXACT>(x, w, f, y, st);
  }
}

__global__ __launch_bounds__(256) void fp4_zero_kernel(uint16_t* __restrict__ y, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) y[i] = 0;
}

}  // namespace

hipError_t launch_fp4_zero(uint16_t* y, int64_t n, hipStream_t st) {
  if (n == 0) return hipSuccess;
  fp4_zero_kernel<<<(unsigned)(n < 2048 * 256 ? (n + 255) / 256 : 2048), 256, 0, st>>>(y, n);
  return hipGetLastError();
}

// X's values in bf16 fit 64 KB of LDS
bool fp4_fused(int64_t M, int64_t K) { return M <= 16 && M * fp4_xblocks(K) <= 248; }

Fp4Form fp4_form(int64_t M, int64_t K, int64_t N, bool exact) {
  Fp4Form f = {fp4_fused(M, K) ? FP4_FUSED : M <= (exact ? kFp4FewExact : kFp4Few) ? FP4_FEW : exact ? FP4_EXACT : FP4_MANY,
               1, 1, 1, 0};
  if (f.kind == FP4_FUSED || f.kind == FP4_FEW) {
    f.mf = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    f.cols = part_cols(N, 48);
    f.nb = f.cols <= 16 ? 1 : f.cols <= 32 ? 2 : 3;
    return f;
  }
  // the tile whose rounds of 256 workgroups have the least products in all
  const int64_t mt = (M + 15) / 16, panels = (N + 15) / 16;
  int64_t least = 0;
  for (int mf = 4; mf <= 8; ++mf)
    for (int nb = mf == 8 ? 2 : 1; nb <= 3; ++nb) {  // 8 x 1 costs what 4 x 2 does
      if (mf > most_mf(nb, exact)) continue;
      const int64_t n = (mt + mf - 1) / mf * ((panels + 4 * nb - 1) / (4 * nb));
      // 4 + products: what a block of K costs a wave besides them
      if (nb == 1 && n > 256) continue;
      const int64_t cost = (n + 255) / 256 * (mf * nb + 4);
      if (least == 0 || cost < least) {
        least = cost;
        f.mf = mf;
        f.nb = nb;
        // two groups where a CU has one workgroup at most; else two workgroups share it
        f.groups = n <= 256 ? 2 : 1;
      }
    }
  return f;
}

hipError_t launch_fp4_fused(const Bf16Mat& x, const Fp4Mat& w, uint16_t* y, hipStream_t st) {
  if (x.rows == 0 || w.N == 0) return hipSuccess;
  const Fp4X none = {nullptr, nullptr, 0, 0};
  const Fp4Form f = fp4_form(x.rows, w.K, w.N, true);
  return f.nb == 1   ? run<true, 1, 1, 4>(x, none, w, y, f.cols, st)
         : f.nb == 2 ? run<true, 1, 2, 4>(x, none, w, y, f.cols, st)
                     : run<true, 1, 3, 4>(x, none, w, y, f.cols, st);
}

hipError_t launch_fp4_linear(const Fp4X& x, const Fp4Mat& w, uint16_t* y, bool exact, hipStream_t st) {
  if (x.M == 0 || w.N == 0) return hipSuccess;
  const Fp4Form f = fp4_form(x.M, w.K, w.N, exact);
  if (f.kind == FP4_FEW) {
    const Bf16Mat none = {nullptr, 0, 0, 0};
#define FEW(m, n) \
  if (f.mf == m && f.nb == n) return run<false, m, n, (m > 2 ? 2 : 4)>(none, x, w, y, f.cols, st);
    FEW(1, 1) FEW(1, 2) FEW(1, 3) FEW(2, 1) FEW(2, 2) FEW(2, 3) FEW(4, 1) FEW(4, 2) FEW(4, 3)
#undef FEW
  }
  return exact ? run_tiles<true>(x, w, f, y, st) : run_tiles<false>(x, w, f, y, st);
}

}  // namespace fp8lin
