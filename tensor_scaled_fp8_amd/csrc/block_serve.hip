// The serving linear for few rows: Y [M, N] = X [M, K] W, W stored (E4M3,
// transposed [N, K], a scale for each block of 128). Bound by the one read of
// W, which wants every CU's loads in flight and nothing else to wait for:
//   - a workgroup makes 16 NB columns of Y; its waves share out the k-blocks
//     and add their FP32 sums over LDS in wave order (the same bits always);
//   - a wave loads its share of W to registers, U k-blocks at a time, with no
//     staging in LDS: a lane's 32 bytes of a row are its MFMA operand. The
//     products of a k-block may be summed in any order, so lane l takes
//     columns 16 G .. and 64 + 16 G .. of the block (G = l / 16) of both
//     operands: 64 contiguous bytes of a row an instruction;
//   - of one or a few rows (FUSED) every workgroup quantises X itself, into
//     LDS while its first loads of W fly: one launch, no workspace. Of more,
//     that work, repeated by every workgroup, costs more than a launch, and X
//     comes quantised.
// One row by 4096 x 12288 (50 MB): 12.8 us, 3.9 TB/s with the launch; 13 rows
// by 8192 x 10240 (84 MB): 20.8 us, 4.0 TB/s.
#include <type_traits>

#include "block_quant.h"

namespace fp8lin {
namespace {

typedef int sv_v8i __attribute__((ext_vector_type(8)));

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

// MF: 16-row fragments of X. FUSED: X comes as bf16 x; otherwise stored, as xq.
template <bool FUSED, int MF, int NB, int WAVES, int U>
__global__ __launch_bounds__(64 * WAVES) void block_serve_kernel(Bf16Mat x, BlockMat xq, BlockMat w,
                                                                 uint16_t* __restrict__ y, int cols) {
  // partial sums; FUSED: before them X's codes [rows][pitch], then its scale bytes [rows][nk]
  extern __shared__ uint4 lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, G = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * cols;
  const int64_t n1 = n0 + cols < w.rows ? n0 + cols : w.rows;
  const int nk = (int)(w.pitch / kBlk);
  const int k0 = wave * nk / WAVES, k1 = (wave + 1) * nk / WAVES;
  const int rows = (int)(FUSED ? x.rows : xq.rows);
  const uint8_t* wrow[NB];
  const uint8_t* wscale[NB];
  bool have[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t n = n0 + 16 * b + r16;
    have[b] = n < n1;
    wrow[b] = w.codes + n * w.pitch + 16 * G;
    wscale[b] = w.scales + scale_pos(n);
  }
  bool mine[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) mine[f] = 16 * f + r16 < rows;

  bq_u32x4 wc[U][NB][2], xc[U][MF][2];
  uint32_t ws[U][NB], xs[U];
  bq_f32x4 acc[MF][NB];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[f][b] = (bq_f32x4){0, 0, 0, 0};
  auto load_w = [&](int kb, int u) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      wc[u][b][0] = wc[u][b][1] = (bq_u32x4){0, 0, 0, 0};
      ws[u][b] = 127;
      if (have[b]) {
        wc[u][b][0] = __builtin_nontemporal_load((const bq_u32x4*)(wrow[b] + (int64_t)kb * kBlk));
        wc[u][b][1] = __builtin_nontemporal_load((const bq_u32x4*)(wrow[b] + (int64_t)kb * kBlk + 64));
        ws[u][b] = wscale[b][kb * w.srows];
      }
    }
  };
  uint8_t* const l8 = (uint8_t*)lds;
  auto load_x = [&](int kb, int u) {
    if constexpr (FUSED) {
      xc[u][0][0] = xc[u][0][1] = (bq_u32x4){0, 0, 0, 0};
      xs[u] = 127;
      if (mine[0]) {
        const uint8_t* p = l8 + r16 * w.pitch + kb * kBlk + 16 * G;
        xc[u][0][0] = *(const bq_u32x4*)p;
        xc[u][0][1] = *(const bq_u32x4*)(p + 64);
        xs[u] = l8[rows * w.pitch + r16 * nk + kb];
      }
    } else {
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        xc[u][f][0] = xc[u][f][1] = (bq_u32x4){0, 0, 0, 0};
        if (mine[f]) {
          const uint8_t* p = xq.codes + (16 * f + r16) * xq.pitch + kb * kBlk + 16 * G;
          xc[u][f][0] = *(const bq_u32x4*)p;
          xc[u][f][1] = *(const bq_u32x4*)(p + 64);
        }
      }
      xs[u] = *(const uint32_t*)(xq.scales + kb * xq.srows + 8 * r16);  // of rows r16, 16 + r16, ..
    }
  };

  if constexpr (FUSED) {
    // 16 lanes a block of 128, four turns of 4 WAVES blocks at a time; the
    // first loads are issued before those of W
    const int blocks = rows * nk, c8 = 8 * (int)(threadIdx.x & 15);
    constexpr int kTurn = 4 * WAVES;
    const bool whole = x.cols % kBlk == 0;
    bq_u32x4 v[4];
    auto load = [&](int at) {
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
    };
    const int at0 = threadIdx.x >> 4;
    for (int at = at0; at - at0 < blocks; at += 4 * kTurn) {
      load(at);
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
          *(uint2*)(l8 + (int64_t)b * kBlk + c8) = q[i];
          if (c8 == 0) l8[rows * w.pitch + b] = (uint8_t)byte[i];
        }
      });
    }
    lds_barrier();
  }
  for (int kb = k0; kb < k1; kb += U) {
    static_for<U>([&](auto U_) {
      constexpr int u = decltype(U_)::value;
      if (kb + u < k1) {
        if (!FUSED || kb != k0) load_w(kb + u, u);
        load_x(kb + u, u);
      }
    });
    static_for<U>([&](auto U_) {
      constexpr int u = decltype(U_)::value;
      if (kb + u < k1)
        static_for<MF>([&](auto F_) {
          constexpr int f = decltype(F_)::value;
          const bq_u32x4 p = xc[u][f][0], q = xc[u][f][1];
          const sv_v8i a = {(int)p.x, (int)p.y, (int)p.z, (int)p.w, (int)q.x, (int)q.y, (int)q.z, (int)q.w};
          static_for<NB>([&](auto B_) {
            constexpr int b = decltype(B_)::value;
            const bq_u32x4 lo = wc[u][b][0], hi = wc[u][b][1];
            const sv_v8i e = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
            acc[f][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(e, a, acc[f][b], 0, 0, 0, (int)ws[u][b], f,
                                                                         (int)xs[u]);
          });
        });
    });
  }
  if constexpr (FUSED) lds_barrier();  // the codes are read
  bq_f32x4* const part = (bq_f32x4*)lds;
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) part[(wave * MF * NB + f * NB + b) * 64 + lane] = acc[f][b];
  lds_barrier();
  for (int i = wave; i < MF * NB; i += WAVES) {
    const int row = 16 * (i / NB) + r16;
    bq_f32x4 s = part[i * 64 + lane];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) s += part[(k * MF * NB + i) * 64 + lane];
    // this lane: columns 4 G .. 4 G + 3 of column block i % NB
    const int64_t n = n0 + 16 * (i % NB) + 4 * G;
    if (row >= rows) continue;
    uint16_t* d = y + row * w.rows + n;
    const bq_u32x2 v = {pack_bf16(s.x, s.y), pack_bf16(s.z, s.w)};
    if (n + 4 <= n1) *(bq_u32x2_a2*)d = v;
    else
      for (int k = 0; k < 4 && n + k < n1; ++k) d[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
  }
}

template <bool FUSED, int MF, int NB, int WAVES, int U>
hipError_t run(const Bf16Mat& x, const BlockMat& xq, const BlockMat& w, uint16_t* y, int cols, hipStream_t st) {
  size_t lds = 1024 * WAVES * MF * NB;
  if (FUSED) {
    const size_t codes = (size_t)x.rows * (w.pitch + w.pitch / kBlk);
    if (codes > lds) lds = (codes + 15) / 16 * 16;
  }
  block_serve_kernel<FUSED, MF, NB, WAVES, U>
      <<<dim3((unsigned)((w.rows + cols - 1) / cols)), 64 * WAVES, lds, st>>>(x, xq, w, y, cols);
  return hipGetLastError();
}

// Columns of Y a workgroup makes: all 256 CUs get one workgroup (or C) of
// equal work, since a CU streams from HBM at no more than its share, 20 GB/s
// (of 10240 columns in tiles of 16, 2.5 a CU, 30.7 us; in 256 parts of 40,
// 22.8). At most `most`, what the accumulators of a wave are laid out for.
inline int part_cols(int64_t N, int most) {
  const int64_t c = (N + 256 * most - 1) / (256 * most);
  return (int)((N + 256 * c - 1) / (256 * c));
}

}  // namespace

bool block_serve_fused(int64_t M, int64_t K) { return M <= 16 && M * (round_blk(K) / kBlk) <= kServeBlocks; }

bool block_serve_takes(int64_t M, int64_t N) { return M <= 16 || (M <= 32 && N >= 4096); }

hipError_t launch_block_serve_fused(const Bf16Mat& x, const BlockMat& w, uint16_t* y, hipStream_t st) {
  if (x.rows == 0 || w.rows == 0) return hipSuccess;
  const BlockMat none = {nullptr, nullptr, 0, 0, 0, 0};
  const int cols = part_cols(w.rows, 32);
  return cols <= 16 ? run<true, 1, 1, 8, 4>(x, none, w, y, cols, st) : run<true, 1, 2, 8, 2>(x, none, w, y, cols, st);
}

hipError_t launch_block_serve(const BlockMat& xq, const BlockMat& w, uint16_t* y, hipStream_t st) {
  if (xq.rows == 0 || w.rows == 0) return hipSuccess;
  const Bf16Mat none = {nullptr, 0, 0, 0};
  const int cols = part_cols(w.rows, 48);
  if (xq.rows <= 16)
    return cols <= 16   ? run<false, 1, 1, 8, 4>(none, xq, w, y, cols, st)
           : cols <= 32 ? run<false, 1, 2, 8, 2>(none, xq, w, y, cols, st)
                        : run<false, 1, 3, 8, 2>(none, xq, w, y, cols, st);
  return cols <= 32 ? run<false, 2, 2, 8, 2>(none, xq, w, y, cols, st)
                    : run<false, 2, 3, 8, 2>(none, xq, w, y, cols, st);
}

}  // namespace fp8lin
