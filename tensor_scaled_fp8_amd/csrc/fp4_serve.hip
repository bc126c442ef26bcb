// The linear on a stored 4-bit weight: Y [M, N] = X [M, K] W, X stored in
// E4M3. A workgroup makes a tile of 16 rows and 16 columns; its waves share
// out the k-blocks and add their sums over LDS in wave order. The scaled
// matrix instruction takes W's 4-bit codes and X's 8-bit ones as they are.
#include "fp4.h"

namespace fp8lin {
namespace {

typedef int f4_v8i __attribute__((ext_vector_type(8)));

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void fp4_serve_kernel(BlockMat x, Fp4Mat w, uint16_t* __restrict__ y) {
  __shared__ bq_f32x4 part[WAVES][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, G = lane >> 4;
  const int64_t panel = blockIdx.x, row = (int64_t)blockIdx.y * 16 + r, kblocks = fp4_kblocks(w.K);
  const uint8_t* wc = w.codes + panel * kblocks * 1024 + 16 * lane;
  const uint8_t* ws = w.scales + panel * (kblocks / 4) * 256 + 4 * lane;
  const bool mine = row < x.rows;
  const uint8_t* xc = x.codes + row * x.pitch + 16 * G;
  const uint8_t* xs = x.scales + scale_pos(row);
  const int nk = (int)(x.pitch / kBlk);
  bq_f32x4 acc = {0, 0, 0, 0};
  for (int kb = wave; kb < nk; kb += WAVES) {
    const bq_u32x4 c = *(const bq_u32x4*)(wc + (int64_t)kb * 1024);
    const uint32_t sw = ws[(int64_t)(kb >> 2) * 256 + (kb & 3)];
    bq_u32x4 p = {0, 0, 0, 0}, q = {0, 0, 0, 0};
    uint32_t sx = 127;
    if (mine) {
      p = *(const bq_u32x4*)(xc + (int64_t)kb * kBlk);
      q = *(const bq_u32x4*)(xc + (int64_t)kb * kBlk + 64);
      sx = xs[(int64_t)kb * x.srows];
    }
    const f4_v8i e = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
    const f4_v8i a = {(int)p.x, (int)p.y, (int)p.z, (int)p.w, (int)q.x, (int)q.y, (int)q.z, (int)q.w};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(e, a, acc, 4, 0, 0, (int)sw, 0, (int)sx);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave || !mine) return;
#pragma unroll
  for (int i = 1; i < WAVES; ++i) acc += part[i][lane];
  const int64_t n = panel * 16 + 4 * G;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (n + k < w.N) y[row * w.N + n + k] = (uint16_t)pack_bf16(acc[k], 0.0f);
}

}  // namespace

hipError_t launch_fp4_linear(const BlockMat& x, const Fp4Mat& w, uint16_t* y, hipStream_t st) {
  if (x.rows == 0 || w.N == 0) return hipSuccess;
  fp4_serve_kernel<4><<<dim3((unsigned)((w.N + 15) / 16), (unsigned)((x.rows + 15) / 16)), 256, 0, st>>>(x, w, y);
  return hipGetLastError();
}

}  // namespace fp8lin
