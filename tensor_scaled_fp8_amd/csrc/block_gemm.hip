// Matrix product of two block-scaled FP8 matrices (block.h):
//   C(m, n) = bf16( sum over blocks k of 2^(sA(m,k) + sB(n,k)) *
//                   sum over the 128 elements of A(m, .) B(n, .) ).
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies exactly such a piece: a
// 16 x 16 block of products over one k-block of 128, each lane handing in
// the scale byte of its row, so the scales cost no arithmetic. Sums are
// held in FP32, rounded once to bf16.
//
// Both operands have one row per output index, 128-byte blocks along it.
// A workgroup (4 waves, 2 x 2) makes a BM x BN tile: stages of one k-block
// (BM + BN cache lines) are copied to LDS by buffer loads, kSlots - 1
// stages ahead; the scales of a stage (one byte a row) go to registers. A
// lane's offset past the operand's last row reads zeros, so tiles need no
// bounds in the loop. With few tiles the reduction is split over several
// workgroups, whose FP32 partial sums a second kernel adds in a fixed
// order: results never depend on timing.
#include <type_traits>

#include "block.h"

namespace fp8lin {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
#define LDS_AS __attribute__((address_space(3)))
typedef LDS_AS uint8_t lds_u8;
typedef LDS_AS u32x4 lds_u32x4;
typedef LDS_AS u32x2 lds_u32x2;

constexpr int kRsrcWord3 = 0x00020000;  // buffer resource word 3 for raw byte loads (gfx9 family)

// 16-byte chunk swizzle of a 128-byte LDS row (two rows share one 256-byte
// bank line): the 16 rows of a fragment read fall in distinct bank groups
__device__ inline int swz(int row) { return (row >> 1) & 7; }

template <int N>
__device__ inline void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ inline void block_sync_lds() {
  __builtin_amdgcn_s_waitcnt((63 & 15) | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
template <int N, int I = 0, typename F>
__device__ inline void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<N, I + 1>(f);
  }
}

// One product: operands, sizes, tile grid and the split of its reduction.
struct Problem {
  const uint8_t* a;
  const uint8_t* b;
  const uint8_t* sa;
  const uint8_t* sb;
  uint16_t* c;
  int64_t pa, pb, ldc;   // row pitches (bytes, bytes, elements)
  int64_t sra, srb;      // scale bytes of a k-block
  int M, N, nk;          // nk: k-blocks
  int tiles_m, tiles_n;
  int splits;            // workgroups of a tile; split s takes k-blocks [s nk / splits, (s + 1) nk / splits)
  float* part;           // splits > 1: FP32 partials
};

// tile order: workgroups are dealt round-robin to the 8 XCDs; each XCD gets
// one contiguous range of tiles, in groups of 8 tile rows, so that its
// concurrent tiles share operand panels in its L2
__device__ inline void tile_origin(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int n = tiles_m * tiles_n;
  const int q = n >> 3, r = n & 7, x = pid & 7;
  pid = x * q + min(x, r) + (pid >> 3);
  const int per_group = 8 * tiles_n;
  const int group = pid / per_group;
  const int first = group * 8;
  const int gsize = min(tiles_m - first, 8);
  const int in = pid - group * per_group;
  tm = first + in % gsize;
  tn = in / gsize;
}

// bytes of an operand that a tile starting at row r0 may read
__device__ inline int tile_bytes(int64_t rows, int64_t r0, int tile, int64_t pitch) {
  const int64_t n = rows - r0 < tile ? rows - r0 : tile;
  return (int)(n * pitch);
}

// A wave's FM x FN blocks of 16 x 16 (acc[mi][ni]: lane l holds row
// 16 mi + l % 16, columns 16 ni + 4 (l / 16) .. + 3) to C at (m0, n0),
// through the wave's own LDS so that a store writes whole row pieces: 16
// rows at a time, 32 FN bytes a row, chunks of 16 bytes swizzled.
template <int FM, int FN, typename Acc>
__device__ inline void store_wave(lds_u8* wst, const Acc& acc, uint16_t* c, int64_t ldc, int M, int N, int m0,
                                  int n0) {
  constexpr int kChunks = 2 * FN;              // 16-byte chunks of a row
  constexpr int kRowsPer = 64 / kChunks;       // rows a store instruction covers
  const int lane = threadIdx.x & 63, r16 = lane & 15, G = lane >> 4;
  const int dc = lane % kChunks, dr = lane / kChunks;
  static_for<FM>([&](auto M_) {
    constexpr int mi = decltype(M_)::value;
    static_for<FN>([&](auto N_) {
      constexpr int ni = decltype(N_)::value;
      const f32x4 a = acc(M_, N_);
      const f32x2 lo = {a[0], a[1]}, hi = {a[2], a[3]};
      const u32x2 p = {__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2)),
                       __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2))};
      const int chunk = (2 * ni + (G >> 1)) ^ (r16 & (kChunks - 1));
      *(lds_u32x2*)(wst + r16 * (16 * kChunks) + 16 * chunk + 8 * (G & 1)) = p;
    });
    // one wave's LDS accesses are processed in order: no barrier
    asm volatile("" ::: "memory");
    static_for<16 / kRowsPer>([&](auto K_) {
      const int r = dr + kRowsPer * decltype(K_)::value;
      const u32x4 v = *(const lds_u32x4*)(wst + r * (16 * kChunks) + 16 * (dc ^ (r & (kChunks - 1))));
      const int row = m0 + 16 * mi + r, col = n0 + 8 * dc;
      if (row < M) {
        uint16_t* d = c + (int64_t)row * ldc + col;
        if (col + 8 <= N) {
          __builtin_nontemporal_store(v, (u32x4_a2*)d);
        } else {
          static_for<8>([&](auto E_) {
            constexpr int e = decltype(E_)::value;
            if (col + e < N) d[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
          });
        }
      }
    });
    asm volatile("" ::: "memory");
  });
}

template <int FMT_A, int FMT_B, int BM, int BN, int SLOTS>
__device__ __forceinline__ void gemm_tile(const Problem& p) {
  constexpr int FM = BM / 32, FN = BN / 32;   // 16-row blocks of a wave
  constexpr int LA = BM / 32, LB = BN / 32;   // loads of a wave and stage
  constexpr int kStage = (BM + BN) * kBlk;
  __shared__ uint4 lds[SLOTS * kStage / 16];
  lds_u8* const l8 = (lds_u8*)lds;

  const int ntiles = p.tiles_m * p.tiles_n;
  const int split = blockIdx.x / ntiles;
  int tm, tn;
  tile_origin(blockIdx.x - split * ntiles, p.tiles_m, p.tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int k0 = (int)((int64_t)split * p.nk / p.splits), k1 = (int)((int64_t)(split + 1) * p.nk / p.splits);
  const int nk = k1 - k0;

  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w >> 1, wn = w & 1;

  // loads: instruction i of wave w fills rows 32 i + 8 w .. + 7 of a part;
  // lane l writes LDS chunk l % 8 of row l / 8, which holds global chunk
  // (l % 8) ^ swz(row)
  const uint8_t* const abase = p.a + (int64_t)m0 * p.pa + (int64_t)k0 * kBlk;
  const uint8_t* const bbase = p.b + (int64_t)n0 * p.pb + (int64_t)k0 * kBlk;
  const int abytes = tile_bytes(p.M, m0, BM, p.pa) - k0 * kBlk, bbytes = tile_bytes(p.N, n0, BN, p.pb) - k0 * kBlk;
  int offa[LA], offb[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int row = 32 * i + 8 * w + (lane >> 3);
    offa[i] = row * (int)p.pa + 16 * ((lane & 7) ^ swz(row));
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int row = 32 * i + 8 * w + (lane >> 3);
    offb[i] = row * (int)p.pb + 16 * ((lane & 7) ^ swz(row));
  }
  // a stage past the last is loaded through a resource of no bytes, so that
  // the count of loads in flight is the same in every step
  auto issue = [&](int slot, int s) {
    const int ko = s < nk ? s * kBlk : 0;
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void*)abase, (short)0, s < nk ? abytes : 0, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rb =
        __builtin_amdgcn_make_buffer_rsrc((void*)bbase, (short)0, s < nk ? bbytes : 0, kRsrcWord3);
    lds_u8* d = l8 + slot * kStage + 1024 * w;
#pragma unroll
    for (int i = 0; i < LA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDS_AS void*)(d + 4096 * i), 16, offa[i], ko, 0, 0);
    d += BM * kBlk;
#pragma unroll
    for (int i = 0; i < LB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LDS_AS void*)(d + 4096 * i), 16, offb[i], ko, 0, 0);
  };

  // scales of a stage: the wave's FM (FN) row blocks are FM consecutive
  // bytes of each lane's eight
  const int asz = (int)(p.sra * p.nk), bsz = (int)(p.srb * p.nk);  // below 2^31
  const int sarow = m0 + wm * (BM / 2), sbrow = n0 + wn * (BN / 2);
  const int soffa = (sarow & ~127) + ((sarow >> 4) & 7) + 8 * (lane & 15);
  const int soffb = (sbrow & ~127) + ((sbrow >> 4) & 7) + 8 * (lane & 15);
  auto kblock = [&](int s) { return max(min(k0 + s, p.nk - 1), 0); };  // past the last: read again, not used
  auto scale_load = [&](const uint8_t* base, int bytes, int off, int so, auto F_) -> u32x2 {
    constexpr int F = decltype(F_)::value;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, bytes, kRsrcWord3);
    u32x2 v = {0, 0};
    if constexpr (F == 8) v = __builtin_amdgcn_raw_buffer_load_b64(r, off, so, 0);
    else if constexpr (F == 4) v.x = __builtin_amdgcn_raw_buffer_load_b32(r, off, so, 0);
    else v.x = __builtin_amdgcn_raw_buffer_load_b16(r, off, so, 0);
    return v;
  };

  const int fr = lane & 15, fG = lane >> 4;
  int foff[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) foff[j] = fr * kBlk + (((2 * fG + j) ^ swz(fr)) << 4);
  auto frag = [&](const lds_u8* q) -> v8i {
    const u32x4 lo = *(const lds_u32x4*)(q + foff[0]);
    const u32x4 hi = *(const lds_u32x4*)(q + foff[1]);
    return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};

  using FMc = std::integral_constant<int, FM>;
  using FNc = std::integral_constant<int, FN>;
  u32x2 xa[SLOTS - 1], xb[SLOTS - 1];  // scales of the stages in flight
  static_for<SLOTS - 1>([&](auto S_) {
    constexpr int s = decltype(S_)::value;
    xa[s] = scale_load(p.sa, asz, soffa, kblock(s) * (int)p.sra, FMc{});
    xb[s] = scale_load(p.sb, bsz, soffb, kblock(s) * (int)p.srb, FNc{});
    issue(s, s);
  });
  // step s: the stage's loads are done (the newer stages' may fly) and
  // every wave is past its reads of stage s - 1, whose slot is refilled
  auto step = [&](int s, int slot) {
    wait_vmcnt<(SLOTS - 2) * (LA + LB + 2)>();
    block_sync_lds();
    const u32x2 ca = xa[0], cb = xb[0];
#pragma unroll
    for (int i = 0; i + 1 < SLOTS - 1; ++i) {
      xa[i] = xa[i + 1];
      xb[i] = xb[i + 1];
    }
    xa[SLOTS - 2] = scale_load(p.sa, asz, soffa, kblock(s + SLOTS - 1) * (int)p.sra, FMc{});
    xb[SLOTS - 2] = scale_load(p.sb, bsz, soffb, kblock(s + SLOTS - 1) * (int)p.srb, FNc{});
    issue(slot == 0 ? SLOTS - 1 : slot - 1, s + SLOTS - 1);
    const lds_u8* la = l8 + slot * kStage + wm * (BM / 2) * kBlk;
    const lds_u8* lb = l8 + slot * kStage + (BM + wn * (BN / 2)) * kBlk;
    v8i fb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = frag(lb + 2048 * j);
    static_for<FM>([&](auto I_) {
      constexpr int i = decltype(I_)::value;
      const v8i fa = frag(la + 2048 * i);
      static_for<FN>([&](auto J_) {
        constexpr int j = decltype(J_)::value;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa, acc[i][j], FMT_B, FMT_A, j & 3,
                                                                     (int)cb[j >> 2], i & 3, (int)ca[i >> 2]);
      });
    });
  };
  int slot = 0;
  for (int s = 0; s < nk; ++s) {
    step(s, slot);
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  }
  wait_vmcnt<0>();
  block_sync_lds();

  if (p.splits > 1) {
    // partials in register order: float4 (i FN + j) of thread t
    float* d = p.part + ((int64_t)split * ntiles + (tm * p.tiles_n + tn)) * (BM * BN) + 4 * t;
    static_for<FM>([&](auto I_) {
      static_for<FN>([&](auto J_) {
        constexpr int i = decltype(I_)::value, j = decltype(J_)::value;
        *(f32x4*)(d + 1024 * (i * FN + j)) = acc[i][j];
      });
    });
    return;
  }
  store_wave<FM, FN>(
      l8 + w * (16 * 32 * FN), [&](auto I_, auto J_) { return acc[decltype(I_)::value][decltype(J_)::value]; }, p.c, p.ldc,
      p.M, p.N, m0 + wm * (BM / 2), n0 + wn * (BN / 2));
}

template <int FMT_A, int FMT_B, int BM, int BN, int SLOTS>
__global__ __launch_bounds__(256) void block_gemm_kernel(Problem p) {
  gemm_tile<FMT_A, FMT_B, BM, BN, SLOTS>(p);
}

// sums the partials of one row block (blockIdx.y) of a tile in split order
template <int BM, int BN>
__global__ __launch_bounds__(256) void block_gemm_join_kernel(Problem p) {
  constexpr int FN = BN / 32;
  __shared__ uint4 lds[4 * 32 * FN];
  const int tile = blockIdx.x, i = blockIdx.y;
  const int tm = tile / p.tiles_n, tn = tile - tm * p.tiles_n;
  const int t = threadIdx.x, w = t >> 6;
  const int64_t stride = (int64_t)p.tiles_m * p.tiles_n * (BM * BN);
  const float* s = p.part + (int64_t)tile * (BM * BN) + 1024 * (i * FN) + 4 * t;
  f32x4 acc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[j] = *(const f32x4*)(s + 1024 * j);
  for (int k = 1; k < p.splits; ++k) {
    s += stride;
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[j] += *(const f32x4*)(s + 1024 * j);
  }
  store_wave<1, FN>((lds_u8*)lds + w * (16 * 32 * FN), [&](auto, auto J_) { return acc[decltype(J_)::value]; }, p.c,
                    p.ldc, p.M, p.N, tm * BM + (w >> 1) * (BM / 2) + 16 * i, tn * BN + (w & 1) * (BN / 2));
}

// The tile and the split for a product: see plan().
struct Plan {
  int bm, bn, splits;
};
inline Plan plan(int64_t M, int64_t N, int64_t nk, bool may_split) {
  Plan q{128, 128, 1};
  const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
  if (may_split && tiles < 256) {
    int64_t s = 512 / tiles;
    if (s > nk / 4) s = nk / 4;
    if (s > 1) q.splits = (int)s;
  }
  return q;
}

template <int FA, int FB>
hipError_t run(const Problem& p, hipStream_t st) {
  const int ntiles = p.tiles_m * p.tiles_n;
  block_gemm_kernel<FA, FB, 128, 128, 2><<<dim3(ntiles * p.splits), 256, 0, st>>>(p);
  if (p.splits > 1) block_gemm_join_kernel<128, 128><<<dim3(ntiles, 4), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t block_gemm_ws_bytes(int64_t M, int64_t N, int64_t R) {
  if (M <= 0 || N <= 0) return 0;
  const Plan q = plan(M, N, round_blk(R) / kBlk, true);
  if (q.splits <= 1) return 0;
  return (size_t)q.splits * ((M + q.bm - 1) / q.bm * q.bm) * ((N + q.bn - 1) / q.bn * q.bn) * 4;
}

hipError_t launch_block_gemm(const BlockGemm& g, void* ws, size_t ws_bytes, hipStream_t st) {
  const int64_t M = g.A.rows, N = g.B.rows, nk = round_blk(g.A.cols) / kBlk;
  if (M == 0 || N == 0) return hipSuccess;
  const Plan q = plan(M, N, nk, ws && ws_bytes >= block_gemm_ws_bytes(M, N, g.A.cols));
  Problem p;
  p.a = g.A.codes;
  p.b = g.B.codes;
  p.sa = g.A.scales;
  p.sb = g.B.scales;
  p.c = g.C;
  p.pa = g.A.pitch;
  p.pb = g.B.pitch;
  p.ldc = g.ldc;
  p.sra = g.A.srows;
  p.srb = g.B.srows;
  p.M = (int)M;
  p.N = (int)N;
  p.nk = (int)nk;
  p.tiles_m = (int)((M + q.bm - 1) / q.bm);
  p.tiles_n = (int)((N + q.bn - 1) / q.bn);
  p.splits = q.splits;
  p.part = (float*)ws;
  if (g.fa == FP8_E5M2) return g.fb == FP8_E5M2 ? run<1, 1>(p, st) : run<1, 0>(p, st);
  return g.fb == FP8_E5M2 ? run<0, 1>(p, st) : run<0, 0>(p, st);
}

}  // namespace fp8lin
