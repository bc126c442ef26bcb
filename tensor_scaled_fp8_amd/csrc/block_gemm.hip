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
// (BM + BN cache lines) are copied to LDS by buffer loads, SLOTS of them in
// flight or in use; the scales of a stage (one byte a row) go to registers.
// A wave reads a stage's fragments from LDS to registers during the MFMAs
// of the stage before: read in their own stage, LDS and matrix pipes took
// turns (a k-block of a 256 x 128 tile 1.07 us; this way 0.62). A lane's
// offset past the operand's last row reads zeros, so tiles need no bounds in
// the loop. With few tiles the reduction is split over several workgroups,
// whose FP32 partial sums a second kernel adds in a fixed order: results
// never depend on timing. Bound by the matrix pipes under the power limit
// where the 256 x 256 tile fits (8192^3: 352 us, 3.1 PFLOP/s; the library's FP8
// product 335 in turn with it), by LDS and L2 reads a FLOP below it.
// Within the instruction, the 8 products of 8 consecutive bytes of a lane are
// aligned to the largest of them, and bits below 2^-13 of its power of two are
// dropped towards 0; from there on sums keep 32 bits (measured with products
// that cancel all but a small one). 128 normally distributed products come out
// 2^-16 of their size off (1.5e-5 rms); the length of the reduction adds nothing.
// The 16x16x32 FP8 instructions give the same bits, at half the rate: of the
// matrix instructions only those of wider operands are exact here.
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
  int whole;             // the first tiles: one workgroup each
  int splits;            // workgroups of each other tile; split s takes k-blocks [s nk / splits, (s + 1) nk / splits)
  float* part;           // their FP32 partials
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
__device__ inline void store_wave(lds_u8* wst, int t, const Acc& acc, uint16_t* c, int64_t ldc, int M, int N, int m0,
                                  int n0) {
  constexpr int kChunks = 2 * FN;              // 16-byte chunks of a row
  constexpr int kRowsPer = 64 / kChunks;       // rows a store instruction covers
  const int lane = t & 63, r16 = lane & 15, G = lane >> 4;
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
      // a few blocks at a time, which bounds how many accumulators are
      // moved out of the accumulation registers at once
      if constexpr (ni % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    });
    // one wave's LDS accesses are processed in order: no barrier
    asm volatile("" ::: "memory");
    static_for<16 / kRowsPer>([&](auto K_) {
      const int r = dr + kRowsPer * decltype(K_)::value;
      const lds_u8* src = wst + r * (16 * kChunks) + 16 * (dc ^ (r & (kChunks - 1)));
      const int row = m0 + 16 * mi + r, col = n0 + 8 * dc;
      if (row < M) {
        uint16_t* d = c + (int64_t)row * ldc + col;
        if (col + 8 <= N) {
          __builtin_nontemporal_store(*(const lds_u32x4*)src, (u32x4_a2*)d);
        } else {
#pragma clang loop unroll(disable)
          for (int e = 0; e < N - col; ++e) d[e] = ((const LDS_AS uint16_t*)src)[e];
        }
      }
    });
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  });
}

template <int FMT_A, int FMT_B, int BM, int BN, int SLOTS>
__device__ __forceinline__ void gemm_tile(const Problem& p) {
  constexpr int FM = BM / 32, FN = BN / 32;   // 16-row blocks of a wave
  constexpr int LA = BM / 32, LB = BN / 32;   // loads of a wave and stage
  constexpr int kStage = (BM + BN) * kBlk;
  __shared__ uint4 lds[SLOTS * kStage / 16];
  lds_u8* const l8 = (lds_u8*)lds;

  int pid = blockIdx.x, split = 0, splits = 1;
  if (pid >= p.whole) {
    const int shared = p.tiles_m * p.tiles_n - p.whole;
    split = (pid - p.whole) / shared;
    splits = p.splits;
    pid -= split * shared;
  }
  int tm, tn;
  tile_origin(pid, p.tiles_m, p.tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int k0 = (int)((int64_t)split * p.nk / splits), k1 = (int)((int64_t)(split + 1) * p.nk / splits);
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
  // load i of a stage, A's first; a stage past the last is loaded through a
  // resource of no bytes, so that the count of loads in flight is the same
  // in every step
  auto issue = [&](int slot, int s, auto I_) {
    constexpr int i = decltype(I_)::value;
    const int ko = s < nk ? s * kBlk : 0;
    lds_u8* d = l8 + slot * kStage + 1024 * w;
    if constexpr (i < LA) {
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc((void*)abase, (short)0, s < nk ? abytes : 0, kRsrcWord3);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LDS_AS void*)(d + 4096 * i), 16, offa[i], ko, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc((void*)bbase, (short)0, s < nk ? bbytes : 0, kRsrcWord3);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LDS_AS void*)(d + BM * kBlk + 4096 * (i - LA)), 16, offb[i - LA], ko,
                                               0, 0);
    }
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
  // fragments of stage s in [s % 2], scales in [s % RING]
  constexpr int RING = SLOTS == 3 ? 3 : 4, UNROLL = SLOTS == 3 ? 6 : 4;
  v8i fa[2][FM], fb[2][FN];
  u32x2 xa[RING], xb[RING];
  auto scales = [&](int s, auto R_) {
    constexpr int r = decltype(R_)::value;
    xa[r] = scale_load(p.sa, asz, soffa, kblock(s) * (int)p.sra, FMc{});
    xb[r] = scale_load(p.sb, bsz, soffb, kblock(s) * (int)p.srb, FNc{});
  };
  // fragment r of a stage, B's first
  auto read = [&](int slot, auto P_, auto R_) {
    constexpr int par = decltype(P_)::value, r = decltype(R_)::value;
    if constexpr (r < FN) fb[par][r] = frag(l8 + slot * kStage + (BM + wn * (BN / 2)) * kBlk + 2048 * r);
    else fa[par][r - FN] = frag(l8 + slot * kStage + wm * (BM / 2) * kBlk + 2048 * (r - FN));
  };
  static_for<RING - 1>([&](auto S_) { scales(decltype(S_)::value, S_); });
  static_for<SLOTS>([&](auto S_) {
    static_for<LA + LB>([&](auto I_) { issue(decltype(S_)::value, decltype(S_)::value, I_); });
  });
  wait_vmcnt<(SLOTS - 1) * (LA + LB)>();
  block_sync_lds();
  static_for<FM + FN>([&](auto R_) { read(0, std::integral_constant<int, 0>{}, R_); });
  // step s (J: its index mod UNROLL): stage s is in registers, stage s + 1
  // has landed (newer ones may fly), and stage s + SLOTS goes into the slot
  // of stage s, which every wave is past reading. Loads and the reads of
  // stage s + 1 are spread over the step's MFMAs.
  auto step = [&](auto J_, int s) {
    constexpr int J = decltype(J_)::value, P = J & 1;
    __builtin_amdgcn_sched_barrier(0);
    // (loads of scales may lie anywhere among these, so they are not counted)
    wait_vmcnt<(SLOTS - 2) * (LA + LB)>();
    block_sync_lds();
    scales(s + RING - 1, std::integral_constant<int, (J + RING - 1) % RING>{});
    __builtin_amdgcn_sched_barrier(0);
    static_for<FM * FN>([&](auto T_) {
      constexpr int t = decltype(T_)::value, i = t / FN, j = t % FN;
      constexpr int kReads = FM + FN, kMfma = FM * FN;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[P][j], fa[P][i], acc[i][j], FMT_B, FMT_A, j & 3,
                                                                   (int)xb[J % RING][j >> 2], i & 3,
                                                                   (int)xa[J % RING][i >> 2]);
      constexpr int r0 = t * kReads / kMfma, r1 = (t + 1) * kReads / kMfma;
      static_for<r1 - r0>([&](auto R_) {
        read((J + 1) % SLOTS, std::integral_constant<int, P ^ 1>{}, std::integral_constant<int, r0 + decltype(R_)::value>{});
      });
      constexpr int l0 = t * (LA + LB) / kMfma, l1 = (t + 1) * (LA + LB) / kMfma;
      static_for<l1 - l0>([&](auto L_) {
        issue(J % SLOTS, s + SLOTS, std::integral_constant<int, l0 + decltype(L_)::value>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  int s = 0;
  for (; s + UNROLL <= nk; s += UNROLL)
    static_for<UNROLL>([&](auto J_) { step(J_, s + decltype(J_)::value); });
  const int rest = nk - s;
  static_for<UNROLL - 1>([&](auto J_) {
    if (decltype(J_)::value < rest) step(J_, s + decltype(J_)::value);
  });
  wait_vmcnt<0>();
  block_sync_lds();

  if (splits > 1) {
    // partials in register order: float4 (i FN + j) of thread t
    float* d = p.part + (int64_t)(blockIdx.x - p.whole) * (BM * BN) + 4 * t;
    static_for<FM>([&](auto I_) {
      static_for<FN>([&](auto J_) {
        constexpr int i = decltype(I_)::value, j = decltype(J_)::value;
        *(f32x4*)(d + 1024 * (i * FN + j)) = acc[i][j];
      });
    });
    return;
  }
  store_wave<FM, FN>(
      l8 + w * (16 * 32 * FN), t, [&](auto I_, auto J_) { return acc[decltype(I_)::value][decltype(J_)::value]; }, p.c, p.ldc,
      p.M, p.N, m0 + wm * (BM / 2), n0 + wn * (BN / 2));
}

template <int FMT_A, int FMT_B, int BM, int BN, int SLOTS>
__global__ __launch_bounds__(256, (BM + BN) * SLOTS > 640 ? 1 : 2) void block_gemm_kernel(Problem p) {
  gemm_tile<FMT_A, FMT_B, BM, BN, SLOTS>(p);
}

// ---- the 256 x 256 tile --------------------------------------------------
// 4 waves of 128 x 128 (8 x 8 blocks, 256 accumulators a lane), one wave a
// SIMD, so nothing but the wave's own schedule hides a load or an LDS read:
// a stage's fragments are read under the MFMAs of the stage before it, in
// place where the MFMAs that used a register are past, double-buffered in
// registers otherwise. A is held in two slots of LDS and B in three (160
// KB, all of a CU's); one barrier opens each stage. The slots are objects
// of their own, always named at compile time, so that the compiler can tell
// a slot that is read from one with loads in flight.
constexpr int kBig = 256;
constexpr int kOpBytes = kBig * kBlk;  // 32 KB: one operand's part of a stage
__shared__ uint4 g_a0[kOpBytes / 16];
__shared__ uint4 g_a1[kOpBytes / 16];
__shared__ uint4 g_b0[kOpBytes / 16];
__shared__ uint4 g_b1[kOpBytes / 16];
__shared__ uint4 g_b2[kOpBytes / 16];
template <int S>
__device__ inline lds_u8* a_slot() {
  if constexpr (S % 2 == 0) return (lds_u8*)g_a0;
  else return (lds_u8*)g_a1;
}
template <int S>
__device__ inline lds_u8* b_slot() {
  if constexpr (S % 3 == 0) return (lds_u8*)g_b0;
  else if constexpr (S % 3 == 1) return (lds_u8*)g_b1;
  else return (lds_u8*)g_b2;
}

// c += the scaled product of a 16 x 16 x 128 piece, scale bytes SB and SA of
// the two words. In asm so that the result is tied to the accumulator's
// registers: left free to take others, with all 256 accumulation registers
// in use, the compiler spilled hundreds to memory. Its operands come from
// LDS reads and loads (the compiler waits for those) and nothing reads a
// result before the s_nop after the loop.
template <int FMT_B, int FMT_A, int SB, int SA>
__device__ __forceinline__ void mfma_into(f32x4& c, const v8i& b, const v8i& a, uint32_t sb, uint32_t sa) {
  asm volatile(
      "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] cbsz:%9 blgp:%10"
      : "+a"(c)
      : "v"(b), "v"(a), "v"(sb), "v"(sa), "n"(SB & 1), "n"(SA & 1), "n"(SB >> 1), "n"(SA >> 1), "n"(FMT_B), "n"(FMT_A));
}

template <int FMT_A, int FMT_B>
__device__ __forceinline__ void gemm_tile_big(const Problem& p) {
  int pid = blockIdx.x, split = 0, splits = 1;
  if (pid >= p.whole) {
    const int shared = p.tiles_m * p.tiles_n - p.whole;
    split = (pid - p.whole) / shared;
    splits = p.splits;
    pid -= split * shared;
  }
  int tm, tn;
  tile_origin(pid, p.tiles_m, p.tiles_n, tm, tn);
  const int m0 = tm * kBig, n0 = tn * kBig;
  const int k0 = (int)((int64_t)split * p.nk / splits), k1 = (int)((int64_t)(split + 1) * p.nk / splits);
  const int nk = k1 - k0;

  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w >> 1, wn = w & 1;

  // loads: wave w fills rows 64 w .. 64 w + 63 of either part, 8 rows an
  // instruction (layout as in gemm_tile)
  const uint8_t* const abase = p.a + (int64_t)m0 * p.pa + (int64_t)k0 * kBlk;
  const uint8_t* const bbase = p.b + (int64_t)n0 * p.pb + (int64_t)k0 * kBlk;
  const int abytes = tile_bytes(p.M, m0, kBig, p.pa) - k0 * kBlk, bbytes = tile_bytes(p.N, n0, kBig, p.pb) - k0 * kBlk;
  int offa[8], offb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 8 * (8 * w + i) + (lane >> 3);
    // 32-bit products, kept apart from the sum by an empty asm: fused into
    // a 64-bit multiply-add, each offset would occupy a register pair
    int pa = row * (int)p.pa, pb = row * (int)p.pb;
    asm volatile("" : "+v"(pa), "+v"(pb));
    offa[i] = pa + 16 * ((lane & 7) ^ swz(row));
    offb[i] = pb + 16 * ((lane & 7) ^ swz(row));
  }
  // loads i0 .. i0 + n - 1 of a stage's part; a stage past the last reads
  // zeros through a resource of no bytes, which keeps the counts in flight
  auto issue_a = [&](lds_u8* sl, int s, auto I0_, auto N_) {
    constexpr int i0 = decltype(I0_)::value, n = decltype(N_)::value;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)abase, (short)0, s < nk ? abytes : 0, kRsrcWord3);
    const int ko = s < nk ? s * kBlk : 0;
#pragma unroll
    for (int i = i0; i < i0 + n; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LDS_AS void*)(sl + (8 * w + i) * 1024), 16, offa[i], ko, 0, 0);
  };
  auto issue_b = [&](lds_u8* sl, int s, auto I0_, auto N_) {
    constexpr int i0 = decltype(I0_)::value, n = decltype(N_)::value;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)bbase, (short)0, s < nk ? bbytes : 0, kRsrcWord3);
    const int ko = s < nk ? s * kBlk : 0;
#pragma unroll
    for (int i = i0; i < i0 + n; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LDS_AS void*)(sl + (8 * w + i) * 1024), 16, offb[i], ko, 0, 0);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C8 = std::integral_constant<int, 8>;

  // scales: a lane's eight bytes of A's and of B's 128 rows
  const int asz = (int)(p.sra * p.nk), bsz = (int)(p.srb * p.nk);
  const int soffa = m0 + 128 * wm + 8 * (lane & 15), soffb = n0 + 128 * wn + 8 * (lane & 15);
  auto scales = [&](int s, u32x2& xa, u32x2& xb) {
    const int kb = max(min(k0 + s, p.nk - 1), 0);  // past the last: read again, not used
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void*)p.sa, (short)0, asz, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void*)p.sb, (short)0, bsz, kRsrcWord3);
    xa = __builtin_amdgcn_raw_buffer_load_b64(ra, soffa, kb * (int)p.sra, 0);
    xb = __builtin_amdgcn_raw_buffer_load_b64(rb, soffb, kb * (int)p.srb, 0);
  };

  const int fr = lane & 15, fG = lane >> 4;
  int foff[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) foff[j] = fr * kBlk + (((2 * fG + j) ^ swz(fr)) << 4);
  auto frag = [&](const lds_u8* q, auto M_) -> v8i {
    constexpr int m = decltype(M_)::value;
    const u32x4 lo = *(const lds_u32x4*)(q + foff[0] + 2048 * m);
    const u32x4 hi = *(const lds_u32x4*)(q + foff[1] + 2048 * m);
    return (v8i){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  const int a_row0 = 128 * wm * kBlk, b_row0 = 128 * wn * kBlk;

  f32x4 acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};

  // fragments (P = parity of the stage): A blocks 0..5 in fa, 6 and 7 in
  // fa67[P]; B blocks 0..3 in fb, 4..7 in fb47[P] (176 registers); scales
  // in xa[P], xb[P]
  v8i fa[6], fa67[2][2], fb[4], fb47[2][4];
  u32x2 xa[2], xb[2];
  scales(0, xa[0], xb[0]);
  issue_a(a_slot<0>(), 0, C0{}, C8{});
  issue_b(b_slot<0>(), 0, C0{}, C8{});
  issue_a(a_slot<1>(), 1, C0{}, C8{});
  issue_b(b_slot<1>(), 1, C0{}, C8{});
  issue_b(b_slot<2>(), 2, C0{}, C8{});
  // the accumulators are zeroed while the first loads fly
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
  wait_vmcnt<24>();
  block_sync_lds();
  static_for<6>([&](auto M_) { fa[decltype(M_)::value] = frag(a_slot<0>() + a_row0, M_); });
  static_for<2>([&](auto M_) {
    constexpr int m = decltype(M_)::value;
    fa67[0][m] = frag(a_slot<0>() + a_row0, std::integral_constant<int, 6 + m>{});
  });
  static_for<4>([&](auto N_) {
    constexpr int n = decltype(N_)::value;
    fb[n] = frag(b_slot<0>() + b_row0, N_);
    fb47[0][n] = frag(b_slot<0>() + b_row0, std::integral_constant<int, 4 + n>{});
  });

  // One stage (J: its index mod 6, for compile-time slots and registers).
  // Loads of A of stage s + 2 and B of s + 3 go into the slots of stage s,
  // whose fragments are in registers; reads are of stage s + 1, spread one
  // or two after each MFMA. A fragment register is refilled only after the
  // MFMAs that read it.
  auto stage = [&](auto J_, int s) {
    constexpr int J = decltype(J_)::value, P = J & 1, Q = P ^ 1;
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<8>();   // stage s + 1 and its scales landed; B of s + 2 may fly
    block_sync_lds();  // everyone's loads landed, everyone's reads of stage s are done
    __builtin_amdgcn_sched_barrier(0);
    const lds_u8* na = a_slot<J + 1>() + a_row0;
    const lds_u8* nb = b_slot<J + 1>() + b_row0;
    auto mfma = [&](auto N_, const v8i& a, auto M_) {
      constexpr int n = decltype(N_)::value, m = decltype(M_)::value;
      if constexpr (n < 4)
        mfma_into<FMT_B, FMT_A, n & 3, m & 3>(acc[m][n], fb[n], a, xb[P][n >> 2], xa[P][m >> 2]);
      else
        mfma_into<FMT_B, FMT_A, n & 3, m & 3>(acc[m][n], fb47[P][n - 4], a, xb[P][n >> 2], xa[P][m >> 2]);
    };
    // row blocks 0..3: the next scales, A's loads; A block mi - 1 in place
    // and the double-buffered blocks
    static_for<4>([&](auto MI_) {
      constexpr int mi = decltype(MI_)::value;
      static_for<8>([&](auto N_) {
        constexpr int n = decltype(N_)::value;
        mfma(N_, fa[mi], MI_);
        if constexpr (n == 0 && mi == 0) scales(s + 1, xa[Q], xb[Q]);
        if constexpr (n == 1 || n == 5) issue_a(a_slot<J>(), s + 2, std::integral_constant<int, 2 * mi + (n >> 2)>{}, C1{});
        if constexpr (n == 2) fb47[Q][mi] = frag(nb, std::integral_constant<int, 4 + mi>{});
        if constexpr (n == 4 && mi >= 2) fa67[Q][mi - 2] = frag(na, std::integral_constant<int, 4 + mi>{});
        if constexpr (n == 6 && mi >= 1) fa[mi - 1] = frag(na, std::integral_constant<int, mi - 1>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    // column pairs over rows 4, 5: B's loads; A block 3 in place
    static_for<4>([&](auto C_) {
      constexpr int c = decltype(C_)::value;
      static_for<4>([&](auto D_) {
        constexpr int d = decltype(D_)::value;
        using Nc = std::integral_constant<int, 2 * c + (d >> 1)>;
        mfma(Nc{}, fa[4 + (d & 1)], std::integral_constant<int, 4 + (d & 1)>{});
        if constexpr (d == 1) issue_b(b_slot<J>(), s + 3, C_, C1{});
        if constexpr (d == 2 && c == 0) fa[3] = frag(na, std::integral_constant<int, 3>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    // column pairs over rows 6, 7: B's loads; A blocks 4, 5 and B blocks
    // 0..3 in place
    static_for<4>([&](auto C_) {
      constexpr int c = decltype(C_)::value;
      static_for<4>([&](auto D_) {
        constexpr int d = decltype(D_)::value;
        using Nc = std::integral_constant<int, 2 * c + (d >> 1)>;
        mfma(Nc{}, fa67[P][d & 1], std::integral_constant<int, 6 + (d & 1)>{});
        if constexpr (d == 1) issue_b(b_slot<J>(), s + 3, std::integral_constant<int, 4 + c>{}, C1{});
        if constexpr (c == 0 && d != 1 && d != 3) fa[4 + (d >> 1)] = frag(na, std::integral_constant<int, 4 + (d >> 1)>{});
        if constexpr (c >= 1 && c <= 2 && (d == 0 || d == 2))
          fb[2 * c - 2 + (d >> 1)] = frag(nb, std::integral_constant<int, 2 * c - 2 + (d >> 1)>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };
  // the rest has code of its own: left from within the six, the loop took 3 %
  // longer (the stage index was no longer known to be a scalar)
  int s = 0;
  for (; s + 6 <= nk; s += 6)
    static_for<6>([&](auto J_) { stage(J_, s + decltype(J_)::value); });
  const int rest = nk - s;
  static_for<5>([&](auto J_) {
    if (decltype(J_)::value < rest) stage(J_, s + decltype(J_)::value);
  });
  asm volatile("s_nop 15\n\ts_nop 15");  // the last MFMAs' results may be read
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
  wait_vmcnt<0>();
  block_sync_lds();

  // (the thread index through an empty asm keeps this addressing out of the
  // k-loop, where registers are full)
  int te = t;
  asm volatile("" : "+v"(te));
  if (splits > 1) {
    float* d = p.part + (int64_t)(blockIdx.x - p.whole) * (kBig * kBig) + 4 * te;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) *(f32x4*)(d + 1024 * (i * 8 + j)) = acc[i][j];
    return;
  }
  store_wave<8, 8>(
      (lds_u8*)g_b2 + w * 8192, te, [&](auto I_, auto J_) { return acc[decltype(I_)::value][decltype(J_)::value]; }, p.c,
      p.ldc, p.M, p.N, m0 + 128 * wm, n0 + 128 * wn);
}

template <int FMT_A, int FMT_B>
__global__ __launch_bounds__(256, 1) void block_gemm_big_kernel(Problem p) {
  gemm_tile_big<FMT_A, FMT_B>(p);
}

// sums the partials of one row block (blockIdx.y) of a tile in split order
template <int BM, int BN>
__global__ __launch_bounds__(256) void block_gemm_join_kernel(Problem p) {
  constexpr int FN = BN / 32;
  __shared__ uint4 lds[4 * 32 * FN];
  const int tile = blockIdx.x, i = blockIdx.y;  // the tile of those that are shared
  int tm, tn;
  tile_origin(p.whole + tile, p.tiles_m, p.tiles_n, tm, tn);
  const int t = threadIdx.x, w = t >> 6;
  const int64_t stride = (int64_t)(p.tiles_m * p.tiles_n - p.whole) * (BM * BN);
  const float* s = p.part + (int64_t)tile * (BM * BN) + 1024 * (i * FN) + 4 * t;
  f32x4 acc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[j] = *(const f32x4*)(s + 1024 * j);
  for (int k = 1; k < p.splits; ++k) {
    s += stride;
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[j] += *(const f32x4*)(s + 1024 * j);
  }
  store_wave<1, FN>((lds_u8*)lds + w * (16 * 32 * FN), t, [&](auto, auto J_) { return acc[decltype(J_)::value]; }, p.c,
                    p.ldc, p.M, p.N, tm * BM + (w >> 1) * (BM / 2) + 16 * i, tn * BN + (w & 1) * (BN / 2));
}

// The tile and the split of a product: the least estimated time. Workgroups
// go out in rounds of 256, one a CU, and a k-block takes a round a time of
// its own, less in a round that half fills the chip (the CUs' shares of L2
// and of the power limit are larger). Tiles of full rounds have a workgroup
// each; those of a last round that is not full may have several, which adds
// the join's launch and their FP32 partials' way to memory and back. The
// times are fits to products of 8 .. 288 k-blocks timed alone (256 x 128 by
// its pace among other products, 0.85: alone it runs faster, 0.75, than its
// LDS reads let it under the power limit). In the layers' passes they are
// within 10 % for long reductions and single rounds (4096^3, GPT-175B qkv
// forward and dX, the MLP's dX, 333 rows) and low elsewhere. `fixed` is
// counted once, although a 256 x 256 workgroup has a CU to itself and every
// further round starts and ends anew: dW of 2048 tokens, 16 k-blocks, takes
// 801 us for 631 estimated in 27 rounds, 161 for 121 in 5, 83 for 68 in 2.5; 32
// k-blocks in 2.5 rounds 150 for 131, in 1.25 with a join 95 for 77. The MLP's
// down product takes 83 for 73, products of 10 k-blocks 9 for 7. The shared
// last round
// took the GPT-175B qkv dX from 633 to 601 us and the forward from 706 to
// 692, a 2048 x 10240 x 4096 product from 96 to 95. What each tile is for
// (us, alone; s: the reduction in that many):
//                          256x256       256x128      128x128   128x64    64x64
//   2048 x 36864 x 12288   690           790          1077
//   2048 x 12288 x 36864   676, s2 639   774          986
//   2048 x 10240 x 4096    86            79           84        115       134
//   2048 x 4096 x 20480    157, s2 129   124          150       201       271
//   333 x 15360 x 5120     47            32           43        45        54
//   1024 x 4096 x 8192     66, s2 47     42, s2 39    32
//   997 x 2002 x 1200      22            13           8.9       7.2       8.2
//   64 x 12288 x 4096      38, s3 29     23           15        13        12
struct Plan {
  int bm, bn, splits;
};
inline Plan plan(int64_t M, int64_t N, int64_t nk, bool may_split) {
  struct Tile {
    int bm, bn;
    float fixed;              // us: launch, first loads, stores
    float half, whole, more;  // us a k-block of a round: of at most 128; of 256; of 256 among several
  };
  constexpr Tile kTiles[] = {{256, 256, 5.0f, 1.04f, 1.45f, 1.45f},
                             {256, 128, 5.0f, 0.66f, 0.85f, 0.87f},
                             {128, 128, 3.8f, 0.43f, 0.45f, 0.55f},
                             {128, 64, 3.5f, 0.29f, 0.31f, 0.36f},
                             {64, 64, 3.2f, 0.23f, 0.27f, 0.24f}};
  constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
  Plan best{256, 256, 1};
  float least = 1e30f;
  for (const Tile& t : kTiles) {
    const int64_t tiles = (M + t.bm - 1) / t.bm * ((N + t.bn - 1) / t.bn);
    const int64_t full = tiles / 256, rest = tiles % 256;
    const float round = tiles <= 256 ? t.whole : t.more;
    for (int s : kSplits) {
      const int64_t n = rest * s;  // workgroups after the full rounds
      if (s > 1 && (!may_split || rest == 0 || s > nk / 3 || n > 1024)) break;
      const float part = (float)(n % 256);
      const float last = (float)(n / 256) * t.more +
                         (part == 0 ? 0.0f : part <= 128 ? t.half : t.half + (round - t.half) * (part - 128.0f) / 128.0f);
      const float us = t.fixed + (float)nk * (float)full * round + (float)((nk + s - 1) / s) * last +
                       (s > 1 ? 3.0f + 0.7e-6f * (float)(n * t.bm * t.bn) : 0.0f);
      if (us < least) {
        least = us;
        best = {t.bm, t.bn, s};
      }
    }
  }
  return best;
}

template <int FA, int FB>
hipError_t run(const Problem& p, int bm, int bn, hipStream_t st) {
  const int shared = p.tiles_m * p.tiles_n - p.whole;
  const dim3 grid(p.whole + shared * p.splits);
  const bool join = shared > 0;
  if (bn == 256) {
    block_gemm_big_kernel<FA, FB><<<grid, 256, 0, st>>>(p);
    if (join) block_gemm_join_kernel<256, 256><<<dim3(shared, 8), 256, 0, st>>>(p);
  } else if (bm == 256) {
    block_gemm_kernel<FA, FB, 256, 128, 3><<<grid, 256, 0, st>>>(p);
    if (join) block_gemm_join_kernel<256, 128><<<dim3(shared, 8), 256, 0, st>>>(p);
  } else if (bn == 128) {
    block_gemm_kernel<FA, FB, 128, 128, 4><<<grid, 256, 0, st>>>(p);
    if (join) block_gemm_join_kernel<128, 128><<<dim3(shared, 4), 256, 0, st>>>(p);
  } else if (bm == 128) {
    block_gemm_kernel<FA, FB, 128, 64, 4><<<grid, 256, 0, st>>>(p);
    if (join) block_gemm_join_kernel<128, 64><<<dim3(shared, 4), 256, 0, st>>>(p);
  } else {
    block_gemm_kernel<FA, FB, 64, 64, 4><<<grid, 256, 0, st>>>(p);
    if (join) block_gemm_join_kernel<64, 64><<<dim3(shared, 2), 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

size_t block_gemm_ws_bytes(int64_t M, int64_t N, int64_t R) {
  if (M <= 0 || N <= 0) return 0;
  const Plan q = plan(M, N, round_blk(R) / kBlk, true);
  if (q.splits <= 1) return 0;
  const int64_t tiles = ((M + q.bm - 1) / q.bm) * ((N + q.bn - 1) / q.bn);
  return (size_t)(tiles % 256) * q.splits * q.bm * q.bn * 4;
}

void block_gemm_plan(int64_t M, int64_t N, int64_t R, int* tile_m, int* tile_n, int* splits) {
  const Plan q = plan(M, N, round_blk(R) / kBlk, true);
  *tile_m = q.bm;
  *tile_n = q.bn;
  *splits = q.splits;
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
  p.whole = p.tiles_m * p.tiles_n;
  if (q.splits > 1) p.whole -= p.whole % 256;
  p.part = (float*)ws;
  if (g.fa == FP8_E5M2) return g.fb == FP8_E5M2 ? run<1, 1>(p, q.bm, q.bn, st) : run<1, 0>(p, q.bm, q.bn, st);
  return g.fb == FP8_E5M2 ? run<0, 1>(p, q.bm, q.bn, st) : run<0, 0>(p, q.bm, q.bn, st);
}

}  // namespace fp8lin
