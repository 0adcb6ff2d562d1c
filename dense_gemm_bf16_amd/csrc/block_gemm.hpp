// Products over e4m3 operands with a scale for each block of 128, and the
// experts' products (rows sorted by expert) over e4m3, bf16 and fp16:
//
//   dense     C[m,n] = sum_b SA[b,m] SB[n/128,b] sum_{k in block b} A[m,k] B[n,k]
//   experts   the same for every row p of expert e's range
//             [offsets[e], offsets[e+1]), with A's row rows[p] (or p) and
//             expert e's B and SB; bf16 and fp16 operands carry no scales
//
// Two kernels.  block_tile_kernel stages BM x BN tiles through LDS for many
// rows; block_row_kernel streams B straight into registers for few rows.
// Both walk K in steps of 128 bytes of a row: one scale block of e4m3, 64
// elements of a 16-bit type.
//
// A scale in fp32 cannot ride in the matrix instruction (its own scales are
// powers of two), so each K-step's partial sums of a 16 x 16 block start
// from zero in one 16x16x128 MFMA and are added to the fp32 accumulators by
// one FMA each with SA * SB: 4 FMAs (16 cycles of the SIMD's vector unit)
// per MFMA of 32 cycles, issued while the next MFMA runs.
//
// Measured (MI355X): 8192 x 10240 x 8192 bf16 out 571-608 us, 2260-2410
// TFLOP/s, the matrix cores 58 % busy; 1 x 8192 x 8192 12-13 us (memory); 64,
// 128, 256 rows by 8192 x 8192 15, 20.5, 29 us (the L2: tile traffic of 13-15
// TB/s when the lines come in from the fabric, whatever the ring's depth).
#pragma once

#include "gemm_kernel.hpp"

namespace gemm {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStepBytes = 128;     // bytes of a row in one K-step
constexpr int kMaxKSteps = 1024;    // K-steps whose B scales are held in LDS
constexpr int kScaleBlock = 128;    // rows of B (and columns of C) of one scale

// Operand types.
enum : int { kOpE4m3 = 0, kOpBf16 = 1, kOpF16 = 2 };

struct BlockArgs {
  const uint8_t* A;
  const uint8_t* B;
  void* C;
  const float* SA;         // SA[b * ldsa + row of A]
  const float* SB;         // SB[(n / 128) * ldsb + b]
  const int32_t* offsets;  // experts: E + 1 row offsets; null: dense
  const int32_t* rows;     // experts: A's row of each row of C, or null
  int64_t lda, ldb;        // bytes
  int64_t ldc;             // elements
  int64_t ldsa, ldsb;
  int64_t stride_b;   // bytes from one expert's B to the next
  int64_t stride_sb;  // floats from one expert's SB to the next
  int32_t M;          // rows of C
  int32_t N;
  int32_t kbytes;     // bytes of a row of A or B that count
  int32_t a_rows;     // rows of A
  int32_t E;          // experts (1: dense)
  int32_t tiles_n;
  int32_t k_steps;
  int32_t row_tiles;  // dense: row tiles; experts: an upper bound on them
  int32_t group_m;    // raster group height in tiles
  int32_t k_rot;      // K-step at which tile column j starts: j * k_rot, wrapped around
};

// ------------------------------------------------------------- row tiles

// Expert e's rows of C, clamped so that no offsets, whatever they hold,
// lead outside C.
__device__ __forceinline__ void expert_rows(const BlockArgs& a, int e, int& begin, int& end) {
  const int b = a.offsets[e], n = a.offsets[e + 1];
  begin = b < 0 ? 0 : b;
  end = n > a.M ? a.M : n;
  if (end < begin) end = begin;
}

// Inclusive sum over the wave's lanes, held below 2^30 (ranges that overlap
// could add up to more than an int holds; those that do not stay below it).
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d, 64);
    if (lane >= d) v = min(v + o, (1 << 30) - 1);
  }
  return v;
}

struct RowTile {
  int expert, begin, end;  // rows [begin, end) of C, at most BM of them used
};

// Row tiles (of BM rows) of all experts: expert e has ceil(rows / BM).  At
// most the bound that the grid is made for.
__device__ __forceinline__ int count_row_tiles(const BlockArgs& a, int BM, int lane) {
  int total = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    int b = 0, n = 0;
    if (e0 + lane < a.E) expert_rows(a, e0 + lane, b, n);
    total += __shfl(wave_scan((n - b + BM - 1) / BM, lane), 63, 64);
    total = min(total, a.row_tiles);
  }
  return __builtin_amdgcn_readfirstlane(total);
}

// The t-th row tile, experts in order; false past the last one.
__device__ __forceinline__ bool find_row_tile(const BlockArgs& a, int BM, int t, int lane,
                                              RowTile& r) {
  int before = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    int b = 0, n = 0;
    if (e0 + lane < a.E) expert_rows(a, e0 + lane, b, n);
    const int tiles = (n - b + BM - 1) / BM;
    const int upto = min(before, 1 << 30) + wave_scan(tiles, lane);
    const uint64_t hit = __ballot(t < upto);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);  // the first expert whose tiles pass t
      r.expert = e0 + l;
      r.begin = __builtin_amdgcn_readlane(b, l) +
                (t - __builtin_amdgcn_readlane(upto - tiles, l)) * BM;
      r.end = __builtin_amdgcn_readlane(n, l);
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// A's row of row p of C (p < end), or -1 where the rows array points outside A.
__device__ __forceinline__ int source_row(const BlockArgs& a, int p) {
  if (!a.rows) return p;
  const int r = a.rows[p];
  return r >= 0 && r < a.a_rows ? r : -1;
}

// ------------------------------------------------------------------ MFMA

// What a lane holds of one fragment (16 rows of 128 bytes): two 16-byte
// chunks of its row.  Which k a chunk stands for does not matter as long as
// both operands agree.
//
// e4m3 has two forms.  The 8-bit MFMA adds eight products at a time (those of
// eight consecutive bytes), each cut towards zero to a multiple of 2^(E - 13),
// where E is the largest sum of two codes' exponents among the eight (-6 for
// subnormal codes), and these sums in fp32 (found on MI355X by cancelling
// products, the same in every shape here).  So a block's sum is off by less
// than 7 x 2^-13 of its eights' 2^E: 1.5e-5 of C in norm on normal values, a
// hundredth of a bf16 output's rounding and a tenth of an fp16 one's, so 16-bit
// outputs take it; a product beside one 2^13 times as large that something
// else cancels is lost.  An fp32 output would show it, so there the codes are
// widened to bf16, which holds every e4m3 value, and the bf16 MFMA keeps whole
// fp32 sums, at half the rate.
template <int OP, int OUT>
struct Step {
  static constexpr bool kWide = OP == kOpE4m3 && OUT == kStoreF32;
  static constexpr int kRegs = kWide ? 4 : 2;  // 16-byte registers of a fragment
  struct Frag {
    u32x4 v[kRegs];
  };
  // A fragment from its two chunks.
  static __device__ __forceinline__ Frag make(const u32x4& lo, const u32x4& hi) {
    Frag f;
    if constexpr (kWide) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t c = h ? hi[w] : lo[w];
          f.v[2 * h + w / 2][w % 2 * 2] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
          f.v[2 * h + w / 2][w % 2 * 2 + 1] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
        }
    } else {
      f.v[0] = lo;
      f.v[1] = hi;
    }
    return f;
  }
  // c + the step's sums: D[n][m] += sum_k B[n][k] A[m][k].
  static __device__ __forceinline__ f32x4 mfma(const Frag& b, const Frag& a, f32x4 c) {
    if constexpr (OP == kOpE4m3 && !kWide) {
      const i32x8 vb = {(int)b.v[0][0], (int)b.v[0][1], (int)b.v[0][2], (int)b.v[0][3],
                        (int)b.v[1][0], (int)b.v[1][1], (int)b.v[1][2], (int)b.v[1][3]};
      const i32x8 va = {(int)a.v[0][0], (int)a.v[0][1], (int)a.v[0][2], (int)a.v[0][3],
                        (int)a.v[1][0], (int)a.v[1][1], (int)a.v[1][2], (int)a.v[1][3]};
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, c, 0, 0, 0, 0, 0, 0);
    } else {
#pragma unroll
      for (int h = 0; h < kRegs; ++h) {
        if constexpr (OP == kOpF16)
          c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b.v[h]),
                                                     __builtin_bit_cast(f16x8, a.v[h]), c, 0, 0, 0);
        else
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b.v[h]),
                                                      __builtin_bit_cast(bf16x8, a.v[h]), c, 0, 0, 0);
      }
      return c;
    }
  }
};

// One LDS-DMA load of 4 bytes per lane (see dma16).
__device__ __forceinline__ void dma4(const u32x4& rsrc, uint32_t lds_addr, uint32_t voff,
                                     uint32_t soff) {
  asm volatile(
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, %3 offen lds" ::"{m0}"(
          __builtin_amdgcn_readfirstlane(lds_addr)),
      "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff))
      : "memory");
}

// ----------------------------------------------------------- tile kernel

// BM x BN tiles, WM x WN waves, a ring of S LDS slots of 128-byte rows
// swizzled as in the direct-to-LDS kernel.  Per K-step X: wait until its
// loads have landed (those of the S - 2 steps after it may be in flight),
// barrier (which also frees the slot of step X - 1), then the wave's MFMAs
// with the loads of step X + S - 1 spread between them.  Every step issues
// the same loads, those past K reading zeros, so the waits count them.
template <int BM, int BN, int WM, int WN, int WK, int S, int OP, int OUT>
__global__ __attribute__((amdgpu_flat_work_group_size(WM * WN * WK * 64, WM * WN * WK * 64),
                          amdgpu_waves_per_eu(2))) void
block_tile_kernel(BlockArgs a) {
  using Cfg = TileCfg<BM, BN, 64, WM, WN, S, 3, 16>;
  constexpr int T = Cfg::kThreads, W = WM * WN;  // threads and waves of one K group
  constexpr int FM = Cfg::kFragM, FN = Cfg::kFragN;
  constexpr int LA = Cfg::kLoadsA, LB = Cfg::kLoadsB, L = LA + LB;
  constexpr int RPI = T / 8;  // rows of one load of all threads
  constexpr bool kScaled = OP == kOpE4m3;
  using St = Step<OP, OUT>;
  // A widened fragment takes twice the registers, too many for this form,
  // and a load of all threads has to be half a wave row of A
  constexpr bool kPipe = S == 2 && (FM == 4 || FM == 8) && RPI * 2 == Cfg::kWaveM && !St::kWide;
  constexpr int NB = (BN + kScaleBlock - 1) / kScaleBlock;  // scale blocks across a tile
  constexpr int SA = BM < 64 ? 64 : BM;                     // row scales of a slot
  constexpr int SS = kPipe ? 3 : S;                         // slots of row scales
  constexpr int kInFlight = (S - 2) * (L + (kScaled ? 1 : 0));
  static_assert(RPI % 16 == 0, "the swizzle repeats every 16 rows");
  static_assert(kScaleBlock % Cfg::kWaveN == 0, "a wave's columns share one scale");
  static_assert(SA / 64 <= W, "one wave loads 64 row scales");
  static_assert(kInFlight < 64, "vmcnt range");

  __shared__ __attribute__((aligned(1024))) uint8_t smem_raw[WK * Cfg::kLdsBytes];
  __shared__ float sa_lds[kScaled ? WK * SS * SA : 1];
  __shared__ float sb_lds[kScaled ? NB * kMaxKSteps : 1];
  const int tid = threadIdx.x % T;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = WK > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / T) : 0;
  lds_u8* const smem = (lds_u8*)smem_raw + kg * Cfg::kLdsBytes;
  const uint32_t smem_addr = (uint32_t)(uintptr_t)smem;
  typedef const __attribute__((address_space(3))) float lds_f32;
  lds_f32* const sa_s = (lds_f32*)sa_lds + kg * SS * SA;
  lds_f32* const sb_s = (lds_f32*)sb_lds;
  const int wm = wave / WN, wn = wave % WN;

  // ---- which tile --------------------------------------------------------
  const int row_tiles = a.offsets ? count_row_tiles(a, BM, lane) : a.row_tiles;
  const int units = row_tiles * a.tiles_n;
  if ((int)blockIdx.x >= units) return;  // the grid is an upper bound
  const int logical = xcd_remap(blockIdx.x, units);
  const int span = a.group_m * a.tiles_n;
  const int gid = logical / span;
  const int first = gid * a.group_m;
  const int gsz = min(row_tiles - first, a.group_m);
  const int in = logical - gid * span;
  const int rt = first + in % gsz;
  const int tn = in / gsz, n0 = tn * BN;
  RowTile tile;
  if (a.offsets) {
    if (!find_row_tile(a, BM, rt, lane, tile)) return;
  } else {
    tile = RowTile{0, rt * BM, a.M};
  }
  const int m0 = tile.begin;
  const int rows_a = min(BM, tile.end - m0);
  const int rows_b = min(BN, a.N - n0);

  // ---- loads -------------------------------------------------------------
  const bool gather = a.rows != nullptr;
  const u32x4 rsrc_a = gather ? make_rsrc(a.A, (uint32_t)((int64_t)a.a_rows * a.lda))
                              : make_rsrc(a.A + (int64_t)m0 * a.lda, (uint32_t)(rows_a * a.lda));
  const u32x4 rsrc_b = make_rsrc(a.B + tile.expert * a.stride_b + (int64_t)n0 * a.ldb,
                                 (uint32_t)(rows_b * a.ldb));
  const int r0 = tid / 8;
  const int chunk = (tid & 7) ^ swz<3, 8>(r0);
  uint32_t voff[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int row = (i < LA ? i : i - LA) * RPI + r0;
    if (i < LA) {
      const int src = row < rows_a ? (gather ? source_row(a, m0 + row) : row) : -1;
      voff[i] = src >= 0 ? (uint32_t)(src * (int)a.lda + chunk * 16) : kOOB;
    } else {
      voff[i] = row < rows_b ? (uint32_t)(row * (int)a.ldb + chunk * 16) : kOOB;
    }
  }
  // this lane's row scale; waves past the tile's rows load the same ones
  // again (to the same place), so that all waves issue as many loads
  const int srow = wave % (SA / 64) * 64;
  uint32_t voff_s = kOOB;
  if constexpr (kScaled) {
    const int row = srow + lane;
    if (row < rows_a) {
      const int src = gather ? source_row(a, m0 + row) : m0 + row;
      if (src >= 0) voff_s = (uint32_t)src * 4;
    }
    // the tile's B scales of every K-step, once
    const float* sb = a.SB + tile.expert * a.stride_sb;
    const int per = (a.k_steps + 63) / 64;
    for (int c = kg * W + wave; c < NB * per; c += W * WK) {
      const int nb = c / per, k = (c % per) * 64 + lane;
      const int row = n0 / kScaleBlock + nb;
      const u32x4 rs = make_rsrc(sb + (int64_t)row * a.ldsb,
                                 row * kScaleBlock < a.N ? (uint32_t)a.k_steps * 4 : 0u);
      dma4(rs, (uint32_t)(uintptr_t)sb_s + (nb * kMaxKSteps + (c % per) * 64) * 4, (uint32_t)k * 4,
           0u);
    }
  }
  const bool past_k = (a.k_steps - 1) * kStepBytes + chunk * 16 >= a.kbytes;  // in the last step
  // This group's X-th step of K: X * WK + kg, from the tile's starting point
  // on (k_steps or more: past the last one).
  const int rot = a.k_steps > 0 ? __builtin_amdgcn_readfirstlane(tn * a.k_rot % a.k_steps) : 0;
  auto step_of = [&](int X) __attribute__((always_inline)) {
    const int k = X * WK + kg;
    const int r = k + rot >= a.k_steps ? k + rot - a.k_steps : k + rot;
    return k < a.k_steps ? r : k;
  };
  // load i of K-step k into ring slot `slot`
  auto load_one = [&](int k, int slot, int i) __attribute__((always_inline)) {
    const uint32_t dst = smem_addr + slot * Cfg::kStageBytes + (i < LA ? 0 : Cfg::kABytes) +
                         (((i < LA ? i : i - LA) * T + wave * 64) * 16);
    // past K, and in the steps past the last one, a load reads zeros: no
    // branch splits the loop body
    const uint32_t v = k >= a.k_steps - (past_k ? 1 : 0) ? kOOB : voff[i];
    dma16(i < LA ? rsrc_a : rsrc_b, dst, v, (uint32_t)(k * kStepBytes));
  };
  auto load_scales = [&](int k, int slot) __attribute__((always_inline)) {
    if constexpr (kScaled) {
      const u32x4 rs = make_rsrc(a.SA + k * a.ldsa, k < a.k_steps ? (uint32_t)a.a_rows * 4 : 0u);
      dma4(rs, (uint32_t)(uintptr_t)sa_s + (slot * SA + srow) * 4, voff_s, 0u);
    }
  };
  // Zero the bytes past K of the 16-byte chunk that straddles it, each
  // thread in the chunks it loaded (their loads have landed).
  auto trim_one = [&](int k, int slot, int i) __attribute__((always_inline)) {
    const int keep = a.kbytes - (k * kStepBytes + chunk * 16);
    if (keep > 0 && keep < 16) {
      lds_u32x4* p = (lds_u32x4*)(smem + slot * Cfg::kStageBytes + (i < LA ? 0 : Cfg::kABytes) +
                                  ((i < LA ? i : i - LA) * T + tid) * 16);
      u32x4 v = *p;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int left = keep - 4 * w;
        v[w] &= left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
      }
      *p = v;
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

  if constexpr (!kPipe) {
#pragma unroll
    for (int p = 0; p < S - 1; ++p) {
#pragma unroll
      for (int i = 0; i < L; ++i) load_one(step_of(p), p, i);
      load_scales(step_of(p), p);
    }
  }

  // byte address of this lane's first chunk of its row in fragment 0; the
  // second chunk is 64 bytes away before the swizzle, so 64 by XOR after it
  const int lrow = lane & 15;
  const int at = lrow * kStepBytes + (((lane >> 4) ^ swz<3, 8>(lrow)) << 4);
  const lds_u8* const pa = smem + wm * Cfg::kWaveM * kStepBytes;
  const lds_u8* const pb = smem + Cfg::kABytes + wn * Cfg::kWaveN * kStepBytes;
  using Frag = typename St::Frag;
  auto read_frag = [&](const lds_u8* base, int f) __attribute__((always_inline)) {
    const u32x4 lo = *(const lds_u32x4*)(base + f * 16 * kStepBytes + at);
    const u32x4 hi = *(const lds_u32x4*)(base + f * 16 * kStepBytes + (at ^ 64));
    return St::make(lo, hi);
  };

  const int rounds = (a.k_steps + WK - 1) / WK;
  // A wave whose rows all lie past the tile's last one (an expert's last
  // tile, C's last rows) only loads: the other waves of its SIMD then have
  // the matrix core to themselves.
  const bool idle = wm * Cfg::kWaveM >= rows_a;
  if constexpr (kPipe) {
    // Two slots, each refilled in two parts as soon as a part is read, so
    // that about a whole step's loads are always in flight (with one barrier
    // a step the loads had to land within the step that issued them: 1.4 us
    // a step of 64 KB without any MFMA, against 0.9 us).  Part 1 is B and
    // the A rows of each wave row's first half, part 2 its other half.  Two
    // barriers a step:
    //   P1(X), before the last two rows of step X - 1: part 1 of step X has
    //     landed; step X - 1's last fragments are in registers, so part 2 of
    //     step X + 1 is issued in its place;
    //   P2(X), half way through step X: part 2 of step X has landed; B and
    //     the first half of A are in registers, so part 1 of step X + 2 is
    //     issued in their place.
    // Either way two parts are in flight past the one that is awaited.  The
    // MFMAs of the last two rows cover P1 and the first reads of the next
    // step, whose B fragments replace the old ones one by one as their last
    // MFMAs issue.  MFMA q (row by row, in the last two rows column by
    // column) writes partial sum q % 4, which is added to its accumulator
    // once MFMA q + 3 has issued.
    constexpr int NQ = FM * FN, Q0 = (FM - 2) * FN;  // MFMAs of a step, and of its rows before P1
    constexpr int QP = (FM == 8 ? 3 : 1) * FN;       // the MFMA before which P2 is
    constexpr int kParts = L + (kScaled ? 1 : 0);    // loads of both parts
    static_assert(FM == 4 || FM == 8, "the tables below");
    // Buffer of row i's A fragment, and the row at whose first MFMA it is
    // read (rows 0 and 1: in the last two rows of the step before; the second
    // half's not before P2): rows FM - 2, FM - 1 and the next step's 0 are
    // held at once.  Eight rows make do with three buffers, each reused once
    // its row's MFMAs have issued.
    // (Row 2 not before row 1: until then the last additions of the step
    // before use the scale that its own replaces.)
    constexpr int NBUF = FM == 8 ? 3 : 4;
    auto buf_of = [](int i) constexpr {
      constexpr int b[8] = {2, 0, 1, 0, 1, 2, 0, 1};
      return FM == 8 ? b[i] : i;
    };
    auto read_at = [](int i) constexpr {
      constexpr int at8[8] = {-1, -1, 1, 2, 3, 4, 4, 5}, at4[4] = {-1, -1, 1, 1};
      return FM == 8 ? at8[i] : at4[i % 4];
    };
    typedef std::integral_constant<int, 0> Zero;
    auto row_of = [](int q) constexpr { return q < Q0 ? q / FN : FM - 2 + (q - Q0) % 2; };
    auto col_of = [](int q) constexpr { return q < Q0 ? q % FN : (q - Q0) / 2; };
    // the loads of a part: in the second, A's odd ones
    auto second = [](int l) constexpr { return l < LA && l % 2 == 1; };
    auto load_part = [&](int k, int slot, int sslot, bool two) __attribute__((always_inline)) {
#pragma unroll
      for (int l = 0; l < L; ++l)
        if (second(l) == two) load_one(k, slot, l);
      if (!two) load_scales(k, sslot);
    };
    // wait for the oldest part in flight, and the barrier
    auto publish = [&](int k, int slot, bool two) __attribute__((always_inline)) {
      if (k == a.k_steps - 1 && (a.kbytes & 15) != 0) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int l = 0; l < L; ++l)
          if (second(l) == two) trim_one(k, slot, l);
      }
      ring_wait_barrier<kParts>();
    };
    load_part(step_of(0), 0, 0, false);
    load_part(step_of(0), 0, 0, true);
    load_part(step_of(1), 1, 1, false);
    publish(step_of(0), 0, false);
    load_part(step_of(1), 1, 1, true);
    if (idle) {
      for (int X = 0; X < rounds; ++X) {
        const int slot = X & 1, k_two = step_of(X + 2);
        publish(step_of(X), slot, true);
        load_part(k_two, slot, (X + 2) % 3, false);
        publish(step_of(X + 1), slot ^ 1, false);
        load_part(k_two, slot, 0, true);
      }
    }
    Frag fb[FN], fa[NBUF];
    f32x4 part[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) part[p] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    float sc[4] = {};
    float sb = 0.0f;
    auto scale_b = [&](int k) __attribute__((always_inline)) {
      if constexpr (kScaled)
        sb = k < a.k_steps ? sb_s[(wn * Cfg::kWaveN / kScaleBlock) * kMaxKSteps + k] : 0.0f;
    };
    auto read_row = [&](int slot, int sslot, auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      fa[buf_of(i)] = read_frag(pa + slot * Cfg::kStageBytes, i);
      if constexpr (kScaled) sc[i % 4] = sa_s[sslot * SA + wm * Cfg::kWaveM + i * 16 + lrow] * sb;
    };
    scale_b(step_of(0));
    read_row(0, 0, Zero{});
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = read_frag(pb, j);
    read_row(0, 0, std::integral_constant<int, 1>{});
    int ss = 0;  // X % 3: the slot of step X's row scales, read to the step's end
    for (int X = idle ? rounds : 0; X < rounds; ++X) {
      const int slot = X & 1, next = slot ^ 1;
      const int ss1 = ss == 2 ? 0 : ss + 1, ss2 = ss == 0 ? 2 : ss - 1;
      const int k_now = step_of(X);
      const int k_next = step_of(X + 1);
      const int k_two = step_of(X + 2);
      constexpr_for<NQ>([&](auto qc) __attribute__((always_inline)) {
        constexpr int q = decltype(qc)::value;
        constexpr int i = row_of(q), j = col_of(q);
        if constexpr (q == QP) publish(k_now, slot, true);
        if constexpr (q == Q0) {
          publish(k_next, next, false);
          scale_b(k_next);
        }
        if constexpr (kScaled)
          part[q % 4] = St::mfma(fb[j], fa[buf_of(i)], (f32x4){0.0f, 0.0f, 0.0f, 0.0f});
        else
          acc[i][j] = St::mfma(fb[j], fa[buf_of(i)], acc[i][j]);
        if constexpr (q < Q0 && j == 0)
          constexpr_for<FM>([&](auto rc) __attribute__((always_inline)) {
            if constexpr (read_at(decltype(rc)::value) == i) read_row(slot, ss, rc);
          });
        // loads: part 1 of step X + 2 from P2 to P1, part 2 after P1
        constexpr int L1 = L - LA / 2, L2 = LA / 2;
        constexpr_for<L>([&](auto lc) __attribute__((always_inline)) {
          constexpr int l = decltype(lc)::value;
          constexpr int nth = l < LA ? l / 2 : l - LA / 2;  // place in its part
          if constexpr (second(l)) {
            if constexpr (q == Q0 + nth * (NQ - Q0) / L2) load_one(k_two, slot, l);
          } else {
            if constexpr (q == QP + nth * (Q0 - QP) / L1) load_one(k_two, slot, l);
          }
        });
        if constexpr (q == Q0 - 1) load_scales(k_two, ss2);
        if constexpr (q >= Q0) {
          // the next step's first rows and B fragments
          if constexpr (q == Q0) read_row(next, ss1, Zero{});
          if constexpr ((q - Q0) % 2 == 1) fb[j] = read_frag(pb + next * Cfg::kStageBytes, j);
          if constexpr (q == NQ - 1) read_row(next, ss1, std::integral_constant<int, 1>{});
        }
        if constexpr (kScaled) {
          constexpr int d = q < 3 ? q - 3 + NQ : q - 3;  // MFMA whose sums are added now
          constexpr int di = row_of(d), dj = col_of(d);
          // (before the first step there is nothing to add: part is zero)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[di][dj][r] = __builtin_fmaf(part[d % 4][r], sc[di % 4], acc[di][dj][r]);
          // (keeps the additions here: left free, they gather at the step's
          // end, where their partial sums do not fit the registers)
          asm volatile("" : "+v"(acc[di][dj]));
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      ss = ss1;
    }
    if constexpr (kScaled) {
      constexpr_for<3>([&](auto dc) __attribute__((always_inline)) {
        constexpr int d = NQ - 3 + decltype(dc)::value;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[row_of(d)][col_of(d)][r] =
              __builtin_fmaf(part[d % 4][r], sc[row_of(d) % 4], acc[row_of(d)][col_of(d)][r]);
      });
    }
  } else {
    int at_slot = 0, to_slot = S - 1;  // ring slots of steps X and X + S - 1
    for (int X = 0; X < rounds; ++X) {
      const int k = step_of(X), k_ahead = step_of(X + S - 1);
      if (k == a.k_steps - 1 && (a.kbytes & 15) != 0) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int i = 0; i < L; ++i) trim_one(k, at_slot, i);
      }
      ring_wait_barrier<kInFlight>();
      if (idle) {
#pragma unroll
        for (int l = 0; l < L; ++l) load_one(k_ahead, to_slot, l);
        load_scales(k_ahead, to_slot);
        at_slot = at_slot + 1 == S ? 0 : at_slot + 1;
        to_slot = to_slot + 1 == S ? 0 : to_slot + 1;
        continue;
      }
      const uint32_t slot = at_slot * Cfg::kStageBytes;
      Frag fb[FN], fa[2];
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = read_frag(pb + slot, j);
      fa[0] = read_frag(pa + slot, 0);
      float sb = 0.0f;
      if constexpr (kScaled)
        sb = k < a.k_steps ? sb_s[(wn * Cfg::kWaveN / kScaleBlock) * kMaxKSteps + k] : 0.0f;
      f32x4 part[2][FN];
      float sc[2];
#pragma unroll
      for (int i = 0; i < FM + 1; ++i) {
        if (i < FM) {
          if constexpr (kScaled)
            sc[i & 1] = sa_s[at_slot * SA + wm * Cfg::kWaveM + i * 16 + lrow] * sb;
          if (i + 1 < FM) fa[(i + 1) & 1] = read_frag(pa + slot, i + 1);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            if constexpr (kScaled)
              part[i & 1][j] =
                  St::mfma(fb[j], fa[i & 1], (f32x4){0.0f, 0.0f, 0.0f, 0.0f});
            else
              acc[i][j] = St::mfma(fb[j], fa[i & 1], acc[i][j]);
          }
#pragma unroll
          for (int l = 0; l < L; ++l)
            if (l * FM / L == i) load_one(k_ahead, to_slot, l);
          if (i == 0) load_scales(k_ahead, to_slot);
        }
        if constexpr (kScaled) {
          if (i > 0) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[i - 1][j][r] =
                    __builtin_fmaf(part[(i - 1) & 1][j][r], sc[(i - 1) & 1], acc[i - 1][j][r]);
          }
        }
        // (without it the scheduler reads every fragment first, and spills)
        __builtin_amdgcn_sched_barrier(0);
      }
      at_slot = at_slot + 1 == S ? 0 : at_slot + 1;
      to_slot = to_slot + 1 == S ? 0 : to_slot + 1;
    }
  }

  KernelArgs c{};
  c.C = a.C;
  c.ldc = a.ldc;
  c.M = tile.end;
  c.N = a.N;
  if constexpr (WK > 1) {
    // The groups' sums meet in LDS, added in the order of the groups by the
    // first one, which stores C.
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    static_assert(T * FM * FN * 16 <= Cfg::kLdsBytes, "a group's sums fit its ring");
    lds_f32x4* const mine = (lds_f32x4*)smem + (wave * FM * FN) * 64 + lane;
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < FM * FN; ++i) mine[i * 64] = acc[i / FN][i % FN];
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kg > 0) return;
#pragma unroll
    for (int g = 1; g < WK; ++g)
#pragma unroll
      for (int i = 0; i < FM * FN; ++i)
        acc[i / FN][i % FN] += mine[g * (Cfg::kLdsBytes / 16) + i * 64];
    // (each wave stages C in its own part of the first group's ring: no
    // barrier, which the other groups' waves would not reach)
    finish_tile<Cfg, OUT, false, Cfg::kLdsBytes, false>(c, smem, wave, m0, n0, acc,
                                                        m0 + wm * Cfg::kWaveM,
                                                        n0 + wn * Cfg::kWaveN, lane, 0);
  } else {
    finish_tile<Cfg, OUT, false>(c, smem, wave, m0, n0, acc, m0 + wm * Cfg::kWaveM,
                                 n0 + wn * Cfg::kWaveN, lane, 0);
  }
}

// ------------------------------------------------------------ row kernel

// Buffer resource over num_bytes bytes from base, for the load builtins.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, uint32_t num_bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)num_bytes, 0x00020000);
}

// For single tokens over few columns, where a staged tile has too few
// workgroups or K-steps to fill its ring: 1 x 4096 x 4096 6.5 us against
// 8.1 us for 32 x 32 staged tiles (at 1 x 8192 x 8192 those are level or
// ahead).
//
// 16 FM rows x 16 FN columns per workgroup, its W waves taking every W-th
// K-step.  Operands go from global memory into registers in the MFMA's own
// layout (a lane holds two 16-byte chunks of its row), U steps ahead; the
// waves' sums meet in LDS and are added in the order of the waves.
template <int FM, int FN, int W, int U, int OP, int OUT>
__global__ __attribute__((amdgpu_flat_work_group_size(W * 64, W * 64))) void
block_row_kernel(BlockArgs a) {
  constexpr bool kScaled = OP == kOpE4m3;
  constexpr int BM = 16 * FM, BN = 16 * FN;
  static_assert(kScaleBlock % BN == 0, "the tile's columns share one scale");
  __shared__ f32x4 sums[W][FM * FN][64];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lrow = lane & 15, lchunk = (lane >> 4) * 16;

  const int rt = blockIdx.x / a.tiles_n;
  const int n0 = (blockIdx.x - rt * a.tiles_n) * BN;
  RowTile tile;
  if (a.offsets) {
    if (!find_row_tile(a, BM, rt, lane, tile)) return;
  } else {
    tile = RowTile{0, rt * BM, a.M};
  }
  const int m0 = tile.begin;
  const bool gather = a.rows != nullptr;
  const int rows_a = min(BM, tile.end - m0), rows_b = min(BN, a.N - n0);
  const __amdgpu_buffer_rsrc_t rsrc_a =
      gather ? buffer_of(a.A, (uint32_t)((int64_t)a.a_rows * a.lda))
             : buffer_of(a.A + (int64_t)m0 * a.lda, (uint32_t)(rows_a * a.lda));
  const __amdgpu_buffer_rsrc_t rsrc_b = buffer_of(a.B + tile.expert * a.stride_b + (int64_t)n0 * a.ldb,
                                 (uint32_t)(rows_b * a.ldb));
  uint32_t va[FM], vb[FN], vs[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = i * 16 + lrow;
    const int src = row < rows_a ? (gather ? source_row(a, m0 + row) : row) : -1;
    va[i] = src >= 0 ? (uint32_t)(src * (int)a.lda + lchunk) : kOOB;
    vs[i] = src >= 0 ? (uint32_t)(gather ? src : m0 + src) * 4 : kOOB;
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int row = j * 16 + lrow;
    vb[j] = row < rows_b ? (uint32_t)(row * (int)a.ldb + lchunk) : kOOB;
  }
  const float* sb_row = a.SB + tile.expert * a.stride_sb + (int64_t)(n0 / kScaleBlock) * a.ldsb;

  const int rot =
      a.k_steps > 0 ? __builtin_amdgcn_readfirstlane((n0 / BN) * a.k_rot % a.k_steps) : 0;
  auto step_of = [&](int X) __attribute__((always_inline)) {
    return X + rot >= a.k_steps ? X + rot - a.k_steps : X + rot;
  };
  struct Stage {
    u32x4 fa[FM][2], fb[FN][2];
    float sa[FM], sb;
  };
  Stage st[U];
  auto load = [&](Stage& s, int X) __attribute__((always_inline)) {
    // bytes left of the row at this lane's two chunks; past K reads zero
    const int k0 = X * kStepBytes;
    const bool in0 = k0 + lchunk < a.kbytes, in1 = k0 + 64 + lchunk < a.kbytes;
    auto get = [&](__amdgpu_buffer_rsrc_t rs, uint32_t v, bool in, int off, auto nt)
        __attribute__((always_inline)) {
      return __builtin_amdgcn_raw_buffer_load_b128(rs, in ? v + off : kOOB, k0,
                                                   decltype(nt)::value ? 2 : 0);
    };
    const std::true_type nt{};    // B is read by this workgroup alone
    const std::false_type keep{};
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      s.fb[j][0] = get(rsrc_b, vb[j], in0, 0, nt);
      s.fb[j][1] = get(rsrc_b, vb[j], in1, 64, nt);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      s.fa[i][0] = get(rsrc_a, va[i], in0, 0, keep);
      s.fa[i][1] = get(rsrc_a, va[i], in1, 64, keep);
    }
    if constexpr (kScaled) {
      const __amdgpu_buffer_rsrc_t rs = buffer_of(a.SA + X * a.ldsa, (uint32_t)a.a_rows * 4);
#pragma unroll
      for (int i = 0; i < FM; ++i)
        s.sa[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, vs[i], 0, 0));
      s.sb = sb_row[X];
    }
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  // Zero the bytes past K of a chunk that straddles it.
  auto trim = [&](u32x4& v, int keep) __attribute__((always_inline)) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int left = keep - 4 * w;
      v[w] &= left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
    }
  };
  auto multiply = [&](Stage& s, int X) __attribute__((always_inline)) {
    if (X == a.k_steps - 1 && (a.kbytes & 15) != 0) {
      const int keep = a.kbytes - X * kStepBytes - lchunk;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        trim(s.fa[i][0], keep);
        trim(s.fa[i][1], keep - 64);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        trim(s.fb[j][0], keep);
        trim(s.fb[j][1], keep - 64);
      }
    }
    using St = Step<OP, OUT>;
    typename St::Frag fb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = St::make(s.fb[j][0], s.fb[j][1]);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const typename St::Frag fa = St::make(s.fa[i][0], s.fa[i][1]);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (kScaled) {
          const f32x4 p = St::mfma(fb[j], fa, (f32x4){0.0f, 0.0f, 0.0f, 0.0f});
          const float sc = s.sa[i] * s.sb;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], sc, acc[i][j][r]);
        } else {
          acc[i][j] = St::mfma(fb[j], fa, acc[i][j]);
        }
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (wave + u * W < a.k_steps) load(st[u], step_of(wave + u * W));
  for (int X = wave; X < a.k_steps; X += U * W) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int Y = X + u * W;
      if (Y < a.k_steps) {
        multiply(st[u], step_of(Y));
        if (Y + U * W < a.k_steps) load(st[u], step_of(Y + U * W));
      }
    }
  }

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) sums[wave][i * FN + j][lane] = acc[i][j];
  __syncthreads();
  for (int q = tid; q < FM * FN * 64; q += W * 64) {
    const int f = q >> 6, l = q & 63;
    f32x4 v = sums[0][f][l];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[w][f][l];
    const int row = (f / FN) * 16 + (l & 15);
    if (row < rows_a)
      store_quad<OUT>(a.C, a.ldc, v, m0 + row, n0 + (f % FN) * 16 + 4 * (l >> 4), a.N);
  }
}

}  // namespace gemm
