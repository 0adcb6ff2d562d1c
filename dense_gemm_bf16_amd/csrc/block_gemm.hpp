// Products over e4m3 operands with a scale for each block of 128, and the
// experts' products (rows sorted by expert) over e4m3, bf16 and fp16:
//
//   dense     C[m,n] = sum_b SA[b,m] SB[n/128,b] sum_{k in block b} A[m,k] B[n,k]
//   experts   the same for every row p of expert e's range
//             [offsets[e], offsets[e+1]), with A's row rows[p] (or p) and
//             expert e's B and SB; bf16 and fp16 operands carry no scales
//   integer   C[m,n] = SA[m] SB[n] sum_k A[m,k] B[n,k] over 8-bit integers
//   gated     H[m,f] = act(G[m,f]) U[m,f] with [G | U] a product over bf16,
//             fp16 or 8-bit integers, B's rows f for G and F + f for U
//   gradients C = A . B with B's rows along K, and C = A^T . B with the rows of
//             both along K, over bf16 and fp16: those of a product's operands
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
// per MFMA of 32 cycles, issued while the next MFMA runs.  Sums of 8-bit
// integers stay integers (in the same registers) over all of K and meet their
// scales once, after the last step.
//
// Measured (MI355X): 8192 x 10240 x 8192 bf16 out 571-608 us, 2260-2410
// TFLOP/s, the matrix cores 58 % busy; 1 x 8192 x 8192 12-13 us (memory); 64,
// 128, 256 rows by 8192 x 8192 15, 20.5, 29 us (the L2: tile traffic of 13-15
// TB/s when the lines come in from the fabric, whatever the ring's depth).
// Rows that do not start on 128-byte lines cost 10-40 % where loads bound it.
// Integers, without the FMAs of every step: 8192 x 10240 x 8192 501-571 us by
// the clock (2400-2740 TOP/s, matrix cores 74 % busy), 128, 256 rows by 8192 x
// 8192 17.8, 23.9 us.  Gated bf16, 8192 x 14336 x 4096: 1338-1368 us (1410-1440
// TFLOP/s, 75 % busy, at the power limit).  Both gradients of it: 2797-2950 us
// (1300-1380 TFLOP/s, 71 % busy, likewise).
#pragma once

#include "gemm_kernel.hpp"

namespace gemm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kStepBytes = 128;     // bytes of a row in one K-step
constexpr int kMaxKSteps = 1024;    // K-steps whose B scales are held in LDS
constexpr int kScaleBlock = 128;    // rows of B (and columns of C) of one scale

// Operand types.
enum : int { kOpE4m3 = 0, kOpBf16 = 1, kOpF16 = 2, kOpI8 = 3 };

// What becomes of the sums: C, or (kGated) act(g) * u of paired columns.
enum : int { kPlain = 0, kGated = 1 };

// How the operands lie: rows of K elements (kNT); B's rows along K (kNN: B(k,n)
// = B[k*ldb + n]); those of both (kTN: A(k,m) = A[k*lda + m] too).
enum : int { kNT = 0, kNN = 1, kTN = 2 };

struct BlockArgs {
  const uint8_t* A;
  const uint8_t* B;
  void* C;
  const float* SA;         // SA[b * ldsa + row of A]; integers: SA[row of A]
  const float* SB;         // SB[(n / 128) * ldsb + b]; integers: SB[n]
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
  // gated: N counts the columns of H (in C), and
  int64_t up_b;       // bytes from B's row f (gate) to its row F + f (up)
  int64_t up_sb;      // floats from SB's entry f to its entry F + f
  uint8_t* kept;      // where g and u go as well (see store_kept), or null
  int64_t ld_kept;    // bytes from row to row of it
  int64_t kept_f;     // columns of one of its planes
  int32_t kept_first; // the column there of this launch's first one
  int32_t geglu;      // act: 1: gelu (tanh form), 0: silu
  // kNN and kTN: K in k_steps / seg_steps parts of equal length (kbytes counts
  // one part's), of which the next starts seg_a and seg_b bytes further on;
  int32_t seg_steps;
  int64_t seg_a, seg_b;
  // rows of C in two halves of M rows (or one: half_tiles = row_tiles), the
  // second from half_a bytes on in A and from row M on in C;
  int32_t half_tiles;
  int64_t half_a;
  // and the K-steps split over workgroups, whose sums go to parts of C that
  // lie part_stride elements apart
  int32_t splits, split_steps;
  int64_t part_stride;
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
    } else if constexpr (OP == kOpI8) {
      // exact 32-bit integer sums, held as their bits
      i32x4 d = __builtin_bit_cast(i32x4, c);
#pragma unroll
      for (int h = 0; h < kRegs; ++h)
        d = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b.v[h]),
                                                  __builtin_bit_cast(i32x4, a.v[h]), d, 0, 0, 0);
      return __builtin_bit_cast(f32x4, d);
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

// The sum of two partial sums (of integers: of the integers they hold).
template <int OP>
__device__ __forceinline__ f32x4 add_sums(f32x4 x, f32x4 y) {
  if constexpr (OP == kOpI8)
    return __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, x) + __builtin_bit_cast(i32x4, y));
  else
    return x + y;
}

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

// ---------------------------------------------------------------- epilogue

// SB of columns n .. n+3 (0 past the last one).
__device__ __forceinline__ f32x4 column_scales(const float* sb, int n, int N) {
  f32x4 v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = n + r < N ? sb[n + r] : 0.0f;
  return v;
}

// Integer sums to (fp32(sum) * SA[m]) * SB[n], three roundings; other types'
// are left.  acc[i][j]: row i * 16 + lane % 16 from m_base on, columns j * 16
// + 4 (lane / 16) .. + 3 from n_base on.
template <int OP, int FM, int FN>
__device__ __forceinline__ void scale_sums(const BlockArgs& a, f32x4 (&acc)[FM][FN], int m_end,
                                           int m_base, int n_base, int lane) {
  if constexpr (OP == kOpI8) {
    f32x4 sb[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = column_scales(a.SB, n_base + j * 16 + 4 * (lane >> 4), a.N);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m_base + i * 16 + (lane & 15);
      const float sa = m < m_end ? a.SA[m] : 0.0f;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const i32x4 sum = __builtin_bit_cast(i32x4, acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = (float)sum[r] * sa * sb[j][r];
      }
    }
  }
}

// act(g) * u, with act(g) = g sigmoid(z): z = g for silu; for gelu in its tanh
// form, g (1 + tanh(y)) / 2 = g sigmoid(2 y) with y = sqrt(2 / pi) (g +
// 0.044715 g^3).  For a 16-bit H, sigmoid(z) = 1 / (1 + 2^(-z log2 e)) by the
// vector unit's 2^x and 1/x (1 ulp each); the exponent's roundings (gelu's z has
// five more) are up to 7 |z| 2^-24 relative, 2^-14 where the result nears fp32's
// smallest, against the 2^-9 or 2^-12 of H's own rounding.  An fp32 H shows
// them, so there the exponent is carried past fp32 (silu's product's rounding
// error is made up for, gelu's z is taken in fp64: in fp32 its own roundings
// left results up to 155 2^-24 off) and the power is of -|z|, which neither
// overflows nor cancels: less than 8 2^-24 off for every z (results below
// 2^-120 may be zero).  Six and fourteen operations for silu: with the longer
// form everywhere the activation would take 5 % of a bf16 product's time and 9 %
// of an integer one's at 8192 x 14336 x 4096.  (fp32 H of that size: silu 818-822
// us, gelu 840-842, 834-840 with its z in fp32.)
constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.69314718f;

__device__ __forceinline__ float gate_argument(float g, bool geglu) {
  const float y = g * __builtin_fmaf(0.0713548163f, g * g, 1.59576912f);
  return geglu ? y : g;
}

// exp(-|z|) of the gate's z (|z| is cut at 200, past which it is zero).
__device__ __forceinline__ float exp_of_minus(float g, bool geglu) {
  float t, low;  // -|z| log2 e
  if (geglu) {
    const double d = (double)g;
    const double z = d * __builtin_fma(0.07135481627260025, d * d, 1.5957691216057308);
    const double y = __builtin_fmin(__builtin_fabs(z), 200.0) * -1.4426950408889634;
    t = (float)y;
    low = (float)(y - (double)t);
  } else {
    const float x = fminf(fabsf(g), 200.0f);
    t = x * -kLog2e;
    low = __builtin_fmaf(x, -kLog2e, -t) - x * kLog2eLow;
  }
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, low * kLn2, e);
}

template <int OUT>
__device__ __forceinline__ float gate(float g, float u, bool geglu) {
  if constexpr (OUT == kStoreF32) {
    const float e = exp_of_minus(g, geglu);
    const float r = 1.0f / (1.0f + e);
    return g * (g >= 0.0f ? r : e * r) * u;
  } else {
    const float z = gate_argument(g, geglu);
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -kLog2e)) * u;
  }
}

// Where a wave's sums lie in its tile.  kQuads: quad (i, j) is row i * 16 + lane
// % 16, columns (wn * FN + j) * 16 + 4 (lane / 16) .. + 3.  kHalves (of gated
// tiles whose waves hold an odd number of fragments, see finish_gated): row (2 i
// + lane / 32) * 16 + lane % 16, columns (wn * FN + j) * 8 + 4 (lane / 16 % 2) ..
// + 3.
enum : int { kQuads = 0, kHalves = 1 };
template <int PLACE, int FN>
struct Place {
  __device__ static int row(int i, int lane) {
    return (PLACE == kHalves ? 2 * i + (lane >> 5) : i) * 16 + (lane & 15);
  }
  __device__ static int quad(int wn, int j, int lane) {  // column / 4
    return PLACE == kHalves ? (wn * FN + j) * 2 + (lane >> 4 & 1) : (wn * FN + j) * 4 + (lane >> 4);
  }
};

// Byte offset of 16-byte piece c of row r, rows of PIECES pieces staged in LDS:
// XORed with the bits of the row that tell apart rows of one 256-byte stretch of
// banks.
template <int PIECES>
__device__ __forceinline__ uint32_t staged_at(int r, int c) {
  constexpr int kGroup = (PIECES & -PIECES) < 16 ? PIECES & -PIECES : 16;
  constexpr int kShift = kGroup == 16 ? 0 : kGroup == 8 ? 1 : kGroup == 4 ? 2 : kGroup == 2 ? 3 : 4;
  return (uint32_t)((r * PIECES + (c ^ ((r >> kShift) & (kGroup - 1)))) << 4);
}

// A workgroup's BM x COLS values, staged in LDS by rows and stored in whole
// 16-byte pieces, COLS * size bytes of a row by consecutive lanes.  Waves with
// `mine` write the quads v[i][j] of their WAVE_M rows (see Place), in PASSES of
// FM / PASSES of them where the rows do not fit the region at once.  Every wave
// of the workgroup calls it; the LDS region is free when it is called and in use
// when it returns.
template <int BM, int WAVE_M, int COLS, int THREADS, int OUT, int PLACE, int PASSES, int FM, int FN>
__device__ __forceinline__ void store_staged(lds_u8* region, const f32x4 (&v)[FM][FN], bool mine,
                                             int wm, int wn, int lane, void* out, int64_t ld,
                                             int m0, int m_end, int n0, int N) {
  constexpr int kE = OUT == kStoreF32 ? 4 : 2, kPer = 16 / kE, kPieces = COLS / kPer;
  constexpr int kRows = BM / PASSES, kWaveRows = WAVE_M / PASSES, kQ = FM / PASSES;
  static_assert(FM % PASSES == 0, "whole passes");
  using At = Place<PLACE, FN>;
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) {
    if (pass > 0) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (mine) {
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const int r = wm * kWaveRows + At::row(i, lane);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int q = At::quad(wn, j, lane);
          const f32x4& x = v[pass * kQ + i][j];
          if constexpr (kE == 4)
            *(__attribute__((address_space(3))) f32x4*)(region + staged_at<kPieces>(r, q)) = x;
          else
            *(__attribute__((address_space(3))) u32x2*)(region + staged_at<kPieces>(r, q >> 1) +
                                                        ((q & 1) << 3)) = pack_quad<OUT>(x);
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int p0 = 0; p0 < kRows * kPieces; p0 += THREADS) {
      const int p = p0 + (int)threadIdx.x;
      if (kRows * kPieces % THREADS != 0 && p >= kRows * kPieces) break;
      const int r = p / kPieces, c = p % kPieces, col = n0 + c * kPer;
      const int m = m0 + r / kWaveRows * WAVE_M + pass * kWaveRows + r % kWaveRows;
      const u32x4 x = *(const lds_u32x4*)(region + staged_at<kPieces>(r, c));
      if (m >= m_end || col >= N) continue;
      uint8_t* dst = (uint8_t*)out + ((int64_t)m * ld + col) * kE;
      if (col + kPer <= N) {
        __builtin_nontemporal_store(x, (u32x4*)dst);
        continue;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (col + e >= N) break;
        if constexpr (kE == 4)
          ((uint32_t*)dst)[e] = x[e];
        else
          ((uint16_t*)dst)[e] = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

// g and u for the backward pass, 24 bits each: fp32 without its last eight
// (rounded).  Kept in H's type they would double the error of the gradients
// beside that of dg's and du's own rounding (bf16: 0.0030 of dW in norm, of
// which 0.0017 is its own rounding, against 0.0024); kept in fp32 they would
// take a third more memory and time.  A row of `kept` holds four planes of
// kept_f columns, F rounded up to 16: the upper halves of g, those of u (2
// bytes each), the third bytes of g and of u.
__device__ __forceinline__ uint32_t kept_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) + 0x80u;  // (an infinity or quiet NaN stays one)
}
__device__ __forceinline__ u32x2 kept_high(const f32x4& v) {
  return (u32x2){(kept_bits(v[0]) >> 16) | (kept_bits(v[1]) & 0xFFFF0000u),
                 (kept_bits(v[2]) >> 16) | (kept_bits(v[3]) & 0xFFFF0000u)};
}
__device__ __forceinline__ uint32_t kept_third(const f32x4& v) {
  return (kept_bits(v[0]) >> 8 & 0xFFu) | (kept_bits(v[1]) & 0xFF00u) |
         (kept_bits(v[2]) << 8 & 0xFF0000u) | (kept_bits(v[3]) << 16 & 0xFF000000u);
}
__device__ __forceinline__ float kept_value(uint32_t high, uint32_t third) {
  return __builtin_bit_cast(float, high << 16 | third << 8);
}

// A workgroup's g (up 0) or u (up 1) into `kept`, staged as store_staged
// stages H.  The planes' rows are padded, so pieces are stored whole.
template <int BM, int COLS, int THREADS, int PLACE, int FM, int FN>
__device__ __forceinline__ void store_kept(lds_u8* region, const BlockArgs& a,
                                           const f32x4 (&v)[FM][FN], int up, bool mine, int wm,
                                           int wn, int lane, int m0, int m_end, int f0) {
  constexpr int kWaveM = (PLACE == kHalves ? 32 : 16) * FM;
  using At = Place<PLACE, FN>;
  const std::integral_constant<int, COLS / 8> high{};
  const std::integral_constant<int, COLS / 16> third{};
  lds_u8* const region3 = region + BM * COLS * 2;
  if (mine) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = wm * kWaveM + At::row(i, lane);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int q = At::quad(wn, j, lane);
        *(__attribute__((address_space(3))) u32x2*)(region + staged_at<COLS / 8>(r, q >> 1) +
                                                    ((q & 1) << 3)) = kept_high(v[i][j]);
        *(__attribute__((address_space(3))) uint32_t*)(region3 + staged_at<COLS / 16>(r, q >> 2) +
                                                       ((q & 3) << 2)) = kept_third(v[i][j]);
      }
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  auto rows = [&](auto pieces, const lds_u8* from, int per, int64_t plane, int bytes)
      __attribute__((always_inline)) {
    constexpr int kPieces = decltype(pieces)::value;
#pragma unroll
    for (int p0 = 0; p0 < BM * kPieces; p0 += THREADS) {
      const int p = p0 + (int)threadIdx.x;
      if (BM * kPieces % THREADS != 0 && p >= BM * kPieces) break;
      const int r = p / kPieces, c = p % kPieces, col = f0 + c * per;
      const u32x4 x = *(const lds_u32x4*)(from + staged_at<kPieces>(r, c));
      if (m0 + r < m_end && col < a.N)
        __builtin_nontemporal_store(
            x, (u32x4*)(a.kept + (int64_t)(m0 + r) * a.ld_kept + plane +
                        (int64_t)(a.kept_first + col) * bytes));
    }
  };
  rows(high, region, 8, up * 2 * a.kept_f, 2);
  rows(third, region3, 16, (4 + up) * a.kept_f, 1);
}

// H = act(g) * u (rounded once, from the unrounded sums) and, where asked
// for, g and u to `kept`.  Waves with `mine` hold the sums: with an even number
// of fragments of B, g in the even ones and u in the odd ones; else g in the
// first eight rows of each and u in the other eight, of which two fragments'
// halves are exchanged, so that a lane again holds both of an element.
template <typename Cfg, int OP, int OUT, int THREADS>
__device__ __forceinline__ void finish_gated(const BlockArgs& a, lds_u8* region,
                                             f32x4 (&acc)[Cfg::kFragM][Cfg::kFragN], int m0,
                                             int m_end, int f0, int wm, int wn, int lane,
                                             bool mine) {
  constexpr int PLACE = Cfg::kFragN % 2 == 0 ? kQuads : kHalves;
  constexpr int FM = PLACE == kHalves ? Cfg::kFragM / 2 : Cfg::kFragM;
  constexpr int FN = PLACE == kHalves ? Cfg::kFragN : Cfg::kFragN / 2;
  constexpr int BM = Cfg::kBM, COLS = Cfg::kBN / 2;
  using At = Place<PLACE, FN>;
  f32x4 g[FM][FN], u[FM][FN], h[FM][FN];
  if (mine) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (PLACE == kHalves) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // (copies: the compiler casts the bits of a vector's first element
            // whichever one is named)
            const float first = acc[2 * i][j][r], second = acc[2 * i + 1][j][r];
            const u32x2 x = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, first),
                                                        __builtin_bit_cast(uint32_t, second),
                                                        false, false));
            const uint32_t bits_g = x[0], bits_u = x[1];
            g[i][j][r] = __builtin_bit_cast(float, bits_g);
            u[i][j][r] = __builtin_bit_cast(float, bits_u);
          }
        } else {
          g[i][j] = acc[i][2 * j];
          u[i][j] = acc[i][2 * j + 1];
        }
      }
    if constexpr (OP == kOpI8) {
      f32x4 sg[FN], su[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int f = f0 + At::quad(wn, j, lane) * 4;
        sg[j] = column_scales(a.SB, f, a.N);
        su[j] = column_scales(a.SB + a.up_sb, f, a.N);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int m = m0 + wm * Cfg::kWaveM + At::row(i, lane);
        const float sa = m < m_end ? a.SA[m] : 0.0f;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const i32x4 ig = __builtin_bit_cast(i32x4, g[i][j]);
          const i32x4 iu = __builtin_bit_cast(i32x4, u[i][j]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            g[i][j][r] = (float)ig[r] * sa * sg[j][r];
            u[i][j][r] = (float)iu[r] * sa * su[j][r];
          }
        }
      }
    }
    // (a loop for each activation: a choice in the loop would compute both)
    auto gates = [&](bool geglu) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) h[i][j][r] = gate<OUT>(g[i][j][r], u[i][j][r], geglu);
    };
    if (a.geglu != 0)
      gates(true);
    else
      gates(false);
  }
  // every wave is done with the ring
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  store_staged<BM, Cfg::kWaveM, COLS, THREADS, OUT, PLACE, 1>(region, h, mine, wm, wn, lane, a.C,
                                                              a.ldc, m0, m_end, f0, a.N);
  if constexpr (OP != kOpI8) {
    if (a.kept != nullptr) {
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      store_kept<BM, COLS, THREADS, PLACE>(region, a, g, 0, mine, wm, wn, lane, m0, m_end, f0);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      store_kept<BM, COLS, THREADS, PLACE>(region, a, u, 1, mine, wm, wn, lane, m0, m_end, f0);
    }
  }
}

// ----------------------------------------------------------- tile kernel

// BM x BN tiles, WM x WN waves, a ring of S LDS slots of 128-byte rows
// swizzled as in the direct-to-LDS kernel.  Per K-step X: wait until its
// loads have landed (those of the S - 2 steps after it may be in flight),
// barrier (which also frees the slot of step X - 1), then the wave's MFMAs
// with the loads of step X + S - 1 spread between them.  Every step issues
// the same loads, those past K reading zeros, so the waits count them.
//
// MODE kGated: a tile's BN rows of B are BN / 2 rows of the gate and the BN /
// 2 of the same columns of the up projection, 16 and 16 in turn, so that a
// wave holds g and u of one element of H in the same lane and register and
// the activation costs no exchange (8 and 8 where a wave's fragments of B are
// odd in number: one exchange between half waves then).  NT: B's loads non-temporal, for one row
// of tiles, where no other workgroup reads the same B.
//
// LAYOUT kNN, kTN: an operand whose rows lie along K is staged in pieces of 64
// (K) x 64 (a workgroup of 512) or x 32 (of 256), one load of all threads
// each, so that a load still fills the rows or columns of the tile that it
// does in the other form.  Fragments are transposed on their way out of LDS:
// ds_read_b64_tr_b16 takes 4 (K) x 16 per 16 lanes and gives each lane its
// column's four values, so four reads make the two chunks of a fragment, in
// the same K order as the other form's.  The 32-byte column group that row k
// of a piece holds in place u is u ^ (k / 2 % 2 + 2 (k / 8 % 2)), or u ^ (k /
// 8 % 2) in pieces of 32: the eight rows that half a wave reads then lie in
// eight different 32-byte groups of the 64 banks (no conflicts counted).  Rows
// past K are out of the range of a step's buffer resource and read as zeros.
// Pieces of 32 let two workgroups of 128 x 128 share a CU with two slots each
// (2048 x 2048, 8192 deep: 78 us; one with four slots, in pieces of 64, 106).
typedef const __attribute__((address_space(3))) float lds_f32;

// Sizes of a tile's kernel.
template <int BM, int BN, int WM, int WN, int WK, int S, int OP, int OUT>
struct BlockTile {
  using Cfg = TileCfg<BM, BN, 64, WM, WN, S, 3, 16>;
  static constexpr int kRowsPerLoad = Cfg::kThreads / 8;  // of one load of all threads
  // A widened fragment takes twice the registers, too many for this form,
  // and a load of all threads has to be half a wave row of A
  static constexpr bool kPipe = S == 2 && (Cfg::kFragM == 4 || Cfg::kFragM == 8) &&
                                kRowsPerLoad * 2 == Cfg::kWaveM && !Step<OP, OUT>::kWide;
  static constexpr int kScaleCols = (BN + kScaleBlock - 1) / kScaleBlock;  // across a tile
  static constexpr int kRowScales = BM < 64 ? 64 : BM;                     // of a slot
  static constexpr int kScaleSlots = kPipe ? 3 : S;
  static constexpr int kRingBytes = WK * Cfg::kLdsBytes;
  static constexpr int kRowScaleFloats = OP == kOpE4m3 ? WK * kScaleSlots * kRowScales : 1;
  static constexpr int kColScaleFloats = OP == kOpE4m3 ? kScaleCols * kMaxKSteps : 1;
};

// Workgroup `block`'s tile; ring, sa_lds and sb_lds: BlockTile's LDS.
template <int BM, int BN, int WM, int WN, int WK, int S, int OP, int OUT, int MODE, bool NT,
          int LAYOUT>
__device__ __forceinline__ void block_tile(const BlockArgs& a, int block, lds_u8* ring,
                                           lds_f32* sa_lds, lds_f32* sb_lds) {
  using Tile = BlockTile<BM, BN, WM, WN, WK, S, OP, OUT>;
  using Cfg = typename Tile::Cfg;
  constexpr int T = Cfg::kThreads, W = WM * WN;  // threads and waves of one K group
  constexpr int FM = Cfg::kFragM, FN = Cfg::kFragN;
  constexpr int LA = Cfg::kLoadsA, LB = Cfg::kLoadsB, L = LA + LB;
  constexpr int RPI = Tile::kRowsPerLoad;
  constexpr bool kScaled = OP == kOpE4m3;
  using St = Step<OP, OUT>;
  constexpr bool kPipe = Tile::kPipe;
  constexpr int NB = Tile::kScaleCols, SA = Tile::kRowScales, SS = Tile::kScaleSlots;
  constexpr int kInFlight = (S - 2) * (L + (kScaled ? 1 : 0));
  static_assert(RPI % 16 == 0, "the swizzle repeats every 16 rows");
  static_assert(!kScaled || kScaleBlock % Cfg::kWaveN == 0, "a wave's columns share one scale");
  static_assert(SA / 64 <= W, "one wave loads 64 row scales");
  static_assert(kInFlight < 64, "vmcnt range");

  const int tid = threadIdx.x % T;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = WK > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / T) : 0;
  lds_u8* const smem = ring + kg * Cfg::kLdsBytes;
  const uint32_t smem_addr = (uint32_t)(uintptr_t)smem;
  lds_f32* const sa_s = sa_lds + kg * SS * SA;
  lds_f32* const sb_s = sb_lds;
  const int wm = wave / WN, wn = wave % WN;

  // ---- which tile --------------------------------------------------------
  constexpr bool kGrad = LAYOUT != kNT, kTransA = LAYOUT == kTN, kTransB = kGrad;
  static_assert(!kGrad || (WK == 1 && OP != kOpE4m3 && OP != kOpI8 && MODE == kPlain && !NT),
                "gradients are of 16-bit types");
  constexpr int kPiece = RPI;  // columns of a piece
  static_assert(!kGrad || ((kPiece == 32 || kPiece == 64) && Cfg::kWaveM % kPiece == 0 &&
                           Cfg::kWaveN % kPiece == 0),
                "whole pieces");
  const int row_tiles = a.offsets ? count_row_tiles(a, BM, lane) : a.row_tiles;
  const int units = row_tiles * a.tiles_n;
  if (!kGrad && block >= units) return;  // the grid is an upper bound
  int logical = xcd_remap(block, kGrad ? units * a.splits : units);
  int split = 0;
  if constexpr (kGrad) {
    split = logical / units;
    logical -= split * units;
  }
  const int span = a.group_m * a.tiles_n;
  const int gid = logical / span;
  const int first = gid * a.group_m;
  const int gsz = min(row_tiles - first, a.group_m);
  const int in = logical - gid * span;
  int rt = first + in % gsz;
  int half = 0;
  if constexpr (kGrad) {
    half = rt / a.half_tiles;
    rt -= half * a.half_tiles;
  }
  constexpr bool kPairs = MODE == kGated;
  constexpr int kCols = kPairs ? BN / 2 : BN;  // columns of C
  constexpr bool kEights = kPairs && FN % 2 != 0;  // 8 and 8 rows of B in turn, not 16 and 16
  static_assert(!kPairs || (kEights ? RPI % 16 == 0 && FM % 2 == 0 && WK == 1 : RPI % 32 == 0),
                "whole pairs");
  const int tn = in / gsz, n0 = tn * kCols;
  RowTile tile;
  if (a.offsets) {
    if (!find_row_tile(a, BM, rt, lane, tile)) return;
  } else {
    tile = RowTile{0, rt * BM, a.M};
  }
  const int m0 = tile.begin;
  const int rows_a = min(BM, tile.end - m0);
  const int rows_b = min(kCols, a.N - n0);

  // ---- loads -------------------------------------------------------------
  const bool gather = a.rows != nullptr;
  const uint8_t* const grad_a = a.A + half * a.half_a + (kTransA ? (int64_t)m0 * 2 : 0);
  const uint8_t* const grad_b = a.B + (int64_t)n0 * 2;
  const u32x4 rsrc_a = gather ? make_rsrc(a.A, (uint32_t)((int64_t)a.a_rows * a.lda))
                              : make_rsrc(a.A + (int64_t)m0 * a.lda, (uint32_t)(rows_a * a.lda));
  // (gated: a wave loads 8 rows at a time, all of the gate or all of the up
  // projection)
  const int64_t up = kPairs ? (kEights ? wave & 1 : (wave >> 1) & 1) * a.up_b : 0;
  const u32x4 rsrc_b = make_rsrc(a.B + tile.expert * a.stride_b + up + (int64_t)n0 * a.ldb,
                                 (uint32_t)(rows_b * a.ldb));
  const int r0 = tid / 8;
  const int chunk = (tid & 7) ^ swz<3, 8>(r0);
  uint32_t voff[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int row = (i < LA ? i : i - LA) * RPI + r0;
    if (i < LA ? kTransA : kTransB) {
      // piece i (or i - LA), its row k and the 16 bytes there
      const int k = tid / (kPiece / 8), place = tid % (kPiece / 8);
      const int swap = kPiece == 64 ? ((k >> 1) & 1) << 1 | ((k >> 3) & 1) << 2 : ((k >> 3) & 1) << 1;
      const int col = (i < LA ? i : i - LA) * kPiece + (place ^ swap) * 8;
      const int ld = (int)(i < LA ? a.lda : a.ldb);
      voff[i] = col < (i < LA ? rows_a : rows_b) ? (uint32_t)(k * ld + col * 2) : kOOB;
    } else if (i < LA) {
      const int src = row < rows_a ? (gather ? source_row(a, m0 + row) : row) : -1;
      voff[i] = src >= 0 ? (uint32_t)(src * (int)a.lda + chunk * 16) : kOOB;
    } else {
      const int src = kEights ? row / 16 * 8 + row % 8 : kPairs ? row / 32 * 16 + row % 16 : row;
      voff[i] = src < rows_b ? (uint32_t)(src * (int)a.ldb + chunk * 16) : kOOB;
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
  const int last_step = (kGrad ? a.seg_steps : a.k_steps) - 1;  // (of a part of K)
  const bool past_k = last_step * kStepBytes + chunk * 16 >= a.kbytes;  // in the last step
  const int k_begin = kGrad ? split * a.split_steps : 0;
  const int k_here = kGrad ? min(a.k_steps - k_begin, a.split_steps) : a.k_steps;
  // This group's X-th step of K: X * WK + kg, from the tile's starting point
  // on (k_steps or more: past the last one).
  const int rot = a.k_steps > 0 ? __builtin_amdgcn_readfirstlane(tn * a.k_rot % a.k_steps) : 0;
  auto step_of = [&](int X) __attribute__((always_inline)) {
    if constexpr (kGrad) return X < k_here ? k_begin + X : a.k_steps;
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
    if constexpr (kGrad) {
      const bool second = k >= a.seg_steps;  // (two parts at most)
      const int kk = second ? k - a.seg_steps : k;
      if (i < LA ? kTransA : kTransB) {
        const int64_t ld = i < LA ? a.lda : a.ldb;
        const int left = k < a.k_steps ? min(64, (a.kbytes >> 1) - kk * 64) : 0;
        const uint8_t* base = (i < LA ? grad_a : grad_b) + (int64_t)(kk * 64) * ld +
                              (second ? (i < LA ? a.seg_a : a.seg_b) : 0);
        dma16(make_rsrc(base, (uint32_t)(left * (int)ld)), dst, voff[i], 0u);
      } else {
        const uint32_t v = k >= a.k_steps || (past_k && kk == last_step) ? kOOB : voff[i];
        dma16(rsrc_a, dst, v, (uint32_t)(kk * kStepBytes) + (second ? (uint32_t)a.seg_a : 0u));
      }
      return;
    }
    const uint32_t v = k >= a.k_steps - (past_k ? 1 : 0) ? kOOB : voff[i];
    if (NT && i >= LA)
      dma16<true>(rsrc_b, dst, v, (uint32_t)(k * kStepBytes));
    else
      dma16(i < LA ? rsrc_a : rsrc_b, dst, v, (uint32_t)(k * kStepBytes));
  };
  auto load_scales = [&](int k, int slot) __attribute__((always_inline)) {
    if constexpr (kScaled) {
      const u32x4 rs = make_rsrc(a.SA + k * a.ldsa, k < a.k_steps ? (uint32_t)a.a_rows * 4 : 0u);
      dma4(rs, (uint32_t)(uintptr_t)sa_s + (slot * SA + srow) * 4, voff_s, 0u);
    }
  };
  // Whether step k holds bytes past K that its loads cannot leave out.
  auto trims = [&](int k) __attribute__((always_inline)) {
    if constexpr (kTransA) return false;
    return (k == a.k_steps - 1 || (kGrad && k == last_step)) && (a.kbytes & 15) != 0;
  };
  // Zero the bytes past K of the 16-byte chunk that straddles it, each
  // thread in the chunks it loaded (their loads have landed).
  auto trim_one = [&](int k, int slot, int i) __attribute__((always_inline)) {
    if (i < LA ? kTransA : kTransB) return;  // (whole rows of zeros there)
    if (kGrad && k >= a.seg_steps) k -= a.seg_steps;
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
  // (rows along K: this lane's place in the first 4 x 16 of a piece, and the
  // XOR of its column group)
  constexpr int kPieceRow = kPiece * 2;  // bytes
  const int at_k = ((lane >> 4) * 8 + (lrow >> 2)) * kPieceRow + (lrow & 3) * 8;
  const int group_k = kPiece == 64 ? ((lrow >> 3) & 1) << 5 | ((lane >> 4) & 1) << 6
                                   : ((lane >> 4) & 1) << 5;
  auto read_cols = [&](const lds_u8* base, int f) __attribute__((always_inline)) {
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    constexpr int kGroups = kPiece / 16;
    const lds_u8* p = base + f / kGroups * (64 * kPieceRow) + at_k + (group_k ^ (f % kGroups * 32));
    Frag r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x2 x = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + h * 32 * kPieceRow)));
      const u32x2 y = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + (h * 32 + 4) * kPieceRow)));
      r.v[h] = (u32x4){x[0], x[1], y[0], y[1]};
    }
    return r;
  };
  auto read_frag = [&](const lds_u8* base, int f) __attribute__((always_inline)) {
    const u32x4 lo = *(const lds_u32x4*)(base + f * 16 * kStepBytes + at);
    const u32x4 hi = *(const lds_u32x4*)(base + f * 16 * kStepBytes + (at ^ 64));
    return St::make(lo, hi);
  };
  auto read_a = [&](const lds_u8* base, int f) __attribute__((always_inline)) {
    if constexpr (kTransA) return read_cols(base, f);
    else return read_frag(base, f);
  };
  auto read_b = [&](const lds_u8* base, int f) __attribute__((always_inline)) {
    if constexpr (kTransB) return read_cols(base, f);
    else return read_frag(base, f);
  };

  const int rounds = kGrad ? k_here : (a.k_steps + WK - 1) / WK;
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
      if (trims(k)) {
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
      fa[buf_of(i)] = read_a(pa + slot * Cfg::kStageBytes, i);
      if constexpr (kScaled) sc[i % 4] = sa_s[sslot * SA + wm * Cfg::kWaveM + i * 16 + lrow] * sb;
    };
    scale_b(step_of(0));
    read_row(0, 0, Zero{});
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j] = read_b(pb, j);
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
          if constexpr ((q - Q0) % 2 == 1) fb[j] = read_b(pb + next * Cfg::kStageBytes, j);
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
      if (trims(k)) {
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
      for (int j = 0; j < FN; ++j) fb[j] = read_b(pb + slot, j);
      fa[0] = read_a(pa + slot, 0);
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
          if (i + 1 < FM) fa[(i + 1) & 1] = read_a(pa + slot, i + 1);
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
  if constexpr (kGrad)
    c.C = (uint8_t*)a.C + (half * (int64_t)a.M * a.ldc + split * a.part_stride) *
                              (OUT == kStoreF32 ? 4 : 2);
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
    if constexpr (kPairs) {
      if (kg == 0) {
#pragma unroll
        for (int g = 1; g < WK; ++g)
#pragma unroll
          for (int i = 0; i < FM * FN; ++i)
            acc[i / FN][i % FN] =
                add_sums<OP>(acc[i / FN][i % FN], mine[g * (Cfg::kLdsBytes / 16) + i * 64]);
      }
      finish_gated<Cfg, OP, OUT, T * WK>(a, ring, acc, m0, tile.end, n0, wm, wn, lane,
                                         kg == 0);
      return;
    }
    if (kg > 0) return;
#pragma unroll
    for (int g = 1; g < WK; ++g)
#pragma unroll
      for (int i = 0; i < FM * FN; ++i)
        acc[i / FN][i % FN] =
            add_sums<OP>(acc[i / FN][i % FN], mine[g * (Cfg::kLdsBytes / 16) + i * 64]);
    scale_sums<OP, FM, FN>(a, acc, tile.end, m0 + wm * Cfg::kWaveM, n0 + wn * Cfg::kWaveN, lane);
    // (each wave stages C in its own part of the first group's ring: no
    // barrier, which the other groups' waves would not reach)
    finish_tile<Cfg, OUT, false, Cfg::kLdsBytes, false>(c, smem, wave, m0, n0, acc,
                                                        m0 + wm * Cfg::kWaveM,
                                                        n0 + wn * Cfg::kWaveN, lane, 0);
  } else if constexpr (kPairs) {
    finish_gated<Cfg, OP, OUT, T>(a, smem, acc, m0, tile.end, n0, wm, wn, lane, true);
  } else {
    scale_sums<OP, FM, FN>(a, acc, tile.end, m0 + wm * Cfg::kWaveM, n0 + wn * Cfg::kWaveN, lane);
    if constexpr ((Cfg::kWaveN & (Cfg::kWaveN - 1)) != 0) {
      // (a wave's rows are no power of two: staged by the workgroup)
      constexpr int kPasses = BM * BN * (OUT == kStoreF32 ? 4 : 2) <= Cfg::kLdsBytes ? 1 : 2;
      static_assert(BM * BN * (OUT == kStoreF32 ? 4 : 2) / kPasses <= Cfg::kLdsBytes, "fits the ring");
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      store_staged<BM, Cfg::kWaveM, BN, T, OUT, kQuads, kPasses>(smem, acc, true, wm, wn, lane, a.C,
                                                                 a.ldc, m0, tile.end, n0, a.N);
    } else {
      finish_tile<Cfg, OUT, false>(c, smem, wave, m0, n0, acc, m0 + wm * Cfg::kWaveM,
                                   n0 + wn * Cfg::kWaveN, lane, 0);
    }
  }
}

template <int BM, int BN, int WM, int WN, int WK, int S, int OP, int OUT, int MODE = kPlain,
          bool NT = false>
__global__ __attribute__((amdgpu_flat_work_group_size(WM * WN * WK * 64, WM * WN * WK * 64),
                          amdgpu_waves_per_eu(2))) void
block_tile_kernel(BlockArgs a) {
  using Tile = BlockTile<BM, BN, WM, WN, WK, S, OP, OUT>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[Tile::kRingBytes];
  __shared__ float sa_lds[Tile::kRowScaleFloats];
  __shared__ float sb_lds[Tile::kColScaleFloats];
  block_tile<BM, BN, WM, WN, WK, S, OP, OUT, MODE, NT, kNT>(a, (int)blockIdx.x, (lds_u8*)ring,
                                                            (lds_f32*)sa_lds, (lds_f32*)sb_lds);
}

// Both gradients of a product in one launch, kNN's tiles of `x` (to OUT_X) and
// kTN's of `w` (to OUT_W): each alone would leave CUs idle in its last pass,
// or in its only one.  Workgroups below `first` (a multiple of 8, so that
// each tile stays with its XCD) are x's, or w's where w_first, the others the
// other's; either may have none.  (1000 x 1365 x 520: 28 us for the backward
// pass, 36 in two launches.)
template <int BM, int BN, int WM, int WN, int S, int OP, int OUT_X, int OUT_W>
__global__ __attribute__((amdgpu_flat_work_group_size(WM * WN * 64, WM * WN * 64),
                          amdgpu_waves_per_eu(2))) void
grad_pair_kernel(BlockArgs x, BlockArgs w, int first, int w_first) {
  __shared__ __attribute__((aligned(1024)))
  uint8_t ring[BlockTile<BM, BN, WM, WN, 1, S, OP, OUT_X>::kRingBytes];
  __shared__ float none[1];
  const int block = (int)blockIdx.x < first ? (int)blockIdx.x : (int)blockIdx.x - first;
  if (((int)blockIdx.x < first) == (w_first != 0)) {
    if (block < w.row_tiles * w.tiles_n * w.splits)
      block_tile<BM, BN, WM, WN, 1, S, OP, OUT_W, kPlain, false, kTN>(
          w, block, (lds_u8*)ring, (lds_f32*)none, (lds_f32*)none);
  } else {
    if (block < x.row_tiles * x.tiles_n * x.splits)
      block_tile<BM, BN, WM, WN, 1, S, OP, OUT_X, kPlain, false, kNN>(
          x, block, (lds_u8*)ring, (lds_f32*)none, (lds_f32*)none);
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
//
// MODE kGated: a fragment of B is BR / 2 rows of the gate and the same ones of
// the up projection, so that few columns still make as many workgroups.  BR 8:
// half a fragment's rows, the rest of it left out of the loads, so that twice
// as many CUs read (one takes in about 23 bytes a ns, whatever it has in
// flight: 8 steps ahead, or 16 waves, were no faster): 1 x 1024 x 8192 gated in
// bf16 9.5 us, 13.4 with whole fragments.
template <int FM, int FN, int W, int U, int OP, int OUT, int MODE = kPlain, int BR = 16>
__global__ __attribute__((amdgpu_flat_work_group_size(W * 64, W * 64))) void
block_row_kernel(BlockArgs a) {
  constexpr bool kScaled = OP == kOpE4m3;
  constexpr bool kPairs = MODE == kGated;
  static_assert((!kPairs && BR == 16) || FN == 1, "one fragment of both");
  static_assert(BR == 16 || BR == 8, "whole or half fragments");
  constexpr int BM = 16 * FM, BN = kPairs ? BR / 2 : BR * FN;  // rows and columns of C
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
  // gated: the lanes of a fragment read two places of W, more than a buffer
  // resource may span apart; rows past the last column read its row again
  const uint8_t* const pair_row =
      a.B + (lrow < BR / 2 ? 0 : a.up_b) +
      (int64_t)(n0 + min(lrow % (BR / 2), rows_b - 1)) * a.ldb + lchunk;
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
  const float* sb_row =
      kScaled ? a.SB + tile.expert * a.stride_sb + (int64_t)(n0 / kScaleBlock) * a.ldsb : nullptr;

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
    if constexpr (kPairs) {
      // (a chunk past K: any, `multiply` clears it)
      if (lrow < BR) {
        s.fb[0][0] = __builtin_nontemporal_load((const u32x4*)(pair_row + (in0 ? k0 : -lchunk)));
        s.fb[0][1] = __builtin_nontemporal_load((const u32x4*)(pair_row + (in1 ? k0 + 64 : -lchunk)));
      }
    } else {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        s.fb[j][0] = get(rsrc_b, vb[j], in0, 0, nt);
        s.fb[j][1] = get(rsrc_b, vb[j], in1, 64, nt);
      }
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
    if (X == a.k_steps - 1 && (a.kbytes & (kPairs ? kStepBytes - 1 : 15)) != 0) {
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
  auto total = [&](int f, int l) __attribute__((always_inline)) {
    f32x4 v = sums[0][f][l];
#pragma unroll
    for (int w = 1; w < W; ++w) v = add_sums<OP>(v, sums[w][f][l]);
    return v;
  };
  auto scaled = [&](const f32x4& v, const float* sb, int row, int n) __attribute__((always_inline)) {
    if constexpr (OP == kOpI8) {
      const i32x4 sum = __builtin_bit_cast(i32x4, v);
      const f32x4 s = column_scales(sb, n, a.N);
      const float sa = a.SA[m0 + row];
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = (float)sum[r] * sa * s[r];
      return x;
    } else {
      return v;
    }
  };
  if constexpr (kPairs) {
    for (int q = tid; q < FM * 2 * BR; q += W * 64) {
      const int i = q / (2 * BR), l = q % (2 * BR);
      const int row = i * 16 + (l & 15), n = n0 + 4 * (l >> 4);
      if (row >= rows_a) continue;
      const f32x4 g = scaled(total(i, l), a.SB, row, n);
      const f32x4 u = scaled(total(i, l + 2 * BR), a.SB + a.up_sb, row, n);
      f32x4 h;
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = gate<OUT>(g[r], u[r], a.geglu != 0);
      store_quad<OUT>(a.C, a.ldc, h, m0 + row, n, a.N);
      if constexpr (OP != kOpI8) {
        if (a.kept != nullptr && n < a.N) {
          uint8_t* const at = a.kept + (int64_t)(m0 + row) * a.ld_kept;
          const int64_t f = a.kept_first + n;
          *(u32x2*)(at + f * 2) = kept_high(g);
          *(u32x2*)(at + (a.kept_f + f) * 2) = kept_high(u);
          *(uint32_t*)(at + 4 * a.kept_f + f) = kept_third(g);
          *(uint32_t*)(at + 5 * a.kept_f + f) = kept_third(u);
        }
      }
    }
  } else {
    for (int q = tid; q < FM * FN * 64; q += W * 64) {
      const int f = q >> 6, l = q & 63;
      const int row = (f / FN) * 16 + (l & 15), n = n0 + (f % FN) * 16 + 4 * (l >> 4);
      if (row < rows_a && l < 4 * BR)
        store_quad<OUT>(a.C, a.ldc, scaled(total(f, l), a.SB, row, n), m0 + row, n, a.N);
    }
  }
}

}  // namespace gemm
