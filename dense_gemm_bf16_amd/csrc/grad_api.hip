// C-ABI front end of the gradients of dense and gated products: argument
// checks, the choice of tile and split, launch.  The contract of every entry
// point is stated in include/gemm_bf16.h.  Nothing here allocates or throws.
#include <stdio.h>

#include "../../include/gemm_bf16.h"
#include "gemm_internal.h"
#include "grad_launch.hpp"

namespace gemm {
namespace {

constexpr int64_t k2G = int64_t(1) << 31;
constexpr int64_t kRangeLimit = k2G - 4096;
constexpr int64_t kStrideLimit = int64_t(1) << 40;

bool misaligned(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// ------------------------------------------------------- choice of shape
// One product: C (halves x M rows, N columns), K in `parts` of k each.
struct GradShape {
  int64_t M, N, k;
  int parts, halves;
};

struct GradTile {
  const char* name;
  int bm, bn, threads;
  double step, tile;  // us: of a K-step of 64, of first loads and epilogue
  hipError_t (*launch)(const BlockArgs&, int grid, hipStream_t, int op, int out, int layout);
};
const GradTile kTiles[] = {
    {"b256x256", 256, 256, 512, 1.60, 6.0, &launch_grad_tile<256, 256, 2, 4, 2>},
    {"b128x128", 128, 128, 256, 0.60, 3.5, &launch_grad_tile<128, 128, 2, 2, 2>},
};

struct GradPlan {
  const GradTile* tile;
  int splits;  // ways that K is split over workgroups
};

int64_t tiles_of(const GradTile& t, const GradShape& p) {
  return (p.M + t.bm - 1) / t.bm * p.halves * ((p.N + t.bn - 1) / t.bn);
}
int64_t steps_of(const GradShape& p) { return (p.k + 63) / 64 * p.parts; }

// The cheapest tile and split under the model of the dense products: passes of
// 256 workgroups, a last one that is part full at two thirds to all of a
// pass's time, and for a split the round trip of its fp32 sums.
GradPlan choose(const GradShape& p) {
  GradPlan best{nullptr, 1};
  double best_t = 0;
  const int64_t steps = steps_of(p);
  for (const GradTile& t : kTiles) {
    const int64_t tiles = tiles_of(t, p);
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (s > 1 && (steps / s < 4 || tiles * s > 1024)) break;
      const int64_t per = (steps + s - 1) / s, units = tiles * s;
      if (s > 1 && (steps + per - 1) / per != s) continue;
      double passes = (double)(units / 256);
      if (units % 256) passes += 0.67 + 0.33 * (double)(units % 256) / 256;
      double us = passes * ((double)per * t.step + t.tile);
      if (s > 1) us += 2.5 + 0.32e-6 * 4 * s * (double)p.M * p.halves * (double)up8(p.N);
      if (best.tile && us >= best_t) continue;
      best = GradPlan{&t, s};
      best_t = us;
    }
  }
  return best;
}

int64_t split_bytes(const GradShape& p) {
  const int s = choose(p).splits;
  return s > 1 ? 4 * s * p.halves * p.M * up8(p.N) : 0;
}

// Whether both tiles can run it: what a workgroup loads from one base lies
// within a buffer resource, the grid holds fewer than 2^32 threads.
bool runs(const GradShape& p, bool a_rows_m, int64_t lda, int64_t ldb) {
  for (const GradTile& t : kTiles)
    if ((a_rows_m ? t.bm : 64) * lda * 2 >= kRangeLimit || 64 * ldb * 2 >= kRangeLimit ||
        tiles_of(t, p) >= 2 * k2G / t.threads)
      return false;
  return true;
}

struct Operands {
  const void *A, *B;
  int64_t lda, ldb, seg_a, seg_b, half_a;  // elements
};

hipError_t grad_product(int layout, int type, const GradShape& p, const Operands& o, void* C,
                        int64_t ldc, int c_type, void* work, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  const GradPlan plan = choose(p);
  const GradTile& t = *plan.tile;
  const int64_t row_tiles = (p.M + t.bm - 1) / t.bm * p.halves, cols = (p.N + t.bn - 1) / t.bn;
  const int64_t steps = steps_of(p);
  const int store = c_type == GEMM_TYPE_F32 ? kStoreF32 : c_type == GEMM_TYPE_F16 ? kStoreF16 : kStoreBf16;
  BlockArgs a{};
  a.A = (const uint8_t*)o.A;
  a.B = (const uint8_t*)o.B;
  a.C = C;
  a.lda = o.lda * 2;
  a.ldb = o.ldb * 2;
  a.ldc = ldc;
  a.M = (int32_t)p.M;
  a.N = (int32_t)p.N;
  a.kbytes = (int32_t)(p.k * 2);
  a.a_rows = (int32_t)p.M;
  a.E = 1;
  a.tiles_n = (int32_t)cols;
  a.k_steps = (int32_t)steps;
  a.row_tiles = (int32_t)row_tiles;
  a.group_m = 4;
  a.seg_steps = (int32_t)(steps / p.parts);
  a.seg_a = o.seg_a * 2;
  a.seg_b = o.seg_b * 2;
  a.half_tiles = (int32_t)(row_tiles / p.halves);
  a.half_a = o.half_a * 2;
  a.splits = plan.splits;
  a.split_steps = (int32_t)((steps + plan.splits - 1) / plan.splits);
  const int64_t ldp = up8(p.N), rows = p.M * p.halves;
  if (plan.splits > 1) {
    a.C = work;
    a.ldc = ldp;
    a.part_stride = rows * ldp;
  }
  hipError_t e = t.launch(a, (int)(row_tiles * cols * plan.splits), stream,
                          type == GEMM_TYPE_F16 ? kOpF16 : kOpBf16,
                          plan.splits > 1 ? kStoreF32 : store, layout);
  if (e == hipSuccess && plan.splits > 1)
    e = launch_splitk_reduce((const float*)work, ldp, rows * ldp, plan.splits, C, ldc, (int)rows,
                             (int)p.N, store, stream);
  return e;
}

// dA (M x K) = dC (M x N) . B (N x K), and dB (N x K) = dC^T . A (M x K).
GradShape input_shape(int64_t M, int64_t N, int64_t K) { return GradShape{M, K, N, 1, 1}; }
GradShape weight_shape(int64_t M, int64_t N, int64_t K) { return GradShape{N, K, M, 1, 1}; }
// The same of a gated product, whose dC is [dG | dU].
GradShape gated_input_shape(int64_t M, int64_t F, int64_t K) { return GradShape{M, K, F, 2, 1}; }
GradShape gated_weight_shape(int64_t M, int64_t F, int64_t K) { return GradShape{F, K, M, 1, 2}; }

bool size_refused(int64_t M, int64_t N, int64_t K) {
  return M >= k2G / 2 || N >= k2G / 4 || K >= k2G / 2;
}

thread_local char g_plan_name[32];

const char* plan_name(const GradShape& p) {
  const GradPlan plan = choose(p);
  snprintf(g_plan_name, sizeof g_plan_name, "%s_k%d", plan.tile->name, plan.splits);
  return g_plan_name;
}

int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

int64_t gate_bytes(int64_t M, int64_t F) { return up256(M * 2 * up8(F) * 2); }

}  // namespace
}  // namespace gemm

extern "C" {

size_t gemm_backward_work_size(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || gemm::size_refused(M, N, K)) return 0;
  return (size_t)gemm::larger(gemm::split_bytes(gemm::input_shape(M, N, K)),
                              gemm::split_bytes(gemm::weight_shape(M, N, K)));
}

const char* gemm_backward_config_name(int64_t M, int64_t N, int64_t K, int of_b) {
  if (M < 0 || N < 0 || K < 0 || gemm::size_refused(M, N, K)) return "invalid";
  return gemm::plan_name(of_b ? gemm::weight_shape(M, N, K) : gemm::input_shape(M, N, K));
}

const char* gemm_gated_backward_config_name(int64_t M, int64_t F, int64_t K, int of_w) {
  if (M < 0 || F < 0 || K < 0 || gemm::size_refused(M, F, K)) return "invalid";
  return gemm::plan_name(of_w ? gemm::gated_weight_shape(M, F, K)
                              : gemm::gated_input_shape(M, F, K));
}

int gemm_backward(int type, int64_t M, int64_t N, int64_t K, const void* dC, int64_t lddc,
                  const void* A, int64_t lda, const void* B, int64_t ldb, void* dA, int64_t ldda,
                  void* dB, int64_t lddb, int db_type, void* work, size_t work_bytes,
                  void* stream) {
  using namespace gemm;
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16) return GEMM_ERR_INVALID_ARG;
  if (dB && db_type != type && db_type != GEMM_TYPE_F32) return GEMM_ERR_INVALID_ARG;
  if (size_refused(M, N, K) || lddc >= kStrideLimit || lda >= kStrideLimit ||
      ldb >= kStrideLimit || ldda >= kStrideLimit || lddb >= kStrideLimit)
    return GEMM_ERR_UNSUPPORTED;
  const bool has_a = dA && M > 0 && K > 0, has_b = dB && N > 0 && K > 0;
  if (lddc < N || (dA && (ldb < K || ldda < K)) || (dB && (lda < K || lddb < K)))
    return GEMM_ERR_INVALID_ARG;
  if ((has_a || has_b) && M > 0 && N > 0 &&
      (!dC || (has_a && !B) || (has_b && !A)))
    return GEMM_ERR_INVALID_ARG;
  if (misaligned(dC, 16) || misaligned(A, 16) || misaligned(B, 16) || misaligned(dA, 16) ||
      misaligned(dB, 16) || misaligned(work, 16) || (lddc & 7) || (dA && ((ldb | ldda) & 7)) ||
      (dB && ((lda | lddb) & 7)))
    return GEMM_ERR_MISALIGNED;
  const GradShape pa = input_shape(M, N, K), pb = weight_shape(M, N, K);
  if ((has_a && !runs(pa, true, lddc, ldb)) || (has_b && !runs(pb, false, lddc, lda)))
    return GEMM_ERR_UNSUPPORTED;
  const int64_t need = larger(has_a ? split_bytes(pa) : 0, has_b ? split_bytes(pb) : 0);
  if (need > 0 && (!work || (int64_t)work_bytes < need)) return GEMM_ERR_SCRATCH;
  hipError_t e = hipSuccess;
  if (has_a)
    e = grad_product(kNN, type, pa, Operands{dC, B, lddc, ldb, 0, 0, 0}, dA, ldda, type, work,
                     (hipStream_t)stream);
  if (e == hipSuccess && has_b)
    e = grad_product(kTN, type, pb, Operands{dC, A, lddc, lda, 0, 0, 0}, dB, lddb, db_type, work,
                     (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

size_t gemm_gated_backward_work_size(int64_t M, int64_t F, int64_t K) {
  if (M < 0 || F < 0 || K < 0 || gemm::size_refused(M, F, K)) return 0;
  if (M > 0 && gemm::up8(F) > gemm::kStrideLimit / M) return 0;
  return (size_t)(gemm::gate_bytes(M, F) +
                  gemm::larger(gemm::split_bytes(gemm::gated_input_shape(M, F, K)),
                               gemm::split_bytes(gemm::gated_weight_shape(M, F, K))));
}

int gemm_gated_backward(int type, int64_t M, int64_t F, int64_t K, const void* dH, int64_t lddh,
                        const void* X, int64_t ldx, const void* W, int64_t ldw, int act,
                        const void* GU, int64_t ldgu, void* dX, int64_t lddx, void* dW,
                        int64_t lddw, int dw_type, void* work, size_t work_bytes, void* stream) {
  using namespace gemm;
  if (M < 0 || F < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16) return GEMM_ERR_INVALID_ARG;
  if (act != GEMM_ACT_SWIGLU && act != GEMM_ACT_GEGLU) return GEMM_ERR_INVALID_ARG;
  if (dW && dw_type != type && dw_type != GEMM_TYPE_F32) return GEMM_ERR_INVALID_ARG;
  const int64_t Fp = up8(F < k2G ? F : k2G);
  // (a workgroup of 256 for 2048 values of dGU: a grid holds fewer than 2^32 threads)
  if (size_refused(M, F, K) || (M > 0 && Fp / 8 >= 2 * k2G / M) || lddh >= kStrideLimit ||
      ldx >= kStrideLimit || ldw >= kStrideLimit || ldgu >= kStrideLimit || lddx >= kStrideLimit ||
      lddw >= kStrideLimit)
    return GEMM_ERR_UNSUPPORTED;
  const bool has_x = dX && M > 0 && K > 0, has_w = dW && F > 0 && K > 0;
  if (lddh < F || ldgu < 2 * Fp || (dX && (ldw < K || lddx < K)) || (dW && (ldx < K || lddw < K)))
    return GEMM_ERR_INVALID_ARG;
  if ((has_x || has_w) && M > 0 && F > 0 && (!dH || !GU || (has_x && !W) || (has_w && !X)))
    return GEMM_ERR_INVALID_ARG;
  if (misaligned(dH, 16) || misaligned(X, 16) || misaligned(W, 16) || misaligned(GU, 16) ||
      misaligned(dX, 16) || misaligned(dW, 16) || misaligned(work, 16) || ((lddh | ldgu) & 7) ||
      (dX && ((ldw | lddx) & 7)) || (dW && ((ldx | lddw) & 7)))
    return GEMM_ERR_MISALIGNED;
  const GradShape px = gated_input_shape(M, F, K), pw = gated_weight_shape(M, F, K);
  if ((has_x && !runs(px, true, 2 * Fp, ldw)) || (has_w && !runs(pw, false, 2 * Fp, ldx)))
    return GEMM_ERR_UNSUPPORTED;
  if (!has_x && !has_w) return GEMM_OK;
  const int64_t gate = gate_bytes(M, F);
  const int64_t need =
      gate + larger(has_x ? split_bytes(px) : 0, has_w ? split_bytes(pw) : 0);
  if (need > 0 && (!work || (int64_t)work_bytes < need)) return GEMM_ERR_SCRATCH;
  hipError_t e = hipSuccess;
  if (M > 0 && F > 0) {
    const GateGradArgs g{dH, GU, work, M, Fp, lddh, ldgu, 2 * Fp, act == GEMM_ACT_GEGLU};
    e = launch_gate_grad(g, type == GEMM_TYPE_F16, (hipStream_t)stream);
  }
  void* const parts = (uint8_t*)work + gate;
  if (e == hipSuccess && has_x)
    e = grad_product(kNN, type, px, Operands{work, W, 2 * Fp, ldw, Fp, F * ldw, 0}, dX, lddx, type,
                     parts, (hipStream_t)stream);
  if (e == hipSuccess && has_w)
    e = grad_product(kTN, type, pw, Operands{work, X, 2 * Fp, ldx, 0, 0, Fp}, dW, lddw, dw_type,
                     parts, (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

}  // extern "C"
