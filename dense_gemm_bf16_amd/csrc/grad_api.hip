// C-ABI front end of the gradients of dense and gated products: argument
// checks, the choice of tile and split, launch.  The contract of every entry
// point is stated in include/gemm_bf16.h.  Nothing here allocates or throws.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

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
int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// ------------------------------------------------------- choice of shape
// One product: C (halves x M rows, N columns), K in `parts` of k each.
struct GradShape {
  int64_t M, N, k;
  int parts, halves;
};
constexpr GradShape kNoProduct{0, 0, 0, 1, 1};

// `resident` workgroups a CU; a workgroup's time is steps * step + tile with
// all of them there, `part` of that where it has the GPU to itself (us).
struct GradTile {
  const char* name;
  int bm, bn, threads, resident;
  double step, tile, part;
  hipError_t (*launch)(const GradPair&, hipStream_t, int op, int out_x, int out_w);
};
const GradTile kTiles[] = {
    {"b256x256", 256, 256, 512, 1, 1.226, 9.0, 0.970, &launch_grad_pair<256, 256, 2, 4, 2>},
    {"b128x128", 128, 128, 256, 2, 0.782, 5.8, 0.901, &launch_grad_pair<128, 128, 2, 2, 2>},
};
constexpr double kSumUs = 3.41, kSumUsPerMB = 0.584, kTail = 0.119;

struct GradPlan {
  const GradTile* tile;
  int split_x, split_w;  // ways that K is split over workgroups
};

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }
int64_t tiles_of(const GradTile& t, const GradShape& p) {
  return (p.M + t.bm - 1) / t.bm * p.halves * ((p.N + t.bn - 1) / t.bn);
}
int64_t steps_of(const GradShape& p) { return (p.k + 63) / 64 * p.parts; }
int64_t part_floats(const GradShape& p) { return p.M * p.halves * up4(p.N); }
int64_t split_bytes(const GradShape& p, int splits) {
  return splits > 1 ? 4 * splits * part_floats(p) : 0;
}

// The ways that leave none of n steps' slices empty.
int even_splits(int64_t n, int64_t s) {
  if (s > n) s = n;
  if (s <= 1) return 1;
  const int64_t per = (n + s - 1) / s;
  return (int)((n + per - 1) / per);
}

// The tile and splits whose launch a model finds cheapest: as long as its
// longest workgroup, shorter where the GPU is part empty, or as all of them
// over the places there are; and for splits the round trip of their fp32 sums.
// Its constants were searched for the best choice over 50 products (1 to 8192
// tokens, 256 to 14336 x 128 to 8192), each timed in the plans that were in
// question: 0.9 % from the fastest of them, and 0.9 % over 50 other products
// (22 % at worst).  gated_model.py holds the same model, the sweep, its times
// and the search.
GradPlan choose(const GradShape& x, const GradShape& w) {
  GradPlan best{nullptr, 1, 1};
  double best_t = 0;
  const int64_t steps[2] = {steps_of(x), steps_of(w)};
  for (const GradTile& t : kTiles) {
    const int64_t tiles[2] = {tiles_of(t, x), tiles_of(t, w)};
    const double places = 256.0 * t.resident;
    for (int sx = 1; sx <= 16; sx *= 2) {
      if (sx > 1 && (steps[0] / sx < 4 || tiles[0] * sx > 1024)) break;
      for (int sw = 1; sw <= 16; sw *= 2) {
        if (sw > 1 && (steps[1] / sw < 4 || tiles[1] * sw > 1024)) break;
        const double ux = (double)((steps[0] + sx - 1) / sx) * t.step + t.tile;
        const double uw = (double)((steps[1] + sw - 1) / sw) * t.step + t.tile;
        const double nx = (double)(tiles[0] * sx), nw = (double)(tiles[1] * sw);
        const double longest = nx > 0 && (ux > uw || nw == 0) ? ux : uw;
        const double fill = (nx + nw) / places;
        double us = longest * (t.part + (1 - t.part) * (fill < 1 ? fill : 1));
        const double all = (nx * ux + nw * uw) / places;
        if (fill > 1) us = (all > us ? all : us) + kTail * longest;
        if (sx > 1 || sw > 1)
          us += kSumUs + kSumUsPerMB * 1e-6 * (double)(split_bytes(x, sx) + split_bytes(w, sw));
        if (best.tile && us >= best_t) continue;
        best = GradPlan{&t, sx, sw};
        best_t = us;
      }
    }
  }
  best.split_x = even_splits(steps[0], best.split_x);
  best.split_w = even_splits(steps[1], best.split_w);
  return best;
}

// The plan a call names ("b128x128_k4_k1"), or without a name the chosen one;
// no tile: there is no such plan.
GradPlan plan_of(const char* config, const GradShape& x, const GradShape& w) {
  if (!config || !config[0]) return choose(x, w);
  GradPlan p{nullptr, 1, 1};
  for (const GradTile& t : kTiles) {
    const size_t n = strlen(t.name);
    if (strncmp(config, t.name, n) != 0 || strncmp(config + n, "_k", 2) != 0) continue;
    char* end = nullptr;
    const long sx = strtol(config + n + 2, &end, 10);
    if (strncmp(end, "_k", 2) != 0) continue;
    const long sw = strtol(end + 2, &end, 10);
    if (*end || sx < 1 || sx > 64 || sw < 1 || sw > 64) continue;
    p = GradPlan{&t, even_splits(steps_of(x), sx), even_splits(steps_of(w), sw)};
    // (a grid holds fewer than 2^32 threads: of the products, and of the sums,
    // 1024 columns a workgroup of 256)
    const int64_t sums = (p.split_x > 1 ? part_floats(x) / 1024 + 1 : 0) +
                         (p.split_w > 1 ? part_floats(w) / 1024 + 1 : 0);
    if (tiles_of(t, x) * p.split_x + tiles_of(t, w) * p.split_w >= 2 * k2G / t.threads - 8 ||
        sums >= 2 * k2G / 256)
      p.tile = nullptr;
  }
  return p;
}

int64_t plan_bytes(const GradPlan& p, const GradShape& x, const GradShape& w) {
  return split_bytes(x, p.split_x) + split_bytes(w, p.split_w);
}

// Whether both tiles can run it: what a workgroup loads from one base lies
// within a buffer resource, the grid holds fewer than 2^32 threads.
bool runs(const GradShape& p, bool a_rows_m, int64_t lda, int64_t ldb) {
  for (const GradTile& t : kTiles)
    if ((a_rows_m ? t.bm : 64) * lda * 2 >= kRangeLimit || 64 * ldb * 2 >= kRangeLimit ||
        tiles_of(t, p) >= k2G / t.threads - 8)
      return false;
  return true;
}

struct Operands {
  const void *A, *B;
  int64_t lda, ldb, seg_a, seg_b, half_a;  // elements
  void* C;
  int64_t ldc;
};

BlockArgs product_args(const GradTile& t, const GradShape& p, const Operands& o, int splits,
                       float* parts) {
  const int64_t row_tiles = (p.M + t.bm - 1) / t.bm * p.halves, steps = steps_of(p);
  BlockArgs a{};
  a.A = (const uint8_t*)o.A;
  a.B = (const uint8_t*)o.B;
  a.C = splits > 1 ? parts : o.C;
  a.lda = o.lda * 2;
  a.ldb = o.ldb * 2;
  a.ldc = splits > 1 ? up4(p.N) : o.ldc;
  a.M = (int32_t)p.M;
  a.N = (int32_t)p.N;
  a.kbytes = (int32_t)(p.k * 2);
  a.a_rows = (int32_t)p.M;
  a.E = 1;
  a.tiles_n = (int32_t)((p.N + t.bn - 1) / t.bn);
  a.k_steps = (int32_t)steps;
  a.row_tiles = (int32_t)row_tiles;
  a.group_m = 4;
  a.seg_steps = (int32_t)(steps / p.parts);
  a.seg_a = o.seg_a * 2;
  a.seg_b = o.seg_b * 2;
  a.half_tiles = (int32_t)(row_tiles / p.halves);
  a.half_a = o.half_a * 2;
  a.splits = splits;
  a.split_steps = (int32_t)((steps + splits - 1) / splits);
  a.part_stride = part_floats(p);
  return a;
}

int store_of(int type) {
  return type == GEMM_TYPE_F32 ? kStoreF32 : type == GEMM_TYPE_F16 ? kStoreF16 : kStoreBf16;
}

// Both products (a shape without rows or columns: none) and their sums.
hipError_t grad_products(const GradPlan& plan, int type, const GradShape& x, const Operands& ox,
                         const GradShape& w, const Operands& ow, int w_type, void* work,
                         hipStream_t stream) {
  const GradTile& t = *plan.tile;
  float* const px = (float*)work;
  float* const pw = px + split_bytes(x, plan.split_x) / 4;
  GradPair pair{};
  pair.x = product_args(t, x, ox, plan.split_x, px);
  pair.w = product_args(t, w, ow, plan.split_w, pw);
  const int64_t nx = tiles_of(t, x) * plan.split_x, nw = tiles_of(t, w) * plan.split_w;
  if (nx + nw == 0) return hipSuccess;
  // the longer workgroups first
  pair.w_first = nx == 0 || (nw > 0 && pair.w.split_steps > pair.x.split_steps);
  const int64_t n1 = pair.w_first ? nw : nx, n2 = pair.w_first ? nx : nw;
  pair.first = (int)((n1 + 7) / 8 * 8);
  pair.grid = (int)(n2 > 0 ? pair.first + n2 : n1);
  const int sx = store_of(type), sw = store_of(w_type);
  hipError_t e = t.launch(pair, stream, type == GEMM_TYPE_F16 ? kOpF16 : kOpBf16,
                          plan.split_x > 1 ? kStoreF32 : sx, plan.split_w > 1 ? kStoreF32 : sw);
  if (e != hipSuccess) return e;
  auto sum = [](const GradShape& p, const Operands& o, const float* parts, int splits, int out) {
    return SumParts{parts, p.M * p.halves, up4(p.N), part_floats(p), splits, o.C, o.ldc, p.N, out};
  };
  return launch_sum_parts(sum(x, ox, px, nx > 0 ? plan.split_x : 1, sx),
                          sum(w, ow, pw, nw > 0 ? plan.split_w : 1, sw), stream);
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

int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

thread_local char g_plan_name[48];

const char* plan_name(const GradShape& x, const GradShape& w) {
  const GradPlan plan = choose(x, w);
  snprintf(g_plan_name, sizeof g_plan_name, "%s_k%d_k%d", plan.tile->name, plan.split_x,
           plan.split_w);
  return g_plan_name;
}

// Parts of both gradients, or of either one alone; -1: no such plan.
int64_t most_bytes(const char* config, const GradShape& x, const GradShape& w) {
  int64_t most = 0;
  const GradShape pairs[3][2] = {{x, w}, {x, kNoProduct}, {kNoProduct, w}};
  for (const auto& p : pairs) {
    const GradPlan plan = plan_of(config, p[0], p[1]);
    if (!plan.tile) return -1;
    most = larger(most, plan_bytes(plan, p[0], p[1]));
  }
  return most;
}

// dG and dU lie side by side, each in rows of whole 128-byte lines, so that a
// K-step's 128 bytes of a row are one line (512 x 5001 x 2055: 80.6 us with rows
// of 5008, 74.2; 2048 x 5461 x 2048: 198, 191).
int64_t gate_columns(int64_t F) { return up64(F); }
int64_t gate_bytes(int64_t M, int64_t F) { return up256(M * 2 * gate_columns(F) * 2); }

}  // namespace
}  // namespace gemm

extern "C" {

size_t gemm_backward_work_size(const char* config, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || gemm::size_refused(M, N, K)) return 0;
  const int64_t n =
      gemm::most_bytes(config, gemm::input_shape(M, N, K), gemm::weight_shape(M, N, K));
  return n > 0 ? (size_t)n : 0;
}

const char* gemm_backward_config_name(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || gemm::size_refused(M, N, K)) return "invalid";
  return gemm::plan_name(gemm::input_shape(M, N, K), gemm::weight_shape(M, N, K));
}

const char* gemm_gated_backward_config_name(int64_t M, int64_t F, int64_t K) {
  if (M < 0 || F < 0 || K < 0 || gemm::size_refused(M, F, K)) return "invalid";
  return gemm::plan_name(gemm::gated_input_shape(M, F, K), gemm::gated_weight_shape(M, F, K));
}

int gemm_backward_ex(const char* config, int type, int64_t M, int64_t N, int64_t K, const void* dC,
                     int64_t lddc, const void* A, int64_t lda, const void* B, int64_t ldb, void* dA,
                     int64_t ldda, void* dB, int64_t lddb, int db_type, void* work,
                     size_t work_bytes, void* stream) {
  using namespace gemm;
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16) return GEMM_ERR_INVALID_ARG;
  if (dB && db_type != type && db_type != GEMM_TYPE_F32) return GEMM_ERR_INVALID_ARG;
  if (size_refused(M, N, K) || lddc >= kStrideLimit ||
      (dA && (ldb >= kStrideLimit || ldda >= kStrideLimit)) ||
      (dB && (lda >= kStrideLimit || lddb >= kStrideLimit)))
    return GEMM_ERR_UNSUPPORTED;
  const bool has_a = dA && M > 0 && K > 0, has_b = dB && N > 0 && K > 0;
  if (lddc < N || (dA && (ldb < K || ldda < K)) || (dB && (lda < K || lddb < K)))
    return GEMM_ERR_INVALID_ARG;
  if ((has_a || has_b) && M > 0 && N > 0 &&
      (!dC || (has_a && !B) || (has_b && !A)))
    return GEMM_ERR_INVALID_ARG;
  if (misaligned(dC, 16) || (dB && misaligned(A, 16)) || (dA && misaligned(B, 16)) ||
      misaligned(dA, 16) || misaligned(dB, 16) || misaligned(work, 16) || (lddc & 7) ||
      (dA && ((ldb | ldda) & 7)) || (dB && ((lda | lddb) & 7)))
    return GEMM_ERR_MISALIGNED;
  const GradShape pa = has_a ? input_shape(M, N, K) : kNoProduct;
  const GradShape pb = has_b ? weight_shape(M, N, K) : kNoProduct;
  if ((has_a && !runs(pa, true, lddc, ldb)) || (has_b && !runs(pb, false, lddc, lda)))
    return GEMM_ERR_UNSUPPORTED;
  const GradPlan plan = plan_of(config, pa, pb);
  if (!plan.tile) return GEMM_ERR_UNSUPPORTED;
  const int64_t need = plan_bytes(plan, pa, pb);
  if (need > 0 && (!work || (int64_t)work_bytes < need)) return GEMM_ERR_SCRATCH;
  const hipError_t e =
      grad_products(plan, type, pa, Operands{dC, B, lddc, ldb, 0, 0, 0, dA, ldda}, pb,
                    Operands{dC, A, lddc, lda, 0, 0, 0, dB, lddb}, dB ? db_type : type, work,
                    (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

int gemm_backward(int type, int64_t M, int64_t N, int64_t K, const void* dC, int64_t lddc,
                  const void* A, int64_t lda, const void* B, int64_t ldb, void* dA, int64_t ldda,
                  void* dB, int64_t lddb, int db_type, void* work, size_t work_bytes,
                  void* stream) {
  return gemm_backward_ex(nullptr, type, M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb,
                          db_type, work, work_bytes, stream);
}

size_t gemm_gated_backward_work_size(const char* config, int64_t M, int64_t F, int64_t K) {
  if (M < 0 || F < 0 || K < 0 || gemm::size_refused(M, F, K)) return 0;
  if (M > 0 && gemm::gate_columns(F) > gemm::kStrideLimit / M) return 0;
  const int64_t n = gemm::most_bytes(config, gemm::gated_input_shape(M, F, K),
                                     gemm::gated_weight_shape(M, F, K));
  return n < 0 ? 0 : (size_t)(gemm::gate_bytes(M, F) + n);
}

int gemm_gated_backward_ex(const char* config, int type, int64_t M, int64_t F, int64_t K,
                           const void* dH, int64_t lddh, const void* X, int64_t ldx, const void* W,
                           int64_t ldw, int act, const void* kept, int64_t ld_kept, void* dX,
                           int64_t lddx, void* dW, int64_t lddw, int dw_type, void* work,
                           size_t work_bytes, void* stream) {
  using namespace gemm;
  if (M < 0 || F < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16) return GEMM_ERR_INVALID_ARG;
  if (act != GEMM_ACT_SWIGLU && act != GEMM_ACT_GEGLU) return GEMM_ERR_INVALID_ARG;
  if (dW && dw_type != type && dw_type != GEMM_TYPE_F32) return GEMM_ERR_INVALID_ARG;
  const int64_t Fp = up8(F < k2G ? F : k2G), kept_f = (Fp + 15) / 16 * 16, ld = gate_columns(Fp);
  // (2^32 pieces of eight columns: dG, dU and what was kept would take 340 GB)
  if (size_refused(M, F, K) || (M > 0 && Fp / 8 >= 2 * k2G / M) || lddh >= kStrideLimit ||
      ld_kept >= kStrideLimit || (dX && (ldw >= kStrideLimit || lddx >= kStrideLimit)) ||
      (dW && (ldx >= kStrideLimit || lddw >= kStrideLimit)))
    return GEMM_ERR_UNSUPPORTED;
  const bool has_x = dX && M > 0 && K > 0, has_w = dW && F > 0 && K > 0;
  if (lddh < F || ld_kept < 6 * kept_f || (dX && (ldw < K || lddx < K)) ||
      (dW && (ldx < K || lddw < K)))
    return GEMM_ERR_INVALID_ARG;
  if ((has_x || has_w) && M > 0 && F > 0 && (!dH || !kept || (has_x && !W) || (has_w && !X)))
    return GEMM_ERR_INVALID_ARG;
  if (misaligned(dH, 16) || (dW && misaligned(X, 16)) || (dX && misaligned(W, 16)) ||
      misaligned(kept, 16) || misaligned(dX, 16) || misaligned(dW, 16) || misaligned(work, 16) ||
      (lddh & 7) || (ld_kept & 15) || (dX && ((ldw | lddx) & 7)) || (dW && ((ldx | lddw) & 7)))
    return GEMM_ERR_MISALIGNED;
  const GradShape px = has_x ? gated_input_shape(M, F, K) : kNoProduct;
  const GradShape pw = has_w ? gated_weight_shape(M, F, K) : kNoProduct;
  if ((has_x && !runs(px, true, 2 * ld, ldw)) || (has_w && !runs(pw, false, 2 * ld, ldx)))
    return GEMM_ERR_UNSUPPORTED;
  if (!has_x && !has_w) return GEMM_OK;
  const GradPlan plan = plan_of(config, px, pw);
  if (!plan.tile) return GEMM_ERR_UNSUPPORTED;
  const int64_t gate = gate_bytes(M, F), need = gate + plan_bytes(plan, px, pw);
  if (need > 0 && (!work || (int64_t)work_bytes < need)) return GEMM_ERR_SCRATCH;
  hipError_t e = hipSuccess;
  if (M > 0 && F > 0) {
    const GateGradArgs g{dH,   (const uint8_t*)kept, work,   M, Fp, ld,
                         lddh, ld_kept,              kept_f, act == GEMM_ACT_GEGLU};
    e = launch_gate_grad(g, type == GEMM_TYPE_F16, (hipStream_t)stream);
  }
  if (e == hipSuccess)
    e = grad_products(plan, type, px, Operands{work, W, 2 * ld, ldw, ld, F * ldw, 0, dX, lddx}, pw,
                      Operands{work, X, 2 * ld, ldx, 0, 0, ld, dW, lddw}, dW ? dw_type : type,
                      (uint8_t*)work + gate, (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

int gemm_gated_backward(int type, int64_t M, int64_t F, int64_t K, const void* dH, int64_t lddh,
                        const void* X, int64_t ldx, const void* W, int64_t ldw, int act,
                        const void* kept, int64_t ld_kept, void* dX, int64_t lddx, void* dW,
                        int64_t lddw, int dw_type, void* work, size_t work_bytes, void* stream) {
  return gemm_gated_backward_ex(nullptr, type, M, F, K, dH, lddh, X, ldx, W, ldw, act, kept,
                                ld_kept, dX, lddx, dW, lddw, dw_type, work, work_bytes, stream);
}

}  // extern "C"
