// C-ABI front end of the 8-bit and mixture-of-experts operators: argument
// checks, the choice of kernel shape, launch.  The contract of every entry
// point is stated in include/gemm_bf16.h.  Nothing here allocates or throws.
#include "../../include/gemm_bf16.h"

#include <math.h>
#include <stdio.h>
#include <string.h>

#include "block_launch.hpp"
#include "gemm_internal.h"

namespace gemm {

const BlockConfig* block_configs() {
  static const BlockConfig table[] = {
#define ROW(NAME, A, B, C, D, E, S) \
  {#NAME, A, B, (C) * (D) * (E) * 64, &launch_block_tile<A, B, C, D, E, S>},
      BLOCK_TILES(ROW)
#undef ROW
#define ROW(NAME, A, B, C, D) {#NAME, 16 * A, 16 * B, (C) * 64, &launch_block_row<A, B, C, D>},
      BLOCK_ROWS(ROW)
#undef ROW
      {nullptr, 0, 0, 0, nullptr}};
  return table;
}

namespace {

constexpr int64_t k2G = int64_t(1) << 31;
constexpr int64_t kRangeLimit = k2G - 4096;

const BlockConfig* block_config(const char* name) {
  for (const BlockConfig* c = block_configs(); c->name; ++c)
    if (strcmp(c->name, name) == 0) return c;
  return nullptr;
}

// Row tiles of a product: exact for a dense one, for experts the most that
// R rows over E experts can need (each expert with rows adds at most one
// tile that is not full).
int64_t row_tile_bound(int64_t R, int64_t E, bool experts, int64_t bm) {
  if (!experts) return (R + bm - 1) / bm;
  const int64_t used = R < E ? R : E;
  return used + (R - used) / bm;
}

// ------------------------------------------------------- choice of shape
// The shape that a model of a launch's time on MI355X makes cheapest, fitted
// (least squares on log time) to 167 swept products timed in the shapes below
// that were in question (dense: M 1-4096, N x K from 600 x 1000 to 28672 x
// 1024; experts: 8 to 128 experts, 1 to 8192 tokens, e4m3 and bf16; r16x16
// with dense products only).  Its choice ran within
// 0.9 % of the fastest shape timed (geometric mean; 18 % at worst), 2.0 % (24
// %) for e4m3 with fp32 output, and within 3.7 % over 70 products of 1 to 16
// tokens with experts of 512 x 512 to 4096 x 4096 timed afterwards in every
// shape (33 % at worst: 5.3 us where r16x16 takes 4.0).  block_model.py holds the same model, the
// sweep, its times and the fit, which gives these constants.
//
// A launch of `units` workgroups on CUs that hold `resident` of them each
// makes passes of 256 * resident; a pass costs steps * step + tile (steps:
// K-steps of a workgroup's wave group; tile: first loads and epilogue), a
// last pass with a fraction f of its workgroups part + (1 - part) * f of
// that.  The whole takes at least as long as reading B at 5.2 TB/s (joined as
// fourth powers, so near the floor the cheaper compute still counts).
struct BlockCost {  // of the shape in the same place of block_configs()
  const char* name;
  int k_groups, resident;
  struct Fit {
    float step, tile, part, base;  // us, us, share, us
  } fit, wide;                     // wide: e4m3 with fp32 output (codes widened to bf16)
};
// Two shapes are not chosen for e4m3 with fp32 output.  256 x 256 spills its
// widened fragments: 4.9 us a K-step, where four 128 x 128 tiles on two CUs
// take 3.6.  256 x 128 was the fastest of all for one of the 24 products (2048
// x 4096 x 4096: 60.0 us, 128 x 128 65.6) and slower on the others, up to 15 %
// where it counts (777 x 10240 x 4104: 114.6 us, 128 x 128 99.7), and the
// model misjudges it (13 % rms) and would take it there.
constexpr float kNever = 1e9f;
constexpr BlockCost kBlockCosts[] = {
    {"b256x256", 1, 1, {1.586f, 6.15f, 0.69f, 2.19f}, {kNever, 0, 0, 0}},
    {"b256x128", 1, 1, {0.932f, 4.29f, 0.76f, 1.51f}, {kNever, 0, 0, 0}},
    {"b128x128", 1, 2, {1.032f, 3.95f, 0.55f, 2.44f}, {1.822f, 4.58f, 0.61f, 0.00f}},
    {"b128x128k2", 2, 1, {1.172f, 5.23f, 0.83f, 1.37f}, {1.962f, 5.14f, 0.85f, 0.00f}},
    {"b64x128k2", 2, 1, {0.873f, 3.68f, 0.75f, 1.39f}, {1.299f, 3.53f, 0.86f, 0.73f}},
    {"b64x64", 1, 2, {0.492f, 3.41f, 0.67f, 1.06f}, {0.774f, 1.59f, 0.56f, 2.97f}},
    {"b64x64k2", 2, 1, {0.528f, 3.97f, 0.84f, 0.44f}, {0.799f, 3.88f, 0.85f, 0.57f}},
    {"b32x128", 1, 2, {0.645f, 3.14f, 0.62f, 0.83f}, {1.032f, 0.00f, 0.50f, 2.96f}},
    {"b32x64k4", 4, 1, {0.678f, 4.52f, 0.88f, 0.00f}, {0.932f, 4.82f, 0.90f, 0.00f}},
    {"b32x32k4", 4, 1, {0.508f, 3.15f, 0.96f, 1.30f}, {0.663f, 3.46f, 0.92f, 1.12f}},
    {"r16x16", 8, 4, {2.435f, 1.11f, 0.24f, 3.08f}, {2.435f, 1.11f, 0.24f, 3.08f}}};

// The table is read by place: the same shapes in the same order, with as many
// groups of waves along K as they are built with.
constexpr struct {
  const char* name;
  int k_groups;
} kBuiltShapes[] = {
#define ROW(NAME, A, B, C, D, E, S) {#NAME, E},
    BLOCK_TILES(ROW)
#undef ROW
#define ROW(NAME, A, B, C, D) {#NAME, C},
    BLOCK_ROWS(ROW)
#undef ROW
};
constexpr bool costs_match_shapes() {
  constexpr size_t n = sizeof kBuiltShapes / sizeof *kBuiltShapes;
  if (n != sizeof kBlockCosts / sizeof *kBlockCosts) return false;
  for (size_t i = 0; i < n; ++i) {
    const char *a = kBuiltShapes[i].name, *b = kBlockCosts[i].name;
    while (*a && *a == *b) ++a, ++b;
    if (*a != *b || kBuiltShapes[i].k_groups != kBlockCosts[i].k_groups) return false;
  }
  return true;
}
static_assert(costs_match_shapes(), "a line of kBlockCosts for each built shape, in their order");
constexpr double kStreamMBPerUs = 5.2, kStreamBaseUs = 2.5;

// Row tiles as the model counts them.  How the rows fall to the experts is
// known on the device only: each expert with rows is taken to add half a
// tile to the full ones.
double model_row_tiles(const BlockConfig* shape, int64_t R, int64_t E, bool experts) {
  if (!experts) return (double)((R + shape->bm - 1) / shape->bm);
  const double used = (double)(R < E ? R : E);
  const double rows = (double)R / shape->bm + 0.5 * used;
  return rows < used ? used : rows;
}

// The fourth power of a launch's time under the model.
double model_time4(const BlockCost& c, int bn, bool wide, double row_tiles, double b_rows,
                   int64_t N, double k_bytes) {
  const BlockCost::Fit& f = wide ? c.wide : c.fit;
  const double units = row_tiles * (double)((N + bn - 1) / bn);
  const double pass = 256.0 * c.resident;
  double passes = (double)(int64_t)(units / pass);
  const double rest = units / pass - passes;
  if (rest > 0) passes += f.part + (1 - f.part) * rest;
  const double k_steps = (double)(int64_t)((k_bytes + kStepBytes - 1) / kStepBytes);
  const double steps = (double)(int64_t)((k_steps + c.k_groups - 1) / c.k_groups);
  const double t = passes * (steps * f.step + f.tile) + f.base;
  const double floor_us = b_rows * (double)N * k_bytes * 1e-6 / kStreamMBPerUs + kStreamBaseUs;
  return t * t * t * t + floor_us * floor_us * floor_us * floor_us;
}

// What a call runs: one shape on all of C, or (dense products only) `shape`
// on columns 0 .. split_n - 1 and `tail` on the rest.  No shape: none can.
struct BlockPlan {
  const BlockConfig* shape;
  const BlockConfig* tail;
  int64_t split_n;
};

// How far a call's operands reach: bytes from row to row, and for gathered
// rows how many A has (-1: not gathered).
struct Reach {
  int64_t lda, ldb, gathered;
};
constexpr Reach kNear = {0, 0, -1};

// Whether a shape can run R rows by N columns: what a workgroup loads from one
// base (the tile's rows of B, those of A or all of a gathered A) lies within
// a buffer resource, and the grid holds fewer than 2^32 threads (the tiles fit
// 32 bits, so 64 hold the product).
bool block_fits(const BlockConfig* c, int64_t R, int64_t N, int64_t E, bool experts,
                const Reach& r) {
  if (c->bn * r.ldb >= kRangeLimit) return false;
  if ((r.gathered >= 0 ? r.gathered : (int64_t)c->bm) * r.lda >= kRangeLimit) return false;
  const int64_t tiles_n = (N + c->bn - 1) / c->bn;
  return row_tile_bound(R, E, experts, c->bm) * tiles_n < 2 * k2G / c->threads;
}

BlockPlan choose_block(int type, int64_t R, int64_t N, int64_t K, int64_t E, bool experts,
                       int c_type, const Reach& reach) {
  const bool wide = type == GEMM_TYPE_E4M3 && c_type == GEMM_TYPE_F32;
  const double b_rows = experts ? (double)(R < E ? R : E) : 1.0;  // B's, of N rows each
  const double k_bytes = (double)K * (type == GEMM_TYPE_E4M3 ? 1 : 2);
  const BlockConfig* shapes = block_configs();
  auto cheapest = [&](int64_t n, double* t4) {
    const BlockConfig* best = nullptr;
    for (int i = 0; shapes[i].name; ++i) {
      const BlockConfig* shape = shapes + i;
      if (!block_fits(shape, R, n, E, experts, reach)) continue;
      const double t = model_time4(kBlockCosts[i], shape->bn, wide,
                                   model_row_tiles(shape, R, E, experts), b_rows, n, k_bytes);
      if (best && t >= *t4) continue;
      best = shape;
      *t4 = t;
    }
    return best;
  };
  double t4 = 0;
  BlockPlan plan{cheapest(N, &t4), nullptr, N};
  if (experts || R < 1 || !plan.shape) return plan;
  // Where a shape's last pass over the CUs would be part empty: the columns
  // that fill its whole passes, then the rest in the shape that is cheapest
  // for them (777 x 10240 x 4104 with fp32 output 97 -> 82 us, as 511
  // workgroups of 128 x 128 and 182 of 64 x 64).
  double best = sqrt(sqrt(t4)) * 0.97;
  for (int i = 0; shapes[i].name; ++i) {
    const BlockConfig* shape = shapes + i;
    const BlockCost& c = kBlockCosts[i];
    const int64_t rows = (R + shape->bm - 1) / shape->bm, cols = (N + shape->bn - 1) / shape->bn;
    const int64_t pass = 256 * c.resident;
    if (rows > pass) continue;
    const int64_t head = rows * cols / pass * pass / rows * shape->bn / kScaleBlock * kScaleBlock;
    if (head <= 0 || head >= N || !block_fits(shape, R, head, E, experts, reach)) continue;
    const double t1 =
        sqrt(sqrt(model_time4(c, shape->bn, wide, (double)rows, b_rows, head, k_bytes)));
    if (t1 >= best) continue;
    double tail4 = 0;
    const BlockConfig* tail = cheapest(N - head, &tail4);
    if (!tail) continue;
    const double t = t1 + sqrt(sqrt(tail4));
    if (t >= best) continue;
    best = t;
    plan = BlockPlan{shape, tail, head};
  }
  return plan;
}

int element_bytes(int type) { return type == GEMM_TYPE_E4M3 ? 1 : type == GEMM_TYPE_F32 ? 4 : 2; }
bool misaligned(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }
int op_of(int type) {
  return type == GEMM_TYPE_E4M3 ? kOpE4m3 : type == GEMM_TYPE_BF16 ? kOpBf16 : kOpF16;
}
int store_of(int type) {
  return type == GEMM_TYPE_F32 ? kStoreF32 : type == GEMM_TYPE_F16 ? kStoreF16 : kStoreBf16;
}
bool is_float_type(int type) {
  return type == GEMM_TYPE_BF16 || type == GEMM_TYPE_F16 || type == GEMM_TYPE_F32;
}

// The dense (offsets null, E = 1) and the experts' product.  R rows of C;
// a_rows rows of A.
int block_product(const char* config, int type, int64_t R, int64_t N, int64_t K, int64_t E,
                  bool experts, int64_t a_rows, const void* A, int64_t lda, const float* SA,
                  int64_t ldsa, const int32_t* offsets, const int32_t* rows, const void* B,
                  int64_t ldb, int64_t stride_b, const float* SB, int64_t ldsb, int64_t stride_sb,
                  void* C, int64_t ldc, int c_type, void* stream) {
  if (R < 0 || N < 0 || K < 0 || E < 0 || a_rows < 0) return GEMM_ERR_INVALID_ARG;
  if (type != GEMM_TYPE_E4M3 && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16)
    return GEMM_ERR_INVALID_ARG;
  if (!is_float_type(c_type)) return GEMM_ERR_INVALID_ARG;
  const bool scaled = type == GEMM_TYPE_E4M3;
  const int es = element_bytes(type);
  const int64_t kb = K / 128 + (K % 128 != 0);
  if (lda < K || ldb < K || ldc < N || stride_b < 0 || stride_sb < 0) return GEMM_ERR_INVALID_ARG;
  if (scaled && (ldsa < a_rows || ldsb < kb)) return GEMM_ERR_INVALID_ARG;
  const bool work = R > 0 && N > 0 && E > 0;
  if (work) {
    if (!C || (experts && !offsets)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!B || (a_rows > 0 && !A))) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && scaled && (!SB || (a_rows > 0 && !SA))) return GEMM_ERR_INVALID_ARG;
  }
  if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, 16)) return GEMM_ERR_MISALIGNED;
  if (misaligned(SA, 4) || misaligned(SB, 4) || misaligned(offsets, 4) || misaligned(rows, 4))
    return GEMM_ERR_MISALIGNED;
  const int64_t step = 16 / es - 1;
  if (((lda | ldb | stride_b) & step) != 0 || (ldc & 7) != 0) return GEMM_ERR_MISALIGNED;

  if (R >= k2G || N >= k2G || K >= k2G / 2 || E >= k2G || a_rows >= k2G / 4 || lda >= k2G ||
      ldb >= k2G)
    return GEMM_ERR_UNSUPPORTED;
  if (scaled && kb > kMaxKSteps) return GEMM_ERR_UNSUPPORTED;
  const Reach reach{lda * es, ldb * es, rows ? a_rows : -1};
  BlockPlan plan{nullptr, nullptr, N};
  if (config && config[0]) {
    plan.shape = block_config(config);
    if (plan.shape && !block_fits(plan.shape, R, N, E, experts, reach)) plan.shape = nullptr;
  } else {
    plan = choose_block(type, R, N, K, E, experts, c_type, reach);
  }
  if (!plan.shape) return GEMM_ERR_UNSUPPORTED;
  if (!work) return GEMM_OK;

  BlockArgs a{};
  a.A = (const uint8_t*)A;
  a.B = (const uint8_t*)B;
  a.C = C;
  a.SA = SA;
  a.SB = SB;
  a.offsets = experts ? offsets : nullptr;
  a.rows = rows;
  a.lda = lda * es;
  a.ldb = ldb * es;
  a.ldc = ldc;
  a.ldsa = ldsa;
  a.ldsb = ldsb;
  a.stride_b = stride_b * es;
  a.stride_sb = stride_sb;
  a.M = (int32_t)R;
  a.kbytes = (int32_t)(K * es);
  a.a_rows = (int32_t)a_rows;
  a.E = (int32_t)E;
  a.k_steps = (int32_t)((K * es + kStepBytes - 1) / kStepBytes);
  a.group_m = 4;
  auto launch = [&](const BlockConfig* c, int64_t n) {
    const int64_t tiles_n = (n + c->bn - 1) / c->bn;
    const int64_t row_tiles = row_tile_bound(R, E, experts, c->bm);
    a.N = (int32_t)n;
    a.tiles_n = (int32_t)tiles_n;
    a.row_tiles = (int32_t)row_tiles;
    // Where one row tile takes a whole B, tile column j starts 3 j K-steps
    // in: rows of a power-of-two stride would otherwise send all workgroups
    // to the same memory channels (M = 1 and 16 at 8192 x 8192 4 % faster,
    // few rows an expert 3 %; with more row tiles, whose workgroups share B
    // through the L2, up to 11 % slower).
    const int64_t used = R < E ? R : E;
    a.k_rot = (experts ? R <= used * c->bm : row_tiles == 1) ? 3 : 0;
    return c->launch(a, (int)(row_tiles * tiles_n), (hipStream_t)stream, op_of(type),
                     store_of(c_type));
  };
  hipError_t e = launch(plan.shape, plan.split_n);
  if (e == hipSuccess && plan.tail) {  // (the split lies on a scale block's border)
    a.B += plan.split_n * a.ldb;
    if (SB) a.SB += plan.split_n / kScaleBlock * ldsb;
    a.C = (uint8_t*)C + plan.split_n * element_bytes(c_type);
    e = launch(plan.tail, N - plan.split_n);
  }
  return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

thread_local char g_plan_name[64];

}  // namespace
}  // namespace gemm

extern "C" {

int gemm_fp8_ex(const char* config, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                const float* SA, int64_t ldsa, const void* B, int64_t ldb, const float* SB,
                int64_t ldsb, void* C, int64_t ldc, int c_type, void* stream) {
  return gemm::block_product(config, GEMM_TYPE_E4M3, M, N, K, 1, false, M, A, lda, SA, ldsa,
                             nullptr, nullptr, B, ldb, 0, SB, ldsb, 0, C, ldc, c_type, stream);
}

int gemm_fp8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* SA,
             int64_t ldsa, const void* B, int64_t ldb, const float* SB, int64_t ldsb, void* C,
             int64_t ldc, int c_type, void* stream) {
  return gemm_fp8_ex(nullptr, M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, c_type, stream);
}

int gemm_moe_ex(const char* config, int type, int64_t R, int64_t N, int64_t K, int64_t E,
                int64_t T, const void* A, int64_t lda, const float* SA, int64_t ldsa,
                const int32_t* offsets, const int32_t* rows, const void* B, int64_t ldb,
                int64_t stride_b, const float* SB, int64_t ldsb, int64_t stride_sb, void* C,
                int64_t ldc, int c_type, void* stream) {
  if (!rows && T < R) return GEMM_ERR_INVALID_ARG;
  return gemm::block_product(config, type, R, N, K, E, true, T, A, lda, SA, ldsa, offsets, rows, B,
                             ldb, stride_b, SB, ldsb, stride_sb, C, ldc, c_type, stream);
}

int gemm_moe(int type, int64_t R, int64_t N, int64_t K, int64_t E, int64_t T, const void* A,
             int64_t lda, const float* SA, int64_t ldsa, const int32_t* offsets,
             const int32_t* rows, const void* B, int64_t ldb, int64_t stride_b, const float* SB,
             int64_t ldsb, int64_t stride_sb, void* C, int64_t ldc, int c_type, void* stream) {
  return gemm_moe_ex(nullptr, type, R, N, K, E, T, A, lda, SA, ldsa, offsets, rows, B, ldb,
                     stride_b, SB, ldsb, stride_sb, C, ldc, c_type, stream);
}

const char* gemm_fp8_config_name(int64_t M, int64_t N, int64_t K, int c_type) {
  if (M < 0 || N < 0 || K < 0 || M >= gemm::k2G || N >= gemm::k2G || K >= gemm::k2G / 2)
    return "invalid";
  if (!gemm::is_float_type(c_type) || K > gemm::kScaleBlock * gemm::kMaxKSteps) return "invalid";
  const gemm::BlockPlan p =
      gemm::choose_block(GEMM_TYPE_E4M3, M, N, K, 1, false, c_type, gemm::kNear);
  if (!p.shape) return "invalid";
  if (!p.tail) return p.shape->name;
  snprintf(gemm::g_plan_name, sizeof gemm::g_plan_name, "%s+%s", p.shape->name, p.tail->name);
  return gemm::g_plan_name;
}

const char* gemm_moe_config_name(int type, int64_t R, int64_t N, int64_t K, int64_t E, int c_type) {
  if (R < 0 || N < 0 || K < 0 || E < 0 || R >= gemm::k2G || N >= gemm::k2G ||
      K >= gemm::k2G / 2 || E >= gemm::k2G)
    return "invalid";
  if (!gemm::is_float_type(c_type)) return "invalid";
  if (type != GEMM_TYPE_E4M3 && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16) return "invalid";
  if (type == GEMM_TYPE_E4M3 && K > gemm::kScaleBlock * gemm::kMaxKSteps) return "invalid";
  const gemm::BlockPlan p = gemm::choose_block(type, R, N, K, E, true, c_type, gemm::kNear);
  return p.shape ? p.shape->name : "invalid";
}

const char* gemm_fp8_config_at(int i) {
  if (i < 0) return nullptr;
  for (const gemm::BlockConfig* c = gemm::block_configs(); c->name; ++c)
    if (i-- == 0) return c->name;
  return nullptr;
}

int gemm_fp8_quantize(int64_t M, int64_t K, const void* X, int64_t ldx, int x_type, int act,
                      int block_rows, void* Q, int64_t ldq, float* S, int64_t lds, void* stream) {
  if (M < 0 || K < 0 || !gemm::is_float_type(x_type)) return GEMM_ERR_INVALID_ARG;
  if (act != GEMM_ACT_NONE && act != GEMM_ACT_SWIGLU) return GEMM_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != 128) return GEMM_ERR_INVALID_ARG;
  if (block_rows == 128 && act != GEMM_ACT_NONE) return GEMM_ERR_UNSUPPORTED;
  if (K >= gemm::k2G || M >= gemm::k2G || ldx >= (int64_t(1) << 40) || ldq >= (int64_t(1) << 40))
    return GEMM_ERR_UNSUPPORTED;
  const int64_t width = act == GEMM_ACT_SWIGLU ? 2 * K : K;
  if (ldx < width || ldq < K) return GEMM_ERR_INVALID_ARG;
  if (lds < (block_rows == 1 ? M : (K + 127) / 128)) return GEMM_ERR_INVALID_ARG;
  if (M > 0 && K > 0 && (!X || !Q || !S)) return GEMM_ERR_INVALID_ARG;
  if (gemm::misaligned(X, gemm::element_bytes(x_type)) || gemm::misaligned(Q, 16) ||
      gemm::misaligned(S, 4) || (ldq & 15) != 0)
    return GEMM_ERR_MISALIGNED;
  // (a workgroup of 256 for each block: at most 65535 rows of blocks, and fewer than 2^32 threads
  // across a row of them)
  if (block_rows == 128 && ((M + 127) / 128 > 65535 || (K + 127) / 128 >= 2 * gemm::k2G / 256))
    return GEMM_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) return GEMM_OK;
  const gemm::QuantArgs a{X, (uint8_t*)Q, S, M, K, ldx, ldq, lds};
  const int t = gemm::store_of(x_type);
  const hipError_t e =
      block_rows == 1
          ? gemm::launch_quantize_rows(a, t, act == GEMM_ACT_SWIGLU, (hipStream_t)stream)
          : gemm::launch_quantize_blocks(a, t, (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : gemm::hip_fail(e);
}

int gemm_moe_route(int64_t T, int64_t E, int64_t k, const void* X, int64_t ldx, int x_type,
                   const float* bias, int score, int64_t groups, int64_t topk_groups,
                   int group_top, int renorm, float scale, int32_t* ids, float* weights,
                   void* stream) {
  if (T < 0 || E < 1 || k < 1 || groups < 1 || topk_groups < 1) return GEMM_ERR_INVALID_ARG;
  if (!gemm::is_float_type(x_type) || ldx < E) return GEMM_ERR_INVALID_ARG;
  if (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID) return GEMM_ERR_INVALID_ARG;
  if (group_top != 1 && group_top != 2) return GEMM_ERR_INVALID_ARG;
  if (groups > E || E % groups != 0 || topk_groups > groups) return GEMM_ERR_INVALID_ARG;
  if (k > topk_groups * (E / groups)) return GEMM_ERR_INVALID_ARG;
  if (T > 0 && (!X || !ids || !weights)) return GEMM_ERR_INVALID_ARG;
  if (gemm::misaligned(X, gemm::element_bytes(x_type)) || gemm::misaligned(bias, 4) ||
      gemm::misaligned(ids, 4) || gemm::misaligned(weights, 4))
    return GEMM_ERR_MISALIGNED;
  // (64 threads a token: a grid holds fewer than 2^32)
  if (E > 1024 || k > 64 || groups > 64 || T >= (int64_t(1) << 26)) return GEMM_ERR_UNSUPPORTED;
  if (T == 0) return GEMM_OK;
  const gemm::RouteArgs a{X,        bias,     ids,      weights,          T,
                          ldx,      (int)E,   (int)k,   (int)groups,      (int)topk_groups,
                          group_top, score == GEMM_SCORE_SIGMOID, renorm != 0, scale,
                          (int)(E / groups), 1.0f / (float)(E / groups)};
  const hipError_t e = gemm::launch_route(a, gemm::store_of(x_type), (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : gemm::hip_fail(e);
}

int gemm_moe_plan(int64_t T, int64_t k, int64_t E, const int32_t* ids, int32_t* offsets,
                  int32_t* rows, int32_t* pos, void* stream) {
  if (T < 0 || k < 1 || E < 1 || !offsets) return GEMM_ERR_INVALID_ARG;
  if (T > 0 && (!ids || !rows || !pos)) return GEMM_ERR_INVALID_ARG;
  if (gemm::misaligned(ids, 4) || gemm::misaligned(offsets, 4) || gemm::misaligned(rows, 4) ||
      gemm::misaligned(pos, 4))
    return GEMM_ERR_MISALIGNED;
  if (E > 65535 || k >= gemm::k2G / 2 || T >= gemm::k2G / 2 || T * k >= gemm::k2G / 2)
    return GEMM_ERR_UNSUPPORTED;
  const hipError_t e =
      gemm::launch_plan(ids, T, (int)k, (int)E, offsets, rows, pos, (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : gemm::hip_fail(e);
}

int gemm_moe_combine(int64_t T, int64_t k, int64_t N, int64_t R, const void* Y, int64_t ldy,
                     int y_type, const int32_t* pos, const float* weights, void* out, int64_t ldo,
                     int out_type, void* stream) {
  if (T < 0 || k < 0 || N < 0 || R < 0) return GEMM_ERR_INVALID_ARG;
  if (!gemm::is_float_type(y_type) || !gemm::is_float_type(out_type)) return GEMM_ERR_INVALID_ARG;
  if (ldy < N || ldo < N) return GEMM_ERR_INVALID_ARG;
  if (T > 0 && N > 0) {
    if (!out || (k > 0 && (!pos || !weights || (R > 0 && !Y)))) return GEMM_ERR_INVALID_ARG;
  }
  if (gemm::misaligned(Y, gemm::element_bytes(y_type)) || gemm::misaligned(out, 16) ||
      gemm::misaligned(pos, 4) || gemm::misaligned(weights, 4) || (ldo & 7) != 0)
    return GEMM_ERR_MISALIGNED;
  if (T >= gemm::k2G || N >= gemm::k2G || R >= gemm::k2G || k >= gemm::k2G ||
      T * ((N + 7) / 8) >= 2 * gemm::k2G - 256)  // (a grid holds fewer than 2^32 threads)
    return GEMM_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return GEMM_OK;
  const gemm::CombineArgs a{Y, pos, weights, out, T, N, R, ldy, ldo, (int)k};
  const hipError_t e = gemm::launch_combine(a, gemm::store_of(y_type), gemm::store_of(out_type),
                                            (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : gemm::hip_fail(e);
}

}  // extern "C"
