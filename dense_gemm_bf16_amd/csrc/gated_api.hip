// C-ABI front end of the integer products and the gated products: argument
// checks, the choice of kernel shape, launch.  The contract of every entry
// point is stated in include/gemm_bf16.h.  Nothing here allocates or throws.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "../../include/gemm_bf16.h"
#include "gated_launch.hpp"
#include "gemm_internal.h"

namespace gemm {
namespace {

constexpr int64_t k2G = int64_t(1) << 31;
constexpr int64_t kRangeLimit = k2G - 4096;
constexpr int64_t kMaxIntK = 131071;  // 2^14 K stays below 2^31

// ------------------------------------------------------- choice of shape
// As the block products choose theirs: the shape that a model of a launch's
// time makes cheapest.  `units` workgroups on CUs that hold `resident` of them
// each make passes of 256 * resident; a pass costs steps * step + tile (steps:
// K-steps of a workgroup's wave group; tile: first loads and epilogue), a last
// pass with a fraction f of its workgroups, up to n on a CU, part + stair * (n -
// 1) / (resident - 1) + (1 - part - stair) * f of that (without the stair, 256
// workgroups of a shape of which a CU holds four were taken to be 1.4 times as
// slow as 128); the whole takes at least as long as reading B.  Where the last
// pass would be part empty, the columns that fill whole passes may go to one
// shape and the rest to a second launch, if the model finds that 4 % cheaper, 2.5
// us for the launch counted.  (Of 70 products that might, those it finds 7 to 15 %
// cheaper ran 9 % faster, 4 to 7 % 3 %, 2 to 4 % as fast.)
//
// Fitted to 591 products (M 1 to 4096, B from 512 x 1024 to 28672 x 4096 and down
// to 128 bytes deep, integers plain and gated, bf16 gated), each timed in the
// shapes that were in question, with a bf16 output and without keeping g and u;
// the same constants choose for the other outputs and for fp16.  What it chooses
// ran within 1.2 % of the fastest timed (geometric mean; 27 % at worst); the
// eleven of them that are two launches took 2 % less than the fastest single
// shape (12 % less to 9 % more).  gated_model.py holds the same model, the sweep,
// its times and the fit, which gives these constants.
struct Cost {
  float step, tile, part, stair, base;  // us, us, share, share, us
};
struct Shape {
  GatedConfig built;
  int k_groups, resident;
  Cost ints, halves;  // of 8-bit integers, of 16-bit types
};
const Shape kShapes[] = {
#define ROW(NAME, A, B, C, D, E, S, RESIDENT, ...)                                        \
  {{#NAME, A, B, (C) * (D) * (E) * 64, (B) / (D) / 16 % 2 == 0 || (A) / (C) / 16 % 2 == 0, \
    &launch_gated_tile<A, B, C, D, E, S>}, E, RESIDENT, __VA_ARGS__},
    ROW(b256x256, 256, 256, 2, 4, 1, 2, 1,
        {1.453f, 12.12f, 0.65f, 0.00f, 0.00f}, {1.418f, 8.37f, 0.80f, 0.00f, 0.00f})
    ROW(b256x192, 256, 192, 2, 4, 1, 2, 1,
        {1.087f, 10.04f, 0.72f, 0.00f, 0.00f}, {1.155f, 7.06f, 0.72f, 0.00f, 1.29f})
    ROW(b256x128, 256, 128, 4, 2, 1, 3, 1,
        {0.864f, 6.62f, 0.71f, 0.00f, 0.95f}, {0.891f, 4.29f, 0.76f, 0.00f, 1.49f})
    ROW(b128x128, 128, 128, 2, 2, 1, 2, 2,
        {0.963f, 5.41f, 0.46f, 0.24f, 2.44f}, {1.012f, 2.61f, 0.48f, 0.26f, 2.87f})
    ROW(b128x128k2, 128, 128, 2, 2, 2, 2, 1,
        {1.051f, 5.45f, 0.80f, 0.00f, 1.72f}, {1.091f, 4.07f, 0.84f, 0.00f, 1.90f})
    ROW(b64x128k2, 64, 128, 2, 2, 2, 3, 1,
        {0.714f, 3.47f, 0.86f, 0.00f, 1.57f}, {0.761f, 2.45f, 0.85f, 0.00f, 1.94f})
    ROW(b64x64, 64, 64, 2, 2, 1, 4, 2,
        {0.430f, 2.40f, 0.58f, 0.23f, 2.00f}, {0.449f, 1.55f, 0.60f, 0.31f, 2.28f})
    ROW(b64x64k2, 64, 64, 2, 2, 2, 4, 1,
        {0.461f, 2.73f, 0.83f, 0.00f, 1.80f}, {0.471f, 2.33f, 0.87f, 0.00f, 1.99f})
    ROW(b32x128, 32, 128, 1, 4, 1, 3, 2,
        {0.550f, 2.17f, 0.58f, 0.25f, 1.90f}, {0.589f, 1.16f, 0.57f, 0.27f, 2.23f})
    ROW(b32x64k4, 32, 64, 2, 2, 4, 3, 1,
        {0.666f, 3.12f, 0.89f, 0.00f, 1.61f}, {0.699f, 2.92f, 0.88f, 0.00f, 1.86f})
    ROW(b32x32k4, 32, 32, 2, 2, 4, 4, 1,
        {0.425f, 3.00f, 0.95f, 0.00f, 1.15f}, {0, 0, 0, 0, 0})
#undef ROW
#define ROW(NAME, A, B, C, D, E, RESIDENT, ...)                                             \
  {{#NAME, 16 * (A), (E) * (B), (C) * 64, true, &launch_gated_row<A, B, C, D, E>}, C, RESIDENT, \
   __VA_ARGS__},
    ROW(r16x16, 1, 1, 8, 4, 16, 4,
        {3.922f, 0.00f, 0.22f, 0.61f, 2.59f}, {3.725f, 0.25f, 0.25f, 0.70f, 2.52f})
    ROW(r16x8, 1, 1, 8, 4, 8, 4,
        {2.512f, 1.28f, 0.23f, 0.53f, 2.30f}, {2.544f, 1.27f, 0.21f, 0.52f, 2.60f})
    ROW(r32x16, 2, 1, 8, 4, 16, 4,
        {4.322f, 0.00f, 0.25f, 0.49f, 2.55f}, {4.579f, 0.09f, 0.25f, 0.59f, 2.54f})
#undef ROW
};
constexpr double kStreamMBPerUs = 6.3, kStreamBaseUs = 2.2;
constexpr double kSecondLaunchUs = 2.5, kSplitGain = 0.96;

// A product as the choice sees it: rows of A and of B, bytes of a row and from
// row to row, and whether B's rows are paired.
struct Product {
  int64_t M, rows_b, k_bytes, lda, ldb;
  bool gated, ints;
};

int64_t tiles_n(const Shape& s, int64_t rows_b) {
  return (rows_b + s.built.bn - 1) / s.built.bn;
}

// Whether a shape can run rows_b rows of B (see the block products).
bool fits(const Shape& s, const Product& p, int64_t rows_b) {
  if (p.gated && !s.built.gated) return false;
  if (s.built.bn * p.ldb >= kRangeLimit || s.built.bm * p.lda >= kRangeLimit) return false;
  return (p.M + s.built.bm - 1) / s.built.bm * tiles_n(s, rows_b) < 2 * k2G / s.built.threads;
}

double model_time(const Shape& s, const Product& p, int64_t rows_b) {
  const Cost& c = p.ints ? s.ints : s.halves;
  const int64_t units = (p.M + s.built.bm - 1) / s.built.bm * tiles_n(s, rows_b);
  const int64_t pass = 256 * s.resident, rest = units % pass;
  double passes = (double)(units / pass);
  if (rest > 0)
    passes += c.part +
              c.stair * (double)((rest - 1) / 256) / (s.resident > 1 ? s.resident - 1 : 1) +
              (1 - (double)c.part - c.stair) * (double)rest / (double)pass;
  const int64_t k_steps = (p.k_bytes + kStepBytes - 1) / kStepBytes;
  const double steps = (double)((k_steps + s.k_groups - 1) / s.k_groups);
  const double t = passes * (steps * c.step + c.tile) + c.base;
  const double floor_us =
      (double)rows_b * (double)p.k_bytes * 1e-6 / kStreamMBPerUs + kStreamBaseUs;
  return sqrt(sqrt(t * t * t * t + floor_us * floor_us * floor_us * floor_us));
}

const Shape* cheapest(const Product& p, int64_t rows_b, double* time) {
  const Shape* best = nullptr;
  for (const Shape& s : kShapes) {
    if (!fits(s, p, rows_b)) continue;
    const double t = model_time(s, p, rows_b);
    if (best && t >= *time) continue;
    best = &s;
    *time = t;
  }
  return best;
}

// `shape` on the first split_b rows of B (all of them, or those that fill its
// whole passes over the CUs), `tail` on the rest.  No shape: none can.
struct DensePlan {
  const Shape* shape;
  const Shape* tail;
  int64_t split_b;
};

DensePlan choose(const Product& p) {
  double best = 0;
  DensePlan plan{cheapest(p, p.rows_b, &best), nullptr, p.rows_b};
  if (p.M < 1 || !plan.shape) return plan;
  best *= kSplitGain;
  for (const Shape& s : kShapes) {
    const int64_t rows = (p.M + s.built.bm - 1) / s.built.bm, cols = tiles_n(s, p.rows_b);
    const int64_t pass = 256 * s.resident;
    if (rows > pass) continue;
    const int64_t head = rows * cols / pass * pass / rows * s.built.bn / 128 * 128;
    if (head <= 0 || head >= p.rows_b || !fits(s, p, head)) continue;
    const double t1 = model_time(s, p, head);
    if (t1 >= best) continue;
    double t2 = 0;
    const Shape* tail = cheapest(p, p.rows_b - head, &t2);
    if (!tail || t1 + t2 + kSecondLaunchUs >= best) continue;
    best = t1 + t2 + kSecondLaunchUs;
    plan = DensePlan{&s, tail, head};
  }
  return plan;
}

const Shape* shape_named(const char* name) {
  for (const Shape& s : kShapes)
    if (strcmp(s.built.name, name) == 0) return &s;
  return nullptr;
}

bool misaligned(const void* p, int bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }
bool is_float_type(int type) {
  return type == GEMM_TYPE_BF16 || type == GEMM_TYPE_F16 || type == GEMM_TYPE_F32;
}
int store_of(int type) {
  return type == GEMM_TYPE_F32 ? kStoreF32 : type == GEMM_TYPE_F16 ? kStoreF16 : kStoreBf16;
}
int op_of(int type) {
  return type == GEMM_TYPE_I8 ? kOpI8 : type == GEMM_TYPE_F16 ? kOpF16 : kOpBf16;
}
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// C (M x N) of A and B's N rows, or with `gated` H (M x N) of B's 2 N rows.
int dense_product(const char* config, int type, bool gated, int64_t M, int64_t N, int64_t K,
                  const void* A, int64_t lda, const float* SA, const void* B, int64_t ldb,
                  const float* SB, int act, void* C, int64_t ldc, int c_type, void* kept,
                  int64_t ld_kept, void* stream) {
  const bool ints = type == GEMM_TYPE_I8;
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (!ints && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16) return GEMM_ERR_INVALID_ARG;
  if (!is_float_type(c_type) || (!ints && c_type != type)) return GEMM_ERR_INVALID_ARG;
  if (gated && act != GEMM_ACT_SWIGLU && act != GEMM_ACT_GEGLU) return GEMM_ERR_INVALID_ARG;
  if (M >= k2G || N >= (gated ? k2G / 2 : k2G) || K >= k2G / 2 || lda >= k2G || ldb >= k2G ||
      ldc >= (int64_t(1) << 40) || ld_kept >= (int64_t(1) << 40) || (ints && K > kMaxIntK))
    return GEMM_ERR_UNSUPPORTED;
  if (lda < K || ldb < K || ldc < N || (kept && ld_kept < 6 * up16(N))) return GEMM_ERR_INVALID_ARG;
  const bool work = M > 0 && N > 0;
  if (work && (!C || (K > 0 && (!A || !B)) || (ints && (!SA || !SB)))) return GEMM_ERR_INVALID_ARG;
  const int es = ints ? 1 : 2;
  if (misaligned(A, 16) || misaligned(B, 16) || misaligned(C, 16) || misaligned(kept, 16) ||
      misaligned(SA, 4) || misaligned(SB, 4) || ((lda | ldb) & (16 / es - 1)) != 0 ||
      (ldc & 7) != 0 || (kept && (ld_kept & 15) != 0))
    return GEMM_ERR_MISALIGNED;

  const Product p{M, gated ? 2 * N : N, K * es, lda * es, ldb * es, gated, ints};
  DensePlan plan{nullptr, nullptr, p.rows_b};
  if (config && config[0]) {
    plan.shape = shape_named(config);
    if (plan.shape && !fits(*plan.shape, p, p.rows_b)) plan.shape = nullptr;
  } else {
    plan = choose(p);
  }
  if (!plan.shape) return GEMM_ERR_UNSUPPORTED;
  if (!work) return GEMM_OK;

  BlockArgs a{};
  a.A = (const uint8_t*)A;
  a.B = (const uint8_t*)B;
  a.C = C;
  a.SA = SA;
  a.SB = SB;
  a.lda = p.lda;
  a.ldb = p.ldb;
  a.ldc = ldc;
  a.M = (int32_t)M;
  a.kbytes = (int32_t)p.k_bytes;
  a.a_rows = (int32_t)M;
  a.E = 1;
  a.k_steps = (int32_t)((p.k_bytes + kStepBytes - 1) / kStepBytes);
  a.group_m = 4;
  if (gated) {
    a.up_b = N * p.ldb;
    a.up_sb = N;
    a.kept = (uint8_t*)kept;
    a.ld_kept = ld_kept;
    a.kept_f = up16(N);
    a.geglu = act == GEMM_ACT_GEGLU;
  }
  auto launch = [&](const Shape& s, int64_t rows_b) {
    const int64_t row_tiles = (M + s.built.bm - 1) / s.built.bm;
    a.N = (int32_t)(gated ? rows_b / 2 : rows_b);
    a.tiles_n = (int32_t)tiles_n(s, rows_b);
    a.row_tiles = (int32_t)row_tiles;
    // Rows of a power-of-two stride would send all workgroups to the same
    // memory channels: tile column j starts 3 j K-steps in where one row of
    // tiles reads all of B (see the block products), j where several share B
    // and its rows lie whole pages of 4 KB apart (bf16: 64, 128, 256 rows by
    // 8192 x 8192 37.4, 44.0, 58.3 us without, 33.5, 40.0, 55.5 with, 4096^3
    // 107.7, 101.9; integers: 4096^3 64.8, 59.5; larger ones level, and with
    // other strides 0-2 % slower).
    a.k_rot = row_tiles == 1 ? 3 : p.ldb % 4096 == 0 ? 1 : 0;
    return s.built.launch(a, (int)(row_tiles * a.tiles_n), (hipStream_t)stream, op_of(type),
                          store_of(c_type), gated, row_tiles == 1);
  };
  hipError_t e = launch(*plan.shape, plan.split_b);
  if (e == hipSuccess && plan.tail) {
    const int64_t col = gated ? plan.split_b / 2 : plan.split_b;
    a.B += col * p.ldb;
    if (SB) a.SB += col;
    a.C = (uint8_t*)C + col * (c_type == GEMM_TYPE_F32 ? 4 : 2);
    a.kept_first = (int32_t)col;
    e = launch(*plan.tail, p.rows_b - plan.split_b);
  }
  return e == hipSuccess ? GEMM_OK : hip_fail(e);
}

thread_local char g_plan_name[64];

const char* plan_name(int type, bool gated, int64_t M, int64_t N, int64_t K) {
  const bool ints = type == GEMM_TYPE_I8;
  if (M < 0 || N < 0 || K < 0 || M >= k2G || N >= (gated ? k2G / 2 : k2G) || K >= k2G / 2 ||
      (ints && K > kMaxIntK) || (!ints && type != GEMM_TYPE_BF16 && type != GEMM_TYPE_F16))
    return "invalid";
  const DensePlan p = choose(Product{M, gated ? 2 * N : N, ints ? K : 2 * K, 0, 0, gated, ints});
  if (!p.shape) return "invalid";
  if (!p.tail) return p.shape->built.name;
  snprintf(g_plan_name, sizeof g_plan_name, "%s+%s", p.shape->built.name, p.tail->built.name);
  return g_plan_name;
}

}  // namespace
}  // namespace gemm

extern "C" {

int gemm_i8_ex(const char* config, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
               const float* SA, const void* B, int64_t ldb, const float* SB, void* C, int64_t ldc,
               int c_type, void* stream) {
  return gemm::dense_product(config, GEMM_TYPE_I8, false, M, N, K, A, lda, SA, B, ldb, SB,
                             GEMM_ACT_NONE, C, ldc, c_type, nullptr, 0, stream);
}

int gemm_i8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* SA,
            const void* B, int64_t ldb, const float* SB, void* C, int64_t ldc, int c_type,
            void* stream) {
  return gemm_i8_ex(nullptr, M, N, K, A, lda, SA, B, ldb, SB, C, ldc, c_type, stream);
}

int gemm_i8_gated_ex(const char* config, int64_t M, int64_t F, int64_t K, const void* A,
                     int64_t lda, const float* SA, const void* W, int64_t ldw, const float* SW,
                     int act, void* H, int64_t ldh, int h_type, void* stream) {
  return gemm::dense_product(config, GEMM_TYPE_I8, true, M, F, K, A, lda, SA, W, ldw, SW, act, H,
                             ldh, h_type, nullptr, 0, stream);
}

int gemm_i8_gated(int64_t M, int64_t F, int64_t K, const void* A, int64_t lda, const float* SA,
                  const void* W, int64_t ldw, const float* SW, int act, void* H, int64_t ldh,
                  int h_type, void* stream) {
  return gemm_i8_gated_ex(nullptr, M, F, K, A, lda, SA, W, ldw, SW, act, H, ldh, h_type, stream);
}

int gemm_gated_ex(const char* config, int type, int64_t M, int64_t F, int64_t K, const void* X,
                  int64_t ldx, const void* W, int64_t ldw, int act, void* H, int64_t ldh, void* kept,
                  int64_t ld_kept, void* stream) {
  if (type == GEMM_TYPE_I8) return GEMM_ERR_INVALID_ARG;
  return gemm::dense_product(config, type, true, M, F, K, X, ldx, nullptr, W, ldw, nullptr, act, H,
                             ldh, type, kept, ld_kept, stream);
}

int gemm_gated(int type, int64_t M, int64_t F, int64_t K, const void* X, int64_t ldx,
               const void* W, int64_t ldw, int act, void* H, int64_t ldh, void* kept, int64_t ld_kept,
               void* stream) {
  return gemm_gated_ex(nullptr, type, M, F, K, X, ldx, W, ldw, act, H, ldh, kept, ld_kept, stream);
}

size_t gemm_gated_kept_row(int64_t F) {
  return F < 0 || F >= gemm::k2G / 2 ? 0 : (size_t)(6 * gemm::up16(F));
}

const char* gemm_i8_config_name(int64_t M, int64_t N, int64_t K) {
  return gemm::plan_name(GEMM_TYPE_I8, false, M, N, K);
}

const char* gemm_i8_config_at(int i) {
  const int n = (int)(sizeof gemm::kShapes / sizeof *gemm::kShapes);
  return i >= 0 && i < n ? gemm::kShapes[i].built.name : nullptr;
}

const char* gemm_gated_config_name(int type, int64_t M, int64_t F, int64_t K) {
  return gemm::plan_name(type, true, M, F, K);
}

int gemm_i8_quantize(int64_t M, int64_t K, const void* X, int64_t ldx, int x_type, void* Q,
                     int64_t ldq, float* S, void* stream) {
  if (M < 0 || K < 0 || !gemm::is_float_type(x_type)) return GEMM_ERR_INVALID_ARG;
  // (a workgroup of up to 1024 a row: a grid holds fewer than 2^32 threads)
  if (K >= gemm::k2G || M >= 2 * gemm::k2G / 1024 || ldx >= (int64_t(1) << 40) ||
      ldq >= (int64_t(1) << 40))
    return GEMM_ERR_UNSUPPORTED;
  if (ldx < K || ldq < K) return GEMM_ERR_INVALID_ARG;
  if (M > 0 && (!S || (K > 0 && (!X || !Q)))) return GEMM_ERR_INVALID_ARG;
  if (gemm::misaligned(X, x_type == GEMM_TYPE_F32 ? 4 : 2) || gemm::misaligned(Q, 16) ||
      gemm::misaligned(S, 4) || (ldq & 15) != 0)
    return GEMM_ERR_MISALIGNED;
  if (M == 0) return GEMM_OK;
  const gemm::Int8QuantArgs a{X, (uint8_t*)Q, S, M, K, ldx, ldq};
  const hipError_t e = gemm::launch_quantize_int8(a, gemm::store_of(x_type), (hipStream_t)stream);
  return e == hipSuccess ? GEMM_OK : gemm::hip_fail(e);
}

}  // extern "C"
