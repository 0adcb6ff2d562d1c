// Routing to experts: the top-k experts of each token, and the plan that
// sorts (token, slot) pairs by expert.
//
// Routing, per token with logits x:
//   s  = softmax(x) or sigmoid(x)
//   c  = s + bias                      (the order of choice)
//   a group's score = its largest c, or the sum of its two largest; the
//   topk_groups best groups stay
//   ids = the k largest c of those groups, equal values by lowest index
//   w  = s[ids], divided by their sum if renorm, times scale
//
// The order of choice is that of the exact values.  Without a bias it is the
// order of the logits (both scores grow with x), which needs no arithmetic.
// With one, c is computed in fp32 with a bound on its error; where two
// neighbours that matter lie closer than the bound (a fraction of a percent
// of the rows of ordinary logits), the wave decides its row again in fp64.
//
// One wave per token.  A group's experts are dealt over 64 / (groups rounded
// up to a power of two) neighbouring lanes, so a group's best two and its
// score stay within those lanes, and the k rounds of a maximum over the wave
// cost six DPP steps each.
#include "block_internal.h"

namespace gemm {
namespace {

template <int TYPE>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  float v;
  if constexpr (TYPE == kStoreF32) v = ((const float*)p)[i];
  else if constexpr (TYPE == kStoreF16) v = (float)((const _Float16*)p)[i];
  else v = (float)((const __bf16*)p)[i];
  // NaN counts as -infinity, +infinity as the largest finite number
  v = v != v ? -INFINITY : v;
  return fminf(v, 3.402823466e38f);
}

// Largest value over the wave's lanes (unsigned), by row shifts within 16
// lanes and two broadcasts across rows; lane 63 ends with it.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111>(v);  // row_shr 1
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);  // row_bcast 15
  v = dpp_max<0x143>(v);  // row_bcast 31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Keys: unsigned integers in the order of the floating-point values they
// stand for; 0 is below the key of every value (-infinity included).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);  // -0 counts as 0
  return b ^ ((int32_t)b < 0 ? ~0u : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((int32_t)k < 0 ? 0x80000000u : ~0u));
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return b ^ ((int64_t)b < 0 ? ~0ull : 1ull << 63);
}

// Bounds on the error of a difference of two c (of two group scores) in
// fp32.  expf is off by at most 2 ulp, the sum over up to 32 values a lane
// and 6 steps by 38 half ulps, the division and c's own sum by half an ulp
// each: s is off by less than 2^-18.5 (s <= 1), c by that and 2^-24 |c|.
__device__ __forceinline__ float choice_bound(float c) { return 0x1p-17f + 0x1p-21f * fabsf(c); }
__device__ __forceinline__ float group_bound(float g) { return 0x1p-16f + 0x1p-20f * fabsf(g); }

struct Lane {
  int lane, group, sub, per;  // per: lanes of a group; sub: this lane's place among them
  int size;                   // experts of a group
  __device__ __forceinline__ bool has(int j, int groups) const {
    return group < groups && sub + j * per < size;
  }
  __device__ __forceinline__ int expert(int j) const { return group * size + sub + j * per; }
};

// Whether this lane's group is among the best topk_groups.  F: float or
// double.  `near` is set where fp32 cannot tell.
template <typename F>
__device__ __forceinline__ bool group_stays(const RouteArgs& a, const Lane& l, F best, F second,
                                            bool& near) {
  // the two largest over the group's lanes
  for (int d = 1; d < l.per; d *= 2) {
    const F b = __shfl_xor(best, d, 64), s = __shfl_xor(second, d, 64);
    const F low = best < b ? best : b;
    best = best < b ? b : best;
    second = second < s ? s : second;
    second = second < low ? low : second;
  }
  const F g = a.group_top == 2 && l.size > 1 ? best + second : best;
  int rank = 0;
  F next = -INFINITY;  // the largest score of a group ranked below this one
  for (int o = 0; o < a.groups; ++o) {
    const F v = __shfl(g, o * l.per, 64);
    const bool above = o != l.group && (v > g || (v == g && o < l.group));
    rank += above ? 1 : 0;
    if (!above && o != l.group && v > next) next = v;
  }
  const bool stays = l.group < a.groups && rank < a.topk_groups;
  if constexpr (sizeof(F) == 4) {
    const bool last = l.group < a.groups && rank == a.topk_groups - 1;
    near = __any(last && !(g - next > group_bound(g)));
  }
  return stays;
}

// Rounds of the largest key among the wave's lanes.  WIDE: 64-bit keys, else
// only the high words.  Returns false (fp32 keys, CHECK) if two neighbours
// in the order are closer than their bound.
template <int VPL, bool WIDE, bool CHECK>
__device__ __forceinline__ bool choose(const RouteArgs& a, const Lane& l, uint32_t (&hi)[VPL],
                                       uint32_t (&lo)[VPL], int& my_id) {
  auto local = [&](uint32_t& bh, uint32_t& bl, int& be) __attribute__((always_inline)) {
    bh = hi[0];
    bl = WIDE ? lo[0] : 0;
    be = l.expert(0);
#pragma unroll
    for (int j = 1; j < VPL; ++j) {
      const bool more = hi[j] > bh || (WIDE && hi[j] == bh && lo[j] > bl);
      bh = more ? hi[j] : bh;
      if constexpr (WIDE) bl = more ? lo[j] : bl;
      be = more ? l.expert(j) : be;
    }
  };
  uint32_t bh, bl;
  int be;
  local(bh, bl, be);
  float before = 0.0f;
  const int rounds = CHECK ? a.k + 1 : a.k;
  for (int r = 0; r < rounds; ++r) {
    const uint32_t mh = wave_max(bh);
    uint64_t tied = __ballot(bh == mh);
    if constexpr (WIDE) {
      const uint32_t ml = wave_max(bh == mh ? bl : 0u);
      tied = __ballot(bh == mh && bl == ml);
    }
    if constexpr (CHECK) {
      if (mh == 0) return true;  // every candidate is taken
      const float c = of_key(mh);
      if (r > 0 && !(before - c > choice_bound(before))) return false;
      before = c;
      if (r == a.k) return true;
    }
    int w = __builtin_ctzll(tied);
    if ((tied & (tied - 1)) != 0) {  // equal values: the lowest expert
      const bool in = (tied >> l.lane) & 1;
      const uint32_t least = ~wave_max(in ? ~(uint32_t)be : 0u);
      w = __builtin_ctzll(__ballot(in && (uint32_t)be == least));
    }
    const int id = __builtin_amdgcn_readlane(be, w);
    if (l.lane == r) my_id = id;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (l.lane == w && l.expert(j) == id) {
        hi[j] = 0;
        if constexpr (WIDE) lo[j] = 0;
      }
    local(bh, bl, be);
  }
  return true;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
  return v;
}

template <int TYPE, int VPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  Lane l;
  l.lane = threadIdx.x & 63;
  const int g2 = a.groups <= 1 ? 1 : 1 << (32 - __builtin_clz(a.groups - 1));
  l.per = 64 / g2;
  l.group = l.lane / l.per;
  l.sub = l.lane - l.group * l.per;
  l.size = a.E / a.groups;

  float x[VPL], b[VPL];
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    x[j] = -INFINITY;
    b[j] = 0.0f;
    if (l.has(j, a.groups)) {
      x[j] = logit<TYPE>(a.x, t * a.ldx + l.expert(j));
      if (a.bias) b[j] = logit<kStoreF32>(a.bias, l.expert(j));
    }
    m = fmaxf(m, x[j]);
  }
  float z = 1.0f;
  if (!a.sigmoid) {
    m = of_key(wave_max(key_of(m)));
    if (m == -INFINITY) m = 0.0f;  // every logit is masked: every score is 0
    z = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) z += expf(x[j] - m);
    z = wave_sum(z);
    z = z > 0.0f ? z : 1.0f;
  }
  auto score = [&](float v) __attribute__((always_inline)) {
    return a.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - m) / z;
  };

  const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
  uint32_t hi[VPL], lo[VPL];
  int my_id = 0;
  bool done;
  {
    float c[VPL];
    float best = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      c[j] = by_logit ? x[j] : score(x[j]) + b[j];
      if (!l.has(j, a.groups)) c[j] = -INFINITY;
      second = fmaxf(second, fminf(best, c[j]));
      best = fmaxf(best, c[j]);
    }
    bool stays = true, near = false;
    if (a.topk_groups < a.groups) stays = group_stays<float>(a, l, best, second, near);
#pragma unroll
    for (int j = 0; j < VPL; ++j) hi[j] = stays && l.has(j, a.groups) ? key_of(c[j]) : 0u;
    if (by_logit) {
      // (a tie between groups is one between logits: the lowest index)
      done = choose<VPL, false, false>(a, l, hi, lo, my_id);
    } else {
      done = !near && choose<VPL, false, true>(a, l, hi, lo, my_id);
    }
  }
  if (!done) {
    double c[VPL];
    double best = -INFINITY, second = -INFINITY, zz = 1.0;
    if (!a.sigmoid) {
      zz = 0.0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) zz += exp((double)x[j] - (double)m);
      zz = wave_sum(zz);
      zz = zz > 0.0 ? zz : 1.0;
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      c[j] = (a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[j])) : exp((double)x[j] - (double)m) / zz) +
             (double)b[j];
      if (!l.has(j, a.groups)) c[j] = -INFINITY;
      second = fmax(second, fmin(best, c[j]));
      best = fmax(best, c[j]);
    }
    bool stays = true, near = false;
    if (a.topk_groups < a.groups) stays = group_stays<double>(a, l, best, second, near);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const uint64_t k = stays && l.has(j, a.groups) ? key_of(c[j]) : 0ull;
      hi[j] = (uint32_t)(k >> 32);
      lo[j] = (uint32_t)k;
    }
    choose<VPL, true, false>(a, l, hi, lo, my_id);
  }

  float w = 0.0f;
  if (l.lane < a.k) w = score(logit<TYPE>(a.x, t * a.ldx + my_id));
  if (a.renorm) {
    const float sum = wave_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  if (l.lane < a.k) {
    a.ids[t * a.k + l.lane] = my_id;
    a.weights[t * a.k + l.lane] = w * a.scale;
  }
}

template <int TYPE>
hipError_t route_of(const RouteArgs& a, hipStream_t s) {
  int g2 = 1;
  while (g2 < a.groups) g2 *= 2;
  const int per = 64 / g2, size = a.E / a.groups;
  const int vpl = (size + per - 1) / per;
  const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
  if (vpl <= 1) hipLaunchKernelGGL((route_kernel<TYPE, 1>), grid, block, 0, s, a);
  else if (vpl <= 2) hipLaunchKernelGGL((route_kernel<TYPE, 2>), grid, block, 0, s, a);
  else if (vpl <= 4) hipLaunchKernelGGL((route_kernel<TYPE, 4>), grid, block, 0, s, a);
  else if (vpl <= 8) hipLaunchKernelGGL((route_kernel<TYPE, 8>), grid, block, 0, s, a);
  else if (vpl <= 16) hipLaunchKernelGGL((route_kernel<TYPE, 16>), grid, block, 0, s, a);
  else if (vpl <= 32) hipLaunchKernelGGL((route_kernel<TYPE, 32>), grid, block, 0, s, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

// A stable counting sort of the R = T * k ids, one workgroup per expert and
// one more for the slots whose id names no expert: each reads every id twice
// (they stay in L2), first to count the ids below its own, which is where
// its rows start, then to place its own in their order.  One launch, no
// atomics, so the order never depends on timing.  Each wave takes a
// contiguous part of the ids, 256 at a time (four neighbours a lane), so the
// waves meet once.
typedef int i32x4u __attribute__((ext_vector_type(4), aligned(4)));

template <int W>
__global__ __launch_bounds__(W * 64) void plan_kernel(const int32_t* __restrict__ ids, int R, int k,
                                                      int E, int32_t* __restrict__ offsets,
                                                      int32_t* __restrict__ rows,
                                                      int32_t* __restrict__ pos) {
  __shared__ int below_of[W], own_of[W];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t e = blockIdx.x;
  const int part = ((R + W - 1) / W + 255) / 256 * 256;
  const int begin = min((int64_t)wave * part, (int64_t)R), end = min((int64_t)begin + part, (int64_t)R);
  // this lane's four ids from i on: an id that names no expert (negative
  // ones are large unsigned) counts as E, a place past the part as E + 1
  auto four = [&](int i, uint32_t (&v)[4]) __attribute__((always_inline)) {
    if (i + 4 <= end) {
      const i32x4u q = *(const i32x4u*)(ids + i);
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = min((uint32_t)q[u], (uint32_t)E);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = i + u < end ? min((uint32_t)ids[i + u], (uint32_t)E) : (uint32_t)E + 1;
    }
  };
  int below = 0, own = 0;
#pragma unroll 4
  for (int i = begin; i < end; i += 256) {
    uint32_t v[4];
    four(i + lane * 4, v);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      below += v[u] < e ? 1 : 0;
      own += v[u] == e ? 1 : 0;
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    below += __shfl_xor(below, d, 64);
    own += __shfl_xor(own, d, 64);
  }
  if (lane == 0) {
    below_of[wave] = below;
    own_of[wave] = own;
  }
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) at += below_of[w] + (w < wave ? own_of[w] : 0);
  if (wave == 0 && lane == 0) offsets[e] = at;
  if (own == 0) return;
#pragma unroll 2
  for (int i = begin; i < end; i += 256) {
    uint32_t v[4];
    four(i + lane * 4, v);
    int p = at;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint64_t mine = __ballot(v[u] == e);
      p += (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mine >> 32),
                                          __builtin_amdgcn_mbcnt_lo((uint32_t)mine, 0u));
      at += __popcll(mine);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v[u] == e) {
        const int slot = i + lane * 4 + u;
        rows[p] = e < (uint32_t)E ? slot / k : -1;
        pos[slot] = e < (uint32_t)E ? p : -1;
        ++p;
      }
  }
}

// out[t] = sum over slots j of w[t,j] Y[pos[t,j]], in fp32 in the order of
// the slots.  Eight columns a thread, Y's rows
// starting at any element; a slot whose pos lies outside Y
// (dropped) adds nothing.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef __bf16 bf16x8u __attribute__((ext_vector_type(8), aligned(2)));

template <int YT, int OT>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t chunks = (a.N + 7) / 8;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= a.T * chunks) return;
  const int64_t t = idx / chunks;
  const int64_t n = (idx - t * chunks) * 8;
  float acc[8] = {};
  for (int j = 0; j < a.k; ++j) {
    const int p = a.pos[t * a.k + j];
    if (p < 0 || p >= a.R) continue;
    const float w = a.w[t * a.k + j];
    float v[8];
    if (n + 8 <= a.N) {
      if constexpr (YT == kStoreF32) {
        const float* y = (const float*)a.Y + (int64_t)p * a.ldy + n;
        const f32x4 lo = *(const f32x4u*)y, hi = *(const f32x4u*)(y + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = lo[i];
          v[4 + i] = hi[i];
        }
      } else {
        using V = std::conditional_t<YT == kStoreF16, f16x8u, bf16x8u>;
        const V y = *(const V*)((const uint16_t*)a.Y + (int64_t)p * a.ldy + n);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)y[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t at = (int64_t)p * a.ldy + n + i;
        v[i] = 0.0f;
        if (n + i < a.N) {
          if constexpr (YT == kStoreF32) v[i] = ((const float*)a.Y)[at];
          else if constexpr (YT == kStoreF16) v[i] = (float)((const _Float16*)a.Y)[at];
          else v[i] = (float)((const __bf16*)a.Y)[at];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x4 q = {acc[4 * h], acc[4 * h + 1], acc[4 * h + 2], acc[4 * h + 3]};
    if (OT == kStoreF32) {
      float* o = (float*)a.out + t * a.ldo + n + 4 * h;
      if (n + 4 * h + 4 <= a.N) {
        *(f32x4*)o = q;
      } else {
        for (int i = 0; i < 4; ++i)
          if (n + 4 * h + i < a.N) o[i] = q[i];
      }
    } else {
      const u32x2 p = pack_quad<OT>(q);
      uint16_t* o = (uint16_t*)a.out + t * a.ldo + n + 4 * h;
      if (n + 4 * h + 4 <= a.N) {
        *(u32x2*)o = p;
      } else {
        for (int i = 0; i < 4; ++i)
          if (n + 4 * h + i < a.N) o[i] = (uint16_t)(p[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
}

template <int YT>
hipError_t combine_of(const CombineArgs& a, int out_type, hipStream_t s) {
  const int64_t blocks = (a.T * ((a.N + 7) / 8) + 255) / 256;
  if (blocks >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(256);
  switch (out_type) {
    case kStoreBf16: hipLaunchKernelGGL((combine_kernel<YT, kStoreBf16>), grid, block, 0, s, a); break;
    case kStoreF16: hipLaunchKernelGGL((combine_kernel<YT, kStoreF16>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((combine_kernel<YT, kStoreF32>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int x_type, hipStream_t s) {
  switch (x_type) {
    case kStoreBf16: return route_of<kStoreBf16>(a, s);
    case kStoreF16: return route_of<kStoreF16>(a, s);
    default: return route_of<kStoreF32>(a, s);
  }
}

hipError_t launch_plan(const int32_t* ids, int64_t T, int k, int E, int32_t* offsets,
                       int32_t* rows, int32_t* pos, hipStream_t s) {
  const int R = (int)(T * k);
  if (R <= 4096)
    hipLaunchKernelGGL(plan_kernel<4>, dim3(E + 1), dim3(256), 0, s, ids, R, k, E, offsets, rows, pos);
  else
    hipLaunchKernelGGL(plan_kernel<16>, dim3(E + 1), dim3(1024), 0, s, ids, R, k, E, offsets, rows, pos);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, int y_type, int out_type, hipStream_t s) {
  switch (y_type) {
    case kStoreBf16: return combine_of<kStoreBf16>(a, out_type, s);
    case kStoreF16: return combine_of<kStoreF16>(a, out_type, s);
    default: return combine_of<kStoreF32>(a, out_type, s);
  }
}

}  // namespace gemm
