// Routing to experts: the top-k experts of each token, and the plan that
// sorts (token, slot) pairs by expert.
//
// Routing, per token with logits x:
//   s  = softmax(x) or sigmoid(x)
//   c  = s + bias                      (the order of choice; -infinity for a
//                                       masked expert, whatever its bias)
//   a group's score = its largest c, or the sum of its two largest; the
//   topk_groups best groups stay
//   ids = the k largest c of those groups, equal values by lowest index
//   w  = s[ids], divided by their sum if renorm, times scale
//
// Without a bias (and by a group's largest c) the order of choice is the
// order of the logits (both scores grow with x), which needs no arithmetic.
// Otherwise it is that of c in fp64: c is computed in fp32 with a bound on
// its error, and where two neighbours that matter lie closer than the bound
// (a fraction of a percent of the rows of ordinary logits), the wave decides
// its row again in fp64.  What is equal there too (sigmoids of 40 and 50 are
// both 1) goes by the logits, and only then by index.  c in fp64 never falls
// as x grows (exp, the sums and the quotient round the same way for every
// expert), so experts of equal bias always stand in the order of their
// logits, and a bias of zeros leaves every choice as it was without one.
//
// One wave per token.  A group's experts are dealt over 64 / (groups rounded
// up to a power of two) neighbouring lanes, so a group's best two and its
// score stay within those lanes, and the k rounds of a maximum over the wave
// cost six DPP steps each.  Bound by instructions (about 35 a round, and as
// many again for the scores, the groups and the weights): 14-15 us for 8192
// tokens of 256 experts, k = 8, with bias and groups, against 2 us for the
// bytes (8 us without a bias; 38 us at 1024 experts); a wave by itself takes 4
// us, 8 at 1024 experts.  Of that the fp64 rounds' ties by logit cost 4 % (10
// % at 1024), the masks and the weights in fp64 where they are needed nothing
// that shows.
#include "block_internal.h"

namespace gemm {
namespace {

// A logit (or bias) as it counts: NaN as -infinity, +infinity as the largest
// finite number.
__device__ __forceinline__ float logit(float v) {
  v = v != v ? -INFINITY : v;
  return fminf(v, 3.402823466e38f);
}

// v of the lane that differs from this one in bit D of its number, within
// groups whose lanes already agree below that bit (so a mirror serves as the
// swap of halves): vector operations only, no trip through LDS.
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if constexpr (D == 1) return __builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true);  // quad 1,0,3,2
  else if constexpr (D == 2) return __builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true);  // quad 2,3,0,1
  else if constexpr (D == 4) return __builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true);  // half mirror
  else if constexpr (D == 8) return __builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true);  // mirror
  else if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? r[0] : r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32) ? r[0] : r[1];
  }
}
template <int D>
__device__ __forceinline__ float across(float v) {
  return __builtin_bit_cast(float, across<D>(__builtin_bit_cast(uint32_t, v)));
}
template <int D>
__device__ __forceinline__ double across(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)across<D>((uint32_t)(b >> 32)) << 32 | across<D>((uint32_t)b));
}

// Calls f for D = 1, 2, .., below `lanes` (a power of two, the same in all
// lanes).
template <typename F>
__device__ __forceinline__ void butterfly(int lanes, F&& f) {
  if (lanes > 1) f(std::integral_constant<int, 1>{});
  if (lanes > 2) f(std::integral_constant<int, 2>{});
  if (lanes > 4) f(std::integral_constant<int, 4>{});
  if (lanes > 8) f(std::integral_constant<int, 8>{});
  if (lanes > 16) f(std::integral_constant<int, 16>{});
  if (lanes > 32) f(std::integral_constant<int, 32>{});
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
  int log_per;                // per = 1 << log_per
  __device__ __forceinline__ bool has(int j, int groups) const {
    return group < groups && sub + j * per < size;
  }
  __device__ __forceinline__ int expert(int j) const { return group * size + sub + j * per; }
};

// v of lane n (the same n in all lanes).
__device__ __forceinline__ float of_lane(float v, int n) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), n));
}
__device__ __forceinline__ double of_lane(double v, int n) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, n);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), n);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Whether this lane's group is among the best topk_groups.  F: float or
// double.  `near` is set where fp32 cannot tell; in fp64 equal scores go by
// `top`, the logit of the group's best expert, then by index.
template <typename F>
__device__ __forceinline__ bool group_stays(const RouteArgs& a, const Lane& l, F best, F second,
                                            float top, bool& near) {
  constexpr bool kTop = sizeof(F) == 8;
  // the two largest over the group's lanes
  butterfly(l.per, [&](auto dc) __attribute__((always_inline)) {
    constexpr int D = decltype(dc)::value;
    const F b = across<D>(best), s = across<D>(second);
    if constexpr (kTop) {
      const float t = across<D>(top);
      top = (b > best) | ((b == best) & (t > top)) ? t : top;
    }
    const F low = best < b ? best : b;
    best = best < b ? b : best;
    second = second < s ? s : second;
    second = second < low ? low : second;
  });
  // (a second one that is masked, or not there, does not count)
  const F g = a.group_top == 2 && second > -INFINITY ? best + second : best;
  int rank = 0;
  F next = -INFINITY;  // the largest score of a group ranked below this one
  for (int o = 0; o < a.groups; ++o) {
    const F v = of_lane(g, o * l.per);
    // (& and |: no branches)
    bool first = o < l.group;
    if constexpr (kTop) {
      const float t = of_lane(top, o * l.per);
      first = (t > top) | ((t == top) & first);
    }
    const bool above = (v > g) | ((v == g) & first);
    rank += above ? 1 : 0;
    const bool below = !above & (o != l.group) & (v > next);
    next = below ? v : next;
  }
  const bool stays = l.group < a.groups && rank < a.topk_groups;
  if constexpr (sizeof(F) == 4) {
    const bool last = l.group < a.groups && rank == a.topk_groups - 1;
    near = __any(last && !(g - next > group_bound(g)));
  }
  return stays;
}

// Rounds of the largest key among the wave's lanes.  WIDE: 64-bit keys, equal
// ones by logit (this lane's j-th at own[j * 64], read only where keys are
// equal), else only the high words.  Up to kSortedVpl keys a lane are sorted
// first, so that a round looks at each lane's first one only and a taken key
// moves the rest up; more are searched again each round (k = 8, 8192 tokens,
// sorted against searched: 10.7 and 12.4 us at 256 experts, 4 a lane; 18.5 and
// 19.9 at 512; 39.4 and 34.6 at 1024, 16 a lane).  Returns false (fp32 keys,
// CHECK) if two neighbours in the order are closer than their bound.
constexpr int kSortedVpl = 8;
template <int VPL, bool WIDE, bool CHECK>
__device__ __forceinline__ bool choose(const RouteArgs& a, const Lane& l, uint32_t (&hi)[VPL],
                                       uint32_t (&lo)[VPL], const float* own, int& my_id) {
  constexpr bool kSorted = VPL <= kSortedVpl;
  // in the order of this lane's experts of equal key
  auto tie = [&](int id) __attribute__((always_inline)) {
    const uint32_t logit = key_of(own[((id - l.expert(0)) >> l.log_per) * 64]);
    return (uint64_t)logit << 32 | ~(uint32_t)id;
  };
  int id[VPL];  // (of sorted keys)
  if constexpr (kSorted) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) id[j] = l.expert(j);
    // Batcher's odd-even merges; equal keys by lowest expert
#pragma unroll
    for (int p = 1; p < VPL; p *= 2)
#pragma unroll
      for (int q = p; q >= 1; q /= 2)
#pragma unroll
        for (int j = q % p; j + q < VPL; j += 2 * q)
#pragma unroll
          for (int i = 0; i < q; ++i) {
            const int x = i + j, y = i + j + q;
            if (y >= VPL || x / (2 * p) != y / (2 * p)) continue;
            bool swap;
            if constexpr (WIDE) {
              swap = hi[y] > hi[x] || (hi[y] == hi[x] && lo[y] > lo[x]);
              if (hi[y] == hi[x] && lo[y] == lo[x] && hi[x] != 0) swap = tie(id[y]) > tie(id[x]);
            } else {
              swap = ((uint64_t)hi[y] << 32 | ~(uint32_t)id[y]) >
                     ((uint64_t)hi[x] << 32 | ~(uint32_t)id[x]);
            }
            const uint32_t h = hi[x];
            hi[x] = swap ? hi[y] : h;
            hi[y] = swap ? h : hi[y];
            const int e = id[x];
            id[x] = swap ? id[y] : e;
            id[y] = swap ? e : id[y];
            if constexpr (WIDE) {
              const uint32_t w = lo[x];
              lo[x] = swap ? lo[y] : w;
              lo[y] = swap ? w : lo[y];
            }
          }
  }
  uint32_t my_key = 0, last = 0;
  const int rounds = CHECK ? a.k + 1 : a.k;
  for (int r = 0; r < rounds; ++r) {
    uint32_t bh = hi[0], bl = WIDE ? lo[0] : 0;
    int be = kSorted ? id[0] : l.expert(0);
    if constexpr (!kSorted) {
#pragma unroll
      for (int j = 1; j < VPL; ++j) {
        const bool more = hi[j] > bh || (WIDE && hi[j] == bh && lo[j] > bl);
        bh = more ? hi[j] : bh;
        if constexpr (WIDE) bl = more ? lo[j] : bl;
        be = more ? l.expert(j) : be;
      }
    }
    const uint32_t mh = wave_max(bh);
    if (CHECK && r == a.k) {
      last = mh;
      break;
    }
    uint64_t tied = __ballot(bh == mh);
    if constexpr (WIDE) {
      const uint32_t ml = wave_max(bh == mh ? bl : 0u);
      const bool in = bh == mh && bl == ml;
      tied = __ballot(in);
      uint64_t once = 0, twice = 0;  // lanes that have the high word so often
      if constexpr (!kSorted) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const uint64_t has = __ballot(hi[j] == mh);
          twice |= once & has;
          once |= has;
        }
      }
      if ((tied & (tied - 1)) != 0 || twice != 0) {  // equal values: the largest logit
        if constexpr (!kSorted) {
#pragma unroll
          for (int j = 0; j < VPL; ++j)
            if (in && hi[j] == mh && lo[j] == ml && tie(l.expert(j)) > tie(be)) be = l.expert(j);
        }
        const uint32_t bt = in ? (uint32_t)(tie(be) >> 32) : 0u;
        const uint32_t mt = wave_max(bt);  // (with all lanes active)
        tied = __ballot(in && bt == mt);
      }
    }
    int w = __builtin_ctzll(tied);
    if ((tied & (tied - 1)) != 0) {  // equal values: the lowest expert
      const bool in = (tied >> l.lane) & 1;
      const uint32_t least = ~wave_max(in ? ~(uint32_t)be : 0u);
      w = __builtin_ctzll(__ballot(in && (uint32_t)be == least));
    }
    const int taken = __builtin_amdgcn_readlane(be, w);
    if (l.lane == r) {
      my_id = taken;
      my_key = mh;
    }
    const bool mine = l.lane == w;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if constexpr (kSorted) {
        hi[j] = mine ? (j + 1 < VPL ? hi[j + 1 < VPL ? j + 1 : j] : 0u) : hi[j];
        id[j] = mine && j + 1 < VPL ? id[j + 1 < VPL ? j + 1 : j] : id[j];
        if constexpr (WIDE) lo[j] = mine ? (j + 1 < VPL ? lo[j + 1 < VPL ? j + 1 : j] : 0u) : lo[j];
      } else if (mine && l.expert(j) == taken) {
        hi[j] = 0;
        if constexpr (WIDE) lo[j] = 0;
      }
    }
  }
  if constexpr (CHECK) {
    // all neighbours at once; key 0: every candidate is taken
    const uint32_t below = __shfl_down(my_key, 1, 64);
    const uint32_t next = l.lane == a.k - 1 ? last : below;
    const float c = of_key(my_key);
    return !__any(l.lane < a.k && next != 0 && !(c - of_key(next) > choice_bound(c)));
  }
  return true;
}

template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
  butterfly(64, [&](auto dc) __attribute__((always_inline)) { v += across<decltype(dc)::value>(v); });
  return v;
}

// Waves of a SIMD that the registers have to leave room for (8192 tokens of
// 1024 experts, 16 a lane: 37 us with four, 41 with the three that the
// compiler leaves by itself for one register more).
constexpr int route_waves(int vpl) { return vpl <= 4 ? 8 : vpl <= 8 ? 6 : vpl <= 16 ? 4 : 2; }

template <int TYPE, int VPL>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256),
                          amdgpu_waves_per_eu(route_waves(VPL)))) void
route_kernel(RouteArgs a) {
  __shared__ float logits[4][VPL * 64];  // a wave's own, by place: lane and j
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  Lane l;
  l.lane = threadIdx.x & 63;
  l.log_per = a.groups <= 1 ? 6 : 6 - (32 - __builtin_clz(a.groups - 1));
  l.per = 1 << l.log_per;
  l.group = l.lane >> l.log_per;
  l.sub = l.lane & (l.per - 1);
  l.size = a.size;

  // All loads go out before the first is used (places past the group read
  // expert 0 and are set aside).
  using X = std::conditional_t<TYPE == kStoreF32, float,
                               std::conditional_t<TYPE == kStoreF16, _Float16, __bf16>>;
  const X* row = (const X*)a.x + t * a.ldx;
  X raw[VPL];
  float b[VPL], x[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    raw[j] = row[l.has(j, a.groups) ? l.expert(j) : 0];
    b[j] = 0.0f;
  }
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) b[j] = a.bias[l.has(j, a.groups) ? l.expert(j) : 0];
  }
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    x[j] = l.has(j, a.groups) ? logit((float)raw[j]) : -INFINITY;
    b[j] = logit(b[j]);
    m = fmaxf(m, x[j]);
    logits[threadIdx.x >> 6][j * 64 + l.lane] = x[j];
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
  // 1 / (1 + exp(-v)), or exp(v - m) / z
  const float sign = a.sigmoid ? -1.0f : 1.0f, shift = a.sigmoid ? 0.0f : m;
  auto score = [&](float v) __attribute__((always_inline)) {
    const float e = expf(sign * (v - shift));
    return a.sigmoid ? 1.0f / (1.0f + e) : e / z;
  };

  const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
  uint32_t hi[VPL], lo[VPL];
  const float* const own = &logits[threadIdx.x >> 6][l.lane];
  int my_id = 0;
  bool done;
  {
    float c[VPL];
    float best = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      c[j] = by_logit ? x[j] : score(x[j]) + b[j];
      if (x[j] == -INFINITY) c[j] = -INFINITY;  // masked, whatever its bias, or no expert here
      second = fmaxf(second, fminf(best, c[j]));
      best = fmaxf(best, c[j]);
    }
    bool stays = true, near = false;
    if (a.topk_groups < a.groups) stays = group_stays<float>(a, l, best, second, 0.0f, near);
#pragma unroll
    for (int j = 0; j < VPL; ++j) hi[j] = stays && l.has(j, a.groups) ? key_of(c[j]) : 0u;
    if (by_logit) {
      // (a tie between groups is one between logits: the lowest index)
      done = choose<VPL, false, false>(a, l, hi, lo, own, my_id);
    } else {
      done = !near && choose<VPL, false, true>(a, l, hi, lo, own, my_id);
    }
  }
  if (!done) {
    double c[VPL];
    double best = -INFINITY, second = -INFINITY, zz = 1.0;
    float top = -INFINITY;  // the logit of the best
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
      if (x[j] == -INFINITY) c[j] = -INFINITY;
      top = (c[j] > best) | ((c[j] == best) & (x[j] > top)) ? x[j] : top;
      second = fmax(second, fmin(best, c[j]));
      best = fmax(best, c[j]);
    }
    bool stays = true, near = false;
    if (a.topk_groups < a.groups) stays = group_stays<double>(a, l, best, second, top, near);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const uint64_t k = stays && l.has(j, a.groups) ? key_of(c[j]) : 0ull;
      hi[j] = (uint32_t)(k >> 32);
      lo[j] = (uint32_t)k;
    }
    choose<VPL, true, false>(a, l, hi, lo, own, my_id);
  }

  float w = 0.0f, v = -INFINITY;
  if (l.lane < a.k) {  // my_id's place: its group's lanes, dealt in turn
    // (my_id / size: the product is off by less than 2^-13 / size, and the
    // quotient at least 1 / (2 size) from a whole number)
    const int group = (int)(((float)my_id + 0.5f) * a.inv_size), in = my_id - group * l.size;
    const int j = in >> l.log_per;
    v = logits[threadIdx.x >> 6][j * 64 + group * l.per + (in & (l.per - 1))];
    w = score(v);
  }
  if (a.renorm) {
    const float sum = wave_sum(w);
    const float each = w;
    w = sum > 0.0f ? w / sum : 0.0f;
    // Scores near fp32's smallest, or below it, have lost their ratios (and
    // sigmoid's exp(-v) is infinite from -88.7 down): again in fp64, whose
    // range goes to a sigmoid of -709 or a softmax score 745 below the largest.
    if (__any(each < 0x1p-100f && v > -INFINITY)) {
      const double x = v;
      const double s = l.lane >= a.k ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)m);
      const double total = wave_sum(s);
      w = total > 0.0 ? (float)(s / total) : 0.0f;
    }
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
  const int per = 64 / g2, size = a.size;
  const int vpl = (size + per - 1) / per;  // at most 32: size <= 1024 / groups, per > 32 / groups
  const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
  if (vpl <= 1) hipLaunchKernelGGL((route_kernel<TYPE, 1>), grid, block, 0, s, a);
  else if (vpl <= 2) hipLaunchKernelGGL((route_kernel<TYPE, 2>), grid, block, 0, s, a);
  else if (vpl <= 4) hipLaunchKernelGGL((route_kernel<TYPE, 4>), grid, block, 0, s, a);
  else if (vpl <= 8) hipLaunchKernelGGL((route_kernel<TYPE, 8>), grid, block, 0, s, a);
  else if (vpl <= 16) hipLaunchKernelGGL((route_kernel<TYPE, 16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((route_kernel<TYPE, 32>), grid, block, 0, s, a);
  return hipGetLastError();
}

// n / k for 0 <= n < 2^30: with 2^s >= k and M = floor(2^(30+s) / k) + 1,
// n M / 2^(30+s) exceeds n / k by less than 2^-s <= 1 / k.
struct Divide {
  uint32_t M;
  int shift;
  explicit Divide(uint32_t k) {
    int s = 0;
    while ((uint64_t(1) << s) < k) ++s;
    shift = 30 + s;
    M = (uint32_t)((uint64_t(1) << shift) / k + 1);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return (int)(((uint64_t)(uint32_t)n * M) >> shift);
  }
};

// A stable counting sort of the R = T * k ids, one workgroup per expert and
// one more for the slots whose id names no expert: each reads every id twice
// (they stay in L2), first to count the ids below its own, which is where
// its rows start, then to place its own in their order.  One launch, no
// atomics, so the order never depends on timing.  Each wave takes a
// contiguous part of the ids, so the waves meet once.
//
// Bound by instructions, R / 64 vectors of ids for each expert, so a vector
// costs as few as can be: two comparisons and one addition in the first
// pass, in the second a comparison and a branch past the vectors without a
// match; a product and a shift in place of the division by k (10 us at 65536
// ids and 256 experts, launched back to back; 41 us with checked loads,
// ballots in both passes and a division).  Sixteen loads wait together, the
// last few in fours (12800 ids: 5.1 us, 7.6 one by one).  Four ids a lane and
// load: no faster.
template <int W>
__global__ __launch_bounds__(W * 64) void plan_kernel(const int32_t* __restrict__ ids, int R,
                                                      Divide by_k, int E,
                                                      int32_t* __restrict__ offsets,
                                                      int32_t* __restrict__ rows,
                                                      int32_t* __restrict__ pos) {
  __shared__ int below_of[W], own_of[W];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t e = blockIdx.x;
  const bool dropped = e == (uint32_t)E;  // the slots of no expert: ids >= E, unsigned
  const uint32_t span = dropped ? 0u - e : 1u;  // own ids: e .. e + span - 1
  const int part = ((R + W - 1) / W + 63) / 64 * 64;
  const int begin = min((int64_t)wave * part, (int64_t)R), end = min((int64_t)begin + part, (int64_t)R);

  // use(first slot, ids, lanes that hold one) for each 64 ids of the part
  auto each = [&](auto&& use) __attribute__((always_inline)) {
    int i = begin;
    auto batches = [&](auto bc) __attribute__((always_inline)) {
      constexpr int B = decltype(bc)::value;
      for (; i + B * 64 <= end; i += B * 64) {
        uint32_t id[B];
#pragma unroll
        for (int b = 0; b < B; ++b) id[b] = (uint32_t)ids[i + b * 64 + lane];
#pragma unroll
        for (int b = 0; b < B; ++b) use(i + b * 64, id[b], true);
      }
    };
    batches(std::integral_constant<int, 16>{});
    batches(std::integral_constant<int, 4>{});
    for (; i < end; i += 64) use(i, (uint32_t)ids[min(i + lane, end - 1)], i + lane < end);
  };
  int below = 0, own = 0;
  each([&](int, uint32_t id, bool in) __attribute__((always_inline)) {
    below += in && id < e ? 1 : 0;
    own += __popcll(__ballot(in && id - e < span));
  });
#pragma unroll
  for (int d = 1; d < 64; d *= 2) below += __shfl_xor(below, d, 64);
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
  each([&](int i, uint32_t id, bool in) __attribute__((always_inline)) {
    const bool match = in && id - e < span;
    const uint64_t mine = __ballot(match);
    if (mine == 0) return;
    if (match) {
      const int p = at + (int)__builtin_amdgcn_mbcnt_hi(
                             (uint32_t)(mine >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mine, 0u));
      rows[p] = dropped ? -1 : by_k(i + lane);
      pos[i + lane] = dropped ? -1 : p;
    }
    at += __popcll(mine);
  });
}

// out[t] = sum over slots j of w[t,j] Y[pos[t,j]], in fp32 in the order of
// the slots.  Eight columns a thread, Y's rows starting at any element; a slot
// whose pos lies outside Y (dropped) adds nothing.  Bound by memory: 604 MB
// (8192 tokens, k = 8, rows of 4096 bf16) in 126 us, 4.8 TB/s.
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
  const Divide by_k((uint32_t)k);
  // (4 against 16 waves: 3.5 against 4.2 us at 4096 ids, 4.8 against 5.7 at
  // 8192, 7.3 against 4.8 at 16384, with 256 experts)
  if (R <= 8192)
    hipLaunchKernelGGL(plan_kernel<4>, dim3(E + 1), dim3(256), 0, s, ids, R, by_k, E, offsets, rows,
                       pos);
  else
    hipLaunchKernelGGL(plan_kernel<16>, dim3(E + 1), dim3(1024), 0, s, ids, R, by_k, E, offsets,
                       rows, pos);
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
