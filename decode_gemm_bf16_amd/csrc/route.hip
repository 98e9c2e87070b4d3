// Routing: router logits to each token's experts and their weights.
//
// With logits l of one token over E experts and an optional bias b:
//   score   s_e = softmax(l)_e or 1 / (1 + exp(-l_e))
//   choice  c_e = s_e + b_e with a bias; without one the order of the scores
//           is the order of the logits, and c_e = l_e (no rounding of a score
//           decides between two experts)
//   groups  (E / groups consecutive experts each) are ordered by their largest
//           c_e, or by the sum of their two largest s_e + b_e; top_groups stay
//   the top_k largest c_e in the kept groups are the token's experts, equal
//   ones by the lowest index; weight = s_e, over the sum of the chosen if
//   renormalised, times a factor.
// Choices that depend on scores are made in 64 bits: two experts whose values
// differ by more than a 64-bit rounding are always ordered as in exact
// arithmetic, whatever the order of the sums.  An expert whose logit is -inf
// or NaN, or whose choice is -inf or NaN, is no candidate; +inf counts as the
// largest finite value.
//
// A token takes W lanes (16, so that a wave works four tokens, or 64).  Lane g * L
// + j of them, L the largest power of two <= W / groups, holds experts of group
// g, so that a group's two largest values are found within L neighbouring lanes.
//
// Choices are first made in 32 bits, on keys whose low bits name the value's
// place in its lane, and the distance of each choice to the next is compared
// with a bound on the errors of both.  Where a distance is within the bound
// (about 1 token in 200) the top_k + 1 values found are ordered again by their
// 64-bit values, which proves the choice if the one after them is far enough.
// What is still open then (more close values, a merit of groups, too few
// candidates) is decided on all values in 64 bits.  bf16 logits without a bias
// need none of it: the low 16 bits of their keys hold the expert itself.
#include "recon.h"
#include "routing.h"

namespace uw {
namespace {

constexpr float kLowF = -__builtin_huge_valf();

template <typename T>
__device__ __forceinline__ T low_of();
template <>
__device__ __forceinline__ float low_of<float>() { return kLowF; }
template <>
__device__ __forceinline__ double low_of<double>() { return -__builtin_huge_val(); }

// NaN as -inf (no candidate), +inf as the type's largest finite value.
__device__ __forceinline__ float clean(float v, bool bf16) {
  return fminf(fmaxf(v, kLowF), bf16 ? 0x1.FEp127f : __FLT_MAX__);
}

__device__ __forceinline__ float load_logit(const void* p, int64_t i, bool bf16) {
  return clean(bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i], bf16);
}

// x combined with the same of another lane; after all steps each of the W lanes
// holds the combination of all.  Within 16 lanes the moves ride on the operation
// (DPP: neighbours, pairs, then mirrored halves, whose lanes already agree).
template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T v) {
  if constexpr (sizeof(T) == 4) {
    const int x = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(x, CTRL, 0xF, 0xF, true));
  } else {
    const u32x2 x = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(T, u32x2{dpp<CTRL>(x.x), dpp<CTRL>(x.y)});
  }
}
// Across rows of 16 lanes: v and itself with neighbouring rows (halves) swapped
// between the two are the even and the odd rows' values in all lanes.  (Moves through
// LDS instead: 1024 experts 5.6 against 4.9 us at 64 tokens, 27.5 against 26.3 at
// 16384; 512 with 20 choices 5.7 against 4.5, but 22.0 against 22.6 at 16384.)
template <int ROW, typename T, typename F>
__device__ __forceinline__ T across(T v, F f) {
  auto swap = [](uint32_t x) {
    if constexpr (ROW == 16)
      return __builtin_amdgcn_permlane16_swap(x, x, false, false);
    else
      return __builtin_amdgcn_permlane32_swap(x, x, false, false);
  };
  if constexpr (sizeof(T) == 4) {
    const auto x = swap(__builtin_bit_cast(uint32_t, v));
    return f(__builtin_bit_cast(T, (uint32_t)x[0]), __builtin_bit_cast(T, (uint32_t)x[1]));
  } else {
    const u32x2 h = __builtin_bit_cast(u32x2, v);
    const auto x = swap(h.x), y = swap(h.y);
    return f(__builtin_bit_cast(T, u32x2{x[0], y[0]}), __builtin_bit_cast(T, u32x2{x[1], y[1]}));
  }
}
template <int W, typename T, typename F>
__device__ __forceinline__ T all_lanes(T v, F f) {
  static_assert(W == 16 || W == 64, "");
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  if constexpr (W == 64) {
    v = across<16>(v, f);
    v = across<32>(v, f);
  }
  return v;
}
struct Max {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Min {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a < b ? a : b; }
  __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct Sum {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// Where a lane's values stand: its i-th is expert base + (i / 4 * L + j) * 4 + i % 4
// with vector loads of 4 logits, base + i * L + j else; per: experts of a group.
struct Place {
  int lane, g, j, lshift, per;
  bool vec;
  __device__ __forceinline__ int in_group(int i) const {
    return vec ? ((((i >> 2) << lshift) + j) << 2) + (i & 3) : (i << lshift) + j;
  }
};

// The bias of a lane's values (0 past the last expert), NaN as -inf.
template <int VPL>
__device__ __forceinline__ void load_bias(const RouteArgs& a, const Place& at, float (&b)[VPL]) {
  const float* src = a.bias + at.g * at.per;
  if (VPL >= 4 && at.vec) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const int m = at.in_group(i);
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      if (at.g < a.groups && m < at.per) v = *(const f32x4*)(src + m);
#pragma unroll
      for (int k = 0; k < 4; ++k) b[i + k] = fmaxf(v[k], kLowF);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int m = at.in_group(i);
      b[i] = at.g < a.groups && m < at.per ? fmaxf(src[m], kLowF) : 0.f;
    }
  }
}

// Whether the lane's group is among the top_groups by merit.
template <int W, typename T>
__device__ __forceinline__ bool group_stays(const RouteArgs& a, const Place& at, T merit) {
  int better = 0;
  for (int q = 0; q < a.groups; ++q) {
    const T other = __shfl(merit, q << at.lshift, W);
    better += other > merit || (other == merit && q < at.g);
  }
  return better < a.top_groups;
}

// The two largest of the group's values from the two largest of its lanes.
template <int W, typename T>
__device__ __forceinline__ void group_two(const Place& at, T& hi, T& lo) {
  for (int o = 1 << at.lshift >> 1; o > 0; o >>= 1) {
    const T h2 = __shfl_xor(hi, o, W), l2 = __shfl_xor(lo, o, W);
    lo = Max()(Min()(hi, h2), Max()(lo, l2));
    hi = Max()(hi, h2);
  }
}

// score + bias in 64 bits, -inf where there is no candidate; total: the
// softmax's sum.
template <int W, int VPL>
__device__ __forceinline__ void values_exact(const RouteArgs& a, const Place& at, const float (&l)[VPL], float top,
                                             double& total, double (&v)[VPL]) {
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  } else {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = l[i] > kLowF ? exp((double)l[i] - (double)top) : 0.0;
      sum += v[i];
    }
    sum = all_lanes<W>(sum, Sum());
    total = sum > 0.0 ? sum : 1.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] /= total;
  }
  if (a.bias) {
    float b[VPL];
    load_bias<VPL>(a, at, b);
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] += (double)b[i];
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (!(l[i] > kLowF) || !(v[i] > low_of<double>())) v[i] = low_of<double>();
}

// Whether the lane's group stays, by merits in 64 bits.
template <int W, int VPL>
__device__ bool stays_exact(const RouteArgs& a, const Place& at, const float (&l)[VPL], float top) {
  double v[VPL], total, hi = low_of<double>(), lo = low_of<double>();
  values_exact<W, VPL>(a, at, l, top, total, v);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    lo = fmax(lo, fmin(hi, v[i]));
    hi = fmax(hi, v[i]);
  }
  group_two<W>(at, hi, lo);
  return group_stays<W>(a, at, a.pairs && lo > low_of<double>() ? hi + lo : hi);
}

// The token's choices in K (float: the logits; double: score + bias) among the
// groups that stay.  Returns the choice of rank `lane`, -1 for none.
template <typename K, int W, int VPL>
__device__ int choose_exact(const RouteArgs& a, const Place& at, const float (&l)[VPL], float top, bool stays,
                            double& total) {
  K c[VPL];
  auto expert = [&](int i) { return at.g * at.per + at.in_group(i); };
  if constexpr (sizeof(K) == 8) {
    values_exact<W, VPL>(a, at, l, top, total, c);
    if (!a.bias) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = l[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = l[i];
  }
  if (!stays) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = low_of<K>();
  }
  int mine = -1;
  for (int r = 0; r < a.top_k; ++r) {
    K best = low_of<K>();
    int e = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (c[i] > best) {
        best = c[i];
        e = expert(i);
      }
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      const K b2 = __shfl_xor(best, o, W);
      const int e2 = __shfl_xor(e, o, W);
      if (b2 > best || (b2 == best && e2 < e)) {
        best = b2;
        e = e2;
      }
    }
    if (at.lane == r) mine = best > low_of<K>() ? e : -1;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (expert(i) == e) c[i] = low_of<K>();
  }
  return mine;
}

// Unsigned order of a float's bits; kOrdered0 and above for candidates.
constexpr uint32_t kOrdered0 = 0x00800000u;  // of the lowest finite value; -inf is below
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Whether all W lanes of the token say so.
template <int W>
__device__ __forceinline__ bool all_say(bool v) {
  const uint64_t no = __ballot(!v);
  return W == 64 ? no == 0 : ((no >> (threadIdx.x & 48)) & 0xFFFFu) == 0;
}

// One token's choice in 32 bits; returns whether it is proved.  `mine`: the choice
// of rank `lane`; stays: whether the lane's group does (always decided).
//
// A value's key is its ordered bits with the low 4 replaced by 15 - i.  The next
// key below M is found without taking any out: key - M wraps to 2^32 - (M - key)
// for the keys below M, which is more than key - M of any other, so that the
// largest difference belongs to the next key.  (Equal keys in two lanes count as
// one step; the lanes that owned a step are counted.)
// Errors: a sigmoid in float32 is within 4 x 2^-24 (v_exp at 1 ulp and its rounded
// argument, both of which reach s by s (1 - s): 0.5 and 0.3; 1 + e: 1; v_rcp at 1
// ulp: 2); a softmax's score within 2^-19 of the largest one (the terms of its sum,
// 2 ulp and the argument's rounding, |x| of each: together at most 2 + ln 1024 of
// 2^-24; the score itself the same, |x| e^x <= 0.37, and two products);
// the sum with the bias 2^-24, and the key's cut 2^-19, of the value.  Logits are
// exact and the cut keeps their order, so any distance proves it.
template <bool BF16_KEYS, int W, int VPL>
__device__ __forceinline__ bool choose_fast(const RouteArgs& a, const Place& at, const float (&l)[VPL], float top,
                                            float rtotal, int64_t row, uint8_t* owner, int& mine, bool& stays) {
  const bool scores = !BF16_KEYS && (a.bias || (a.pairs && a.groups > 1)), biased = !BF16_KEYS && a.bias;
  const float eps = !scores ? 0.f : a.sigmoid ? 0x1p-22f : 0x1p-19f * rtotal;
  auto expert = [&](int i) { return at.g * at.per + at.in_group(i); };
  float c[VPL], hi = kLowF, lo = kLowF;  // choices; the group's two largest
  if (scores) {
    float s[VPL];
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        s[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[i] * -1.44269504f));
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = __builtin_amdgcn_exp2f((l[i] - top) * 1.44269504f) * rtotal;
    }
    if (a.bias) {
      load_bias<VPL>(a, at, c);
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] += c[i];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = l[i] > kLowF ? s[i] : kLowF;
      lo = __builtin_amdgcn_fmed3f(hi, lo, s[i]);
      hi = fmaxf(hi, s[i]);
      c[i] = s[i];
    }
    if (!a.bias) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = l[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = l[i];
      hi = fmaxf(hi, l[i]);
    }
  }
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const uint32_t o = ordered(c[i] + 0.f);  // -0 as 0
    key[i] = BF16_KEYS ? (o & 0xFFFF0000u) | (0xFFFFu - expert(i)) : (o & ~15u) | (15u - i);
  }
  if (a.groups > a.top_groups) {
    group_two<W>(at, hi, lo);
    const float merit = scores && a.pairs && lo > kLowF ? hi + lo : hi;
    stays = group_stays<W>(a, at, merit);
    if (scores) {
      const bool there = at.g < a.groups;
      const float in = all_lanes<W>(there && stays ? merit : -kLowF, Min());
      const float out = all_lanes<W>(there && !stays ? merit : kLowF, Max());
      // The errors of up to two scores on each side, and the roundings of sums of this size.  Without
      // a candidate in the groups left out there is nothing to decide, unless a sum may have passed
      // float32's range: a merit of -inf is then that of a group with candidates (size is infinite).
      const float size = all_lanes<W>((hi > kLowF ? fabsf(hi) : 0.f) + (lo > kLowF ? fabsf(lo) : 0.f), Max());
      if ((out > kLowF || size > __FLT_MAX__) && !(in - out > 4.f * eps + 0x1p-21f * size))
        stays = stays_exact<W, VPL>(a, at, l, top);
    }
    if (!stays) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = 0;
    }
  }
  // W lanes hold ranks 0 .. W - 1, and rank top_k needs one
  if (!BF16_KEYS && a.top_k >= W) return false;
  uint32_t m = 0, chosen = 0, after = 0;  // after: the key behind those of rank 0..top_k
  int owned = 0;
  const int rounds = a.top_k + (BF16_KEYS ? 0 : 2);
  for (int r = 0; r < rounds; ++r) {
    uint32_t best = 0;  // of key - m
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t d = key[i] - m;
      best = d > best ? d : best;
    }
    uint32_t next = m + all_lanes<W>(best, Max());
    if (r > 0 && next >= m) next = 0;  // all keys are through
    if constexpr (!BF16_KEYS) {
      if (r <= a.top_k && best + m == next && next >= kOrdered0) {
        owner[r] = (uint8_t)at.lane;
        ++owned;
      }
    }
    if (at.lane == r) chosen = next;
    after = next;
    if (next < kOrdered0) break;  // the rest has none either
    m = next;
  }
  if constexpr (BF16_KEYS) {
    const bool there = chosen >= kOrdered0 && at.lane < a.top_k;
    mine = there ? (int)(0xFFFFu - (chosen & 0xFFFFu)) : -1;
    return true;
  } else {
    __builtin_amdgcn_wave_barrier();
    const bool listed = at.lane <= a.top_k && chosen >= kOrdered0;
    mine = -1;
    if (listed) {
      const int o = owner[at.lane] & (W - 1);
      const Place there{o, o >> at.lshift, o & ((1 << at.lshift) - 1), at.lshift, at.per, at.vec};
      mine = there.g * at.per + there.in_group(15 - (int)(chosen & 15u));
    }
    const int count = __popcll(__ballot(listed) >> (W == 64 ? 0 : threadIdx.x & 48) & (W == 64 ? ~0ull : 0xFFFFull));
    const bool whole = all_lanes<W>(owned, Sum()) == count;  // no two lanes shared a key
    // distance to the next rank; the last listed one's is to `after`
    const uint32_t below = __shfl_down((int)chosen, 1, W);  // all lanes take part, also the one that does not use it
    const uint32_t follow = at.lane == a.top_k ? after : below;
    const float v = of_ordered(chosen & ~15u), f = of_ordered(follow & ~15u);
    const bool far = follow < kOrdered0 ||
                     v - f > (biased ? 2.f * eps + 0x1p-18f * fmaxf(fabsf(v), fabsf(f)) : 0.f);
    const bool sure = whole && all_say<W>(at.lane >= a.top_k || !listed || far);
    if (sure || !whole) {
      if (at.lane >= a.top_k) mine = -1;
      return sure;
    }
    // order the listed by their 64-bit values; right if rank top_k is far from what is behind
    // it, or was far behind the choice before
    const bool closed = !all_say<W>(!((at.lane == a.top_k || at.lane == a.top_k - 1) && (far || !listed)));
    if (!closed) return false;
    double x = low_of<double>(), total = 1.0;
    if (biased && !a.sigmoid) {  // a total in float32 would shift the scores against the biases
      total = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) total += l[i] > kLowF ? exp((double)l[i] - (double)top) : 0.0;
      total = all_lanes<W>(total, Sum());
    }
    if (listed) {
      x = load_logit(a.logits, row + mine, a.bf16);
      if (biased)
        x = (a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / total) + (double)a.bias[mine];
    }
    int rank = 0;
    for (int q = 0; q <= a.top_k; ++q) {
      const double other = __shfl(x, q, W);
      const int e = __shfl(mine, q, W);
      rank += other > x || (other == x && e < mine);
    }
    uint8_t* place = owner;  // rank -> lane
    __builtin_amdgcn_wave_barrier();
    if (listed) place[rank] = (uint8_t)at.lane;
    __builtin_amdgcn_wave_barrier();
    const int from = at.lane < count && at.lane < a.top_k ? place[at.lane] & (W - 1) : at.lane;
    const int e = __shfl(mine, from, W);
    mine = at.lane < a.top_k && at.lane < count ? e : -1;
    return true;
  }
}

// K: the type in which exact choices are compared.  FAST: choose_fast first.
template <typename K, bool BF16, bool FAST, int W, int VPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, int lshift, bool vec) {
  __shared__ uint8_t owner[256 / W][W];  // rank -> lane
  const int lane = threadIdx.x & (W - 1), token = threadIdx.x / W;
  const int64_t t = (int64_t)blockIdx.x * (256 / W) + token;
  if (t >= a.tokens) return;  // whole sub-waves: the moves below stay within W lanes
  const Place at{lane, lane >> lshift, lane & ((1 << lshift) - 1), lshift, a.experts / a.groups, vec};
  const int64_t row = t * a.ld, base = row + at.g * at.per;
  float l[VPL];
  if (VPL >= 4 && vec) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      const int m = at.in_group(i);
      const bool there = at.g < a.groups && m < at.per;
      if constexpr (BF16) {
        const u32x2 v = there ? *(const u32x2*)((const uint16_t*)a.logits + base + m) : u32x2{0xFF80FF80u, 0xFF80FF80u};
        l[i] = clean(__uint_as_float(v.x << 16), true);
        l[i + 1] = clean(__uint_as_float(v.x & 0xFFFF0000u), true);
        l[i + 2] = clean(__uint_as_float(v.y << 16), true);
        l[i + 3] = clean(__uint_as_float(v.y & 0xFFFF0000u), true);
      } else {
        const f32x4 v = there ? *(const f32x4*)((const float*)a.logits + base + m) : f32x4{kLowF, kLowF, kLowF, kLowF};
#pragma unroll
        for (int k = 0; k < 4; ++k) l[i + k] = clean(v[k], false);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int m = at.in_group(i);
      l[i] = at.g < a.groups && m < at.per ? load_logit(a.logits, base + m, BF16) : kLowF;
    }
  }
  float top = kLowF;   // softmax: the largest logit
  double total = 1.0;  // softmax: the sum of exp(l - top)
  constexpr bool kScores = sizeof(K) == 8;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = fmaxf(top, l[i]);
    top = all_lanes<W>(top, Max());
    if (kScores || !a.renormalise) {
      // Added in 64 bits, as a float sum's own roundings put a weight off by up to 6 x
      // 2^-24 (16384 tokens of 256: 3.3e-7 against 7.3e-8, for 11.4 against 11.7 us).  Its
      // terms stay float32: they are off by 2 ulp and |l - top| 2^-24 at most, which nearly
      // cancels in the sum; exponentials in 64 bits make 7.3e-8 the 6.0e-8 of the result's
      // own rounding, for 15.5 against 12.1 us (16384 tokens of 1024: 44.7 against 34.6).
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += l[i] > kLowF ? (double)expf(l[i] - top) : 0.0;
      sum = all_lanes<W>(sum, Sum());
      total = sum > 0.0 ? sum : 1.0;
    }
  }
  int mine = -1;
  bool sure = false, stays = true;
  if constexpr (FAST) {
    sure = choose_fast<BF16 && !kScores, W, VPL>(a, at, l, top, 1.f / (float)total, row, owner[token], mine, stays);
  } else if (a.groups > a.top_groups) {
    if constexpr (kScores) {
      stays = stays_exact<W, VPL>(a, at, l, top);
    } else {
      float hi = kLowF, lo = kLowF;
#pragma unroll
      for (int i = 0; i < VPL; ++i) hi = fmaxf(hi, l[i]);
      group_two<W>(at, hi, lo);
      stays = group_stays<W>(a, at, hi);
    }
  }
  if (!sure) mine = choose_exact<K, W, VPL>(a, at, l, top, stays, total);
  // lane r < top_k: the weight of the r-th choice, from its logit, in 64 bits
  double w = 0.0;
  if (mine >= 0) {
    const double v = load_logit(a.logits, row + mine, BF16);
    w = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / total;
  }
  if (a.renormalise) {
    const double sum = all_lanes<W>(w, Sum());
    if (sum > 0.0) w /= sum;
  }
  if (lane < a.top_k) {
    a.index[t * a.top_k + lane] = mine;
    a.weight[t * a.top_k + lane] = (float)(w * (double)a.scale);
  }
}

template <typename K, bool BF16, int W>
hipError_t launch_vpl(const RouteArgs& a, int lshift, int vpl, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + 256 / W - 1) / (256 / W))), block(256);
  const int per = a.experts / a.groups;
  const bool vec = vpl >= 4 && per % 4 == 0 && a.ld % 4 == 0 && (uintptr_t)a.logits % (BF16 ? 8 : 16) == 0 &&
                   (uintptr_t)a.bias % 16 == 0;
  if (vpl <= 1)
    hipLaunchKernelGGL((route_kernel<K, BF16, true, W, 1>), grid, block, 0, s, a, lshift, vec);
  else if (vpl <= 2)
    hipLaunchKernelGGL((route_kernel<K, BF16, true, W, 2>), grid, block, 0, s, a, lshift, vec);
  else if (vpl <= 4)
    hipLaunchKernelGGL((route_kernel<K, BF16, true, W, 4>), grid, block, 0, s, a, lshift, vec);
  else if (vpl <= 8)
    hipLaunchKernelGGL((route_kernel<K, BF16, true, W, 8>), grid, block, 0, s, a, lshift, vec);
  else if (vpl <= 16)
    hipLaunchKernelGGL((route_kernel<K, BF16, true, W, 16>), grid, block, 0, s, a, lshift, vec);
  else if constexpr (W == 64)  // groups * L > 32, so at most 1024 / 32 experts a lane
    hipLaunchKernelGGL((route_kernel<K, BF16, false, W, 32>), grid, block, 0, s, a, lshift, vec);
  return hipGetLastError();
}

// Experts per lane with W lanes a token, and the lanes of a group's shift.
int vpl_of(const RouteArgs& a, int W, int* lshift) {
  *lshift = 0;
  while ((a.groups << (*lshift + 1)) <= W) ++*lshift;
  const int per = a.experts / a.groups, L = 1 << *lshift;
  return per % 4 == 0 && per > 3 * L ? (per / 4 + L - 1) / L * 4 : (per + L - 1) / L;
}

// 16 lanes a token wherever its experts, groups and ranks fit them, whatever the
// number of tokens: 64 experts 3.5 against 3.9 us at 64 tokens and 5.1 against 13.6
// at 16384; 256 experts in 8 groups 14 to 16 against 24 to 25 at 16384.  Where few
// waves are at work those 256 take more in 16 lanes (16 values a lane instead of 4):
// 6.5 against 5.9 us at one token, 6.8 against 6.5 to 6.8 at 64, 6.9 to 8 against 6.7
// at 512, 7.4 to 8.5 against 7.2 to 8.6 at 1024, which no rule is made for.  W = 64
// for the rest.
template <typename K, bool BF16>
hipError_t launch_w(const RouteArgs& a, hipStream_t s) {
  int lshift = 0;
  const int v16 = vpl_of(a, 16, &lshift);
  if (a.groups <= 16 && a.top_k < 16 && v16 <= 16)
    return launch_vpl<K, BF16, 16>(a, lshift, v16, s);
  const int v64 = vpl_of(a, 64, &lshift);
  return launch_vpl<K, BF16, 64>(a, lshift, v64, s);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  // scores decide where a bias is added to them or two of them are summed;
  // else the logits do
  if (a.bias || (a.pairs && a.groups > 1)) return a.bf16 ? launch_w<double, true>(a, s) : launch_w<double, false>(a, s);
  return a.bf16 ? launch_w<float, true>(a, s) : launch_w<float, false>(a, s);
}

}  // namespace uw
