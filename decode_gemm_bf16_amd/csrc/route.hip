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
// A token takes W lanes.  Lane g * L + j of them, L the largest power of two
// <= W / groups, holds experts j, j + L, ... of group g, so that a group's two
// largest values are found within L neighbouring lanes.
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

__device__ __forceinline__ float load_logit(const void* p, int64_t i, bool bf16) {
  float v = bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
  if (!(v > kLowF)) return kLowF;  // NaN as well
  return v > __FLT_MAX__ ? __FLT_MAX__ : v;
}

// K: the type in which choices are compared (float: the logits themselves).
template <typename K, int W, int VPL>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a, int lshift) {
  const int lane = threadIdx.x & (W - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / W) + threadIdx.x / W;
  if (t >= a.tokens) return;  // whole sub-waves: the shuffles below stay within W lanes
  const int L = 1 << lshift, g = lane >> lshift, j = lane & (L - 1);
  const int per = a.experts / a.groups;
  const int64_t row = t * a.ld;
  float l[VPL];
  K c[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int m = j + (i << lshift);
    l[i] = g < a.groups && m < per ? load_logit(a.logits, row + g * per + m, a.bf16) : kLowF;
  }
  float top = kLowF;  // softmax: the largest logit
  double total = 1.0;  // softmax: the sum of exp(l - top)
  const bool need_total = !a.sigmoid && (sizeof(K) == 8 || !a.renormalise);
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = fmaxf(top, l[i]);
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, W));
  }
  if constexpr (sizeof(K) == 8) {
    double s[VPL];
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = l[i] > kLowF ? exp((double)l[i] - (double)top) : 0.0;
        sum += s[i];
      }
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, W);
      total = sum > 0.0 ? sum : 1.0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] /= total;
    }
    double hi = low_of<double>(), lo = low_of<double>();  // the group's two largest
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int m = j + (i << lshift);
      double v = s[i];
      if (a.bias && l[i] > kLowF) v += (double)a.bias[g * per + m];
      if (!(l[i] > kLowF) || !(v > low_of<double>())) v = low_of<double>();
      lo = fmax(lo, fmin(hi, v));
      hi = fmax(hi, v);
      c[i] = a.bias ? v : (double)l[i];
    }
    if (a.groups > 1) {
      for (int o = L / 2; o > 0; o >>= 1) {
        const double h2 = __shfl_xor(hi, o, W), l2 = __shfl_xor(lo, o, W);
        lo = fmax(fmin(hi, h2), fmax(lo, l2));
        hi = fmax(hi, h2);
      }
      const double merit = a.pairs && lo > low_of<double>() ? hi + lo : hi;
      int better = 0;
      for (int q = 0; q < a.groups; ++q) {
        const double other = __shfl(merit, q << lshift, W);
        better += other > merit || (other == merit && q < g);
      }
      if (better >= a.top_groups) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = low_of<K>();
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = l[i];
    if (need_total) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += l[i] > kLowF ? expf(l[i] - top) : 0.f;
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, W);
      total = sum > 0.f ? (double)sum : 1.0;
    }
    if (a.groups > 1) {
      float merit = kLowF;
#pragma unroll
      for (int i = 0; i < VPL; ++i) merit = fmaxf(merit, l[i]);
      for (int o = L / 2; o > 0; o >>= 1) merit = fmaxf(merit, __shfl_xor(merit, o, W));
      int better = 0;
      for (int q = 0; q < a.groups; ++q) {
        const float other = __shfl(merit, q << lshift, W);
        better += other > merit || (other == merit && q < g);
      }
      if (better >= a.top_groups) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = kLowF;
      }
    }
  }
  int mine = -1;
  for (int r = 0; r < a.top_k; ++r) {
    K best = low_of<K>();
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (c[i] > best) {
        best = c[i];
        at = g * per + j + (i << lshift);
      }
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      const K b2 = __shfl_xor(best, o, W);
      const int a2 = __shfl_xor(at, o, W);
      if (b2 > best || (b2 == best && a2 < at)) {
        best = b2;
        at = a2;
      }
    }
    if (lane == r) mine = best > low_of<K>() ? at : -1;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (g * per + j + (i << lshift) == at) c[i] = low_of<K>();
  }
  // lane r < top_k: the weight of the r-th choice, from its logit, in 64 bits
  double w = 0.0;
  if (mine >= 0) {
    const double v = load_logit(a.logits, row + mine, a.bf16);
    w = a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / total;
  }
  if (a.renormalise) {
    double sum = w;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, W);
    if (sum > 0.0) w /= sum;
  }
  if (lane < a.top_k) {
    a.index[t * a.top_k + lane] = mine;
    a.weight[t * a.top_k + lane] = (float)(w * (double)a.scale);
  }
}

template <typename K, int W>
hipError_t launch_vpl(const RouteArgs& a, int lshift, hipStream_t s) {
  const int per = a.experts / a.groups, vpl = (per + (1 << lshift) - 1) >> lshift;
  const dim3 grid((unsigned)((a.tokens + 256 / W - 1) / (256 / W))), block(256);
  if (vpl <= 1)
    hipLaunchKernelGGL((route_kernel<K, W, 1>), grid, block, 0, s, a, lshift);
  else if (vpl <= 2)
    hipLaunchKernelGGL((route_kernel<K, W, 2>), grid, block, 0, s, a, lshift);
  else if (vpl <= 4)
    hipLaunchKernelGGL((route_kernel<K, W, 4>), grid, block, 0, s, a, lshift);
  else if (vpl <= 8)
    hipLaunchKernelGGL((route_kernel<K, W, 8>), grid, block, 0, s, a, lshift);
  else if (vpl <= 16)
    hipLaunchKernelGGL((route_kernel<K, W, 16>), grid, block, 0, s, a, lshift);
  else  // groups * L > 32, so at most 1024 / 32 experts a lane
    hipLaunchKernelGGL((route_kernel<K, W, 32>), grid, block, 0, s, a, lshift);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  constexpr int W = 64;
  int lshift = 0;
  while ((a.groups << (lshift + 1)) <= W) ++lshift;
  // scores decide where a bias is added to them or two of them are summed;
  // else the logits do
  const bool scores = a.bias || (a.pairs && a.groups > 1);
  return scores ? launch_vpl<double, W>(a, lshift, s) : launch_vpl<float, W>(a, lshift, s);
}

}  // namespace uw
