// Attention of each sequence's new tokens over its pages of the cache:
//   y_i = sum_k softmax_k(x_ik) v_k,   x = cap tanh(scale q k / cap) - slope |distance|
// over the keys that token i sees.  One pass over the keys with a running maximum
// and sum.  The rows of one workgroup are the tokens of one sequence times the query
// heads that share one key head, so that keys and values are read once for all of them.
//
// Both products run on v_mfma_f32_32x32x16_bf16, transposed: S^T = K Q^T holds a
// query in each lane's column and 16 keys of a block of 32 in its registers, which is,
// as they stand, the second operand of O^T = V^T P^T; the values lie in the cache in
// the matching order of keys.  The weights P never leave their lanes, and a row's
// maximum and sum are one exchange between the halves of a wave.
//
// The weights go to the second product as bf16, the values' own type: up to 2^-8 of a
// weight, half a step, which on random values is about what rounding y to bf16 costs once
// more (0.0022 of a row against 0.0017 with weights of 32 bits).  A float32 y gets it too.
// Scores, maxima, sums, and outputs until their end are float32.
#pragma once

#include <type_traits>

#include "attention.h"
#include "recon.h"

namespace uw {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -INFINITY;
constexpr int kWaves = 4;     // of a workgroup with many rows
constexpr int few_waves(int dim) { return dim > 128 ? 4 : 8; }  // with few
// A row's maximum moves only when a score is this far above it (in powers of two):
// weights stay below 2^8, and most blocks leave the sums as they are.
constexpr float kSlack = 8.f;
// Sums that are not finite are done again with the weights of the second product times
// kLess: of 2^30 values below 2^128 none is infinite then.  (A power of two: the sums' bits stay
// as they are.)  kMore undoes it.
constexpr float kLess = 0x1p-40f, kMore = 0x1p40f;

__device__ __forceinline__ uint32_t pack(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ float other_half(float v) {  // lane ^ 32's
  const auto two = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(threadIdx.x & 32 ? two[0] : two[1]);
}
// The larger of the two halves' values, in both.
__device__ __forceinline__ float larger_half(float v) {
  const auto two = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(two[0]), __uint_as_float(two[1]));
}

// A value that all lanes read, through the scalar cache: its wait is apart from those
// for the vector loads in flight.  (Only of memory that the call does not write.)
__device__ __forceinline__ int32_t scalar(const int32_t* p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p)[i];
}

// Key of register i of S^T, less the lane's first, 4 (lane / 32).
__device__ __forceinline__ constexpr int key_of(int i) { return 8 * (i / 4) + i % 4; }

struct Seq {
  int t0, count, length, keys, start;  // first token, tokens, length, keys in reach of the table, length - tokens
  int prefix;
  const int32_t* table;
};

__device__ __forceinline__ int token_at(const AttendArgs& a, int t) { return t < 0 ? 0 : t > a.tokens ? a.tokens : t; }

__device__ __forceinline__ Seq sequence(const AttendArgs& a, int b) {
  Seq s;
  const int t0 = token_at(a, scalar(a.offsets, b));
  int t1 = token_at(a, scalar(a.offsets, b + 1));
  if (t1 < t0) t1 = t0;
  int len = scalar(a.lengths, b);
  len = len < 0 ? 0 : len > (1 << 30) ? (1 << 30) : len;
  s.t0 = t0;
  s.count = t1 - t0;
  s.length = len;
  const int64_t reach = (int64_t)a.max_pages << a.page_log2;
  s.keys = s.length < reach ? s.length : (int)reach;
  s.start = s.length - s.count;
  s.prefix = a.prefix ? scalar(a.prefix, b) : 0;
  s.table = a.tables + (int64_t)b * a.ldt;
  return s;
}

// What a lane's row sees: keys lower <= k < upper, and of the drafted ones (k >=
// start, where there is a mask) those whose bits are set.
struct Row {
  int token, head;
  int lower, upper, pos, first;
  float slope;  // times log2 e
  bool live;
};

__device__ __forceinline__ int depth_of(const AttendArgs& a, int token) {
  int n = 0;
  for (int w = 0; w < a.words; ++w) n += __popcll(a.mask[(int64_t)token * a.words + w]);
  return n - 1;
}

__device__ __forceinline__ Row row_of(const AttendArgs& a, const Seq& s, int kvh, int r) {
  Row o;
  const int rows = s.count * a.group;
  o.live = r < rows;
  const int rr = o.live ? r : rows - 1;
  const int i = rr / a.group;
  o.token = s.t0 + i;
  o.head = kvh * a.group + rr - i * a.group;
  const int place = s.start + i;
  o.pos = place;
  o.upper = place + 1;
  if (a.mask) {
    o.pos = s.start + depth_of(a, o.token);
    o.upper = s.keys;
  } else if (s.prefix > o.upper) {
    o.upper = s.prefix;
  }
  if (o.upper > s.keys) o.upper = s.keys;
  o.lower = a.window > 0 && o.pos - a.window + 1 > 0 ? o.pos - a.window + 1 : 0;
  o.first = a.first ? a.first[o.token] : 0;
  if (o.first > o.lower) o.lower = o.first;
  if (o.lower > s.keys) o.lower = s.keys;  // (a mark may be any number; sums with this one stay small)
  o.slope = a.slopes ? a.slopes[o.head] * kLog2e : 0.f;
  return o;
}

// Over a wave's rows: no row sees a key outside [lo, hi), every row sees all of
// [lo_all, hi_all) (and, where there are slopes, none of these keys is ahead of it).
struct Range {
  int lo, hi, lo_all, hi_all;
};

__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_xor(v, o, 64);
    v = w < v ? w : v;
  }
  return __builtin_amdgcn_readfirstlane(v);
}

template <int N>
__device__ __forceinline__ Range range_of(const AttendArgs& a, const Seq& s, const Row (&rows)[N]) {
  int lo = 1 << 30, hi = 0, lo_all = 0, hi_all = 1 << 30;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Row& r = rows[i];
    // (of a tree, drafted keys below the lower bound of the context may be seen: their
    // distance goes by their depth)
    int top = a.mask ? s.start : r.upper;
    if (a.slopes && r.pos + 1 < top) top = r.pos + 1;
    const int low = a.mask && r.lower > s.start ? s.start : r.lower;
    if (low < r.upper) {
      lo = low < lo ? low : lo;
      hi = r.upper > hi ? r.upper : hi;
    }
    lo_all = r.lower > lo_all ? r.lower : lo_all;
    hi_all = top < hi_all ? top : hi_all;
  }
  Range g;
  g.lo = wave_min(lo);
  g.hi = -wave_min(-hi);
  g.lo_all = -wave_min(-lo_all);
  g.hi_all = wave_min(hi_all);
  if (g.lo < 0) g.lo = 0;
  return g;
}
__device__ __forceinline__ Range range_of(const AttendArgs& a, const Seq& s, const Row& r) {
  const Row one[1] = {r};
  return range_of<1>(a, s, one);
}

// Bits j .. j + 31 of a row of the mask (bits outside it are 0).
__device__ __forceinline__ uint32_t mask_bits(const AttendArgs& a, int token, int j) {
  const uint64_t* m = a.mask + (int64_t)token * a.words;
  const int w = j >> 6, sh = j & 63;  // (of a negative j: rounded down)
  uint64_t lo = w >= 0 && w < a.words ? m[w] >> sh : 0;
  if (sh > 32 && w + 1 >= 0 && w + 1 < a.words) lo |= m[w + 1] << (64 - sh);
  return (uint32_t)lo;
}

// The position of key kb + lane % 32 as distances take it: a drafted one's depth goes
// by its row of the mask.
__device__ __forceinline__ int key_pos(const AttendArgs& a, const Seq& s, int k) {
  if (k < s.start || k - s.start >= s.count) return k;
  return s.start + depth_of(a, s.t0 + k - s.start);
}

template <int D>
struct Sums {
  f32x16 o[D / 32];
  float m, l;  // maximum in powers of two, and this lane's share of the weights
};

template <int D>
__device__ __forceinline__ void clear(Sums<D>& c) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) c.o[i] = f32x16{};
  c.m = kNone;
  c.l = 0.f;
}

// What a kernel is built for: a cap (a far one, too), slopes, both or neither.
constexpr int kCap = 1, kSlopes = 2, kFar = 4;
template <typename F>  // f(the kernel's)
inline void with_mode(const AttendArgs& a, F f) {
  const bool far = a.cap > kNearCap;
  if (a.slopes)
    far ? f(std::integral_constant<int, kCap | kSlopes | kFar>{})
        : a.cap > 0.f ? f(std::integral_constant<int, kCap | kSlopes>{}) : f(std::integral_constant<int, kSlopes>{});
  else
    far ? f(std::integral_constant<int, kCap | kFar>{})
        : a.cap > 0.f ? f(std::integral_constant<int, kCap>{}) : f(std::integral_constant<int, 0>{});
}

// cap tanh(scale x / cap) of a product x, in powers of two.  tanh u = 1 - 2 / (1 + e^2u) is off
// by up to 4 * 2^-23 of the cap, whatever the score, with exponential and reciprocal within a
// step each: right for caps near the scores, but all of a score of 8 at 1e8.
struct Cap {
  float in, out;
  __device__ __forceinline__ explicit Cap(const AttendArgs& a) : in(a.cap_in), out(a.cap_out) {}
  __device__ __forceinline__ float operator()(float x) const {
    return __builtin_fmaf(-2.f * out, __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * in)), out);
  }
};

// The same for caps further off (kFar): up to u = scale x / cap = 1/2, as hardly any score
// passes, it is scale x times a polynomial in u^2, fitted to tanh(u) / u - 1 within 0.3 * 2^-24,
// so that its error is relative to the score; from there on the other form's is, too, 8 * 2^-23
// of it at most.  A prompt of 8192 tokens 712 us, with the other form 667; where scores do pass
// 1/2 it costs more (trees of 61 tokens over 6000 keys at a cap of 8 234 against 171, prompts of
// 4096 tokens with heads of 256 at 50 416 against 393), so near caps keep theirs.
struct FarCap {
  float in, scale;
  __device__ __forceinline__ explicit FarCap(const AttendArgs& a)
      : in(a.cap_in * (0.5f * kLn2)), scale(a.scale * kLog2e) {}
  // What is capped already stays as it is.
  __device__ __forceinline__ void pass() { in = 0.f, scale = 1.f; }
  __device__ __forceinline__ float operator()(float x) const {  // up to 1/2
#pragma clang fp contract(off)  // (one rounding wherever it is used: rows done again come out the same)
    const float u = x * in, z = u * u;
    float p = __builtin_fmaf(z, 0.01725699f, -0.05305295f);
    p = __builtin_fmaf(z, p, 0.13325988f);
    p = __builtin_fmaf(z, p, -0.3333315f);
    return x * scale * __builtin_fmaf(z, p, 1.f);
  }
  __device__ __forceinline__ float any(const Cap& cap, float x) const {
    return __builtin_fabsf(x * in) <= 0.5f ? (*this)(x) : cap(x);
  }
  // Whether some product of a block passes 1/2.
  template <int N, typename X>
  __device__ __forceinline__ bool passed(const X& x) const {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) most = __builtin_fmaxf(most, __builtin_fabsf(x[i]));
    return __ballot(most * in > 0.5f) != 0;
  }
};

// Scores of a block in powers of two (without a cap or slopes they stay products, which
// a factor turns into such).  ALL: every row sees all of its keys and stands behind
// them; else x of keys that the row does not see becomes -inf.
template <int MODE, bool ALL, int N, typename X>
__device__ __forceinline__ void scores(const AttendArgs& a, const Seq& s, const Row& r, int kb, int lane_key, X& x) {
  const int k0 = kb + lane_key;
  if (MODE & kCap) {
    const Cap cap(a);
    const FarCap far(a);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = MODE & kFar ? far.any(cap, x[i]) : cap(x[i]);
  }
  if (MODE & kSlopes) {
    const float sc = MODE & kCap ? 1.f : a.scale * kLog2e;
    if (ALL || (!a.prefix && !a.mask)) {  // (no key that the row sees is ahead of it)
      const float base = -r.slope * (float)(r.pos - k0);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = __builtin_fmaf(x[i], sc, __builtin_fmaf(r.slope, (float)key_of(i), base));
    } else {
      const float d = (float)(r.pos - k0);
      const float slope = a.mask && kb + 32 > s.start ? 0.f : r.slope;  // (drafted keys: below)
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = x[i] * sc - slope * __builtin_fabsf(d - (float)key_of(i));
    }
  }
  if (ALL) return;
  if (a.mask && kb + 32 > s.start) {  // a block of drafted keys
    const uint32_t bits = mask_bits(a, r.token, kb - s.start) >> lane_key;
    const bool far = a.window > 0 || a.slopes;
    const int pos = far ? key_pos(a, s, kb + (int)(threadIdx.x & 31)) : 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = k0 + key_of(i);
      bool in = k < r.upper && (k < s.start ? k >= r.lower : (bits >> key_of(i) & 1) && k >= r.first);
      if (far) {
        const int d = r.pos - __shfl(pos, lane_key + key_of(i), 64);
        in = in && (a.window == 0 || d < a.window);
        if (MODE & kSlopes) x[i] -= r.slope * __builtin_fabsf((float)d);
      }
      if (!in) x[i] = kNone;
    }
    return;
  }
  const int lower = r.lower - k0, upper = r.upper - k0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (key_of(i) < lower || key_of(i) >= upper) x[i] = kNone;
}

// Values of keys that a row does not see must not reach it, and zero times an
// infinity or NaN would.  The kernels leave out keys that no row sees (memory behind a
// sequence's end may hold anything) and take the others as they are; where a sum is not
// finite then, the rows are done again by careful() below: it sets infinities and NaN to
// zero in blocks that some rows see in part, remembers these blocks and adds what it held
// back to the rows that see it.  The sums of finite values that are large stay finite there;
// whoever adds up sums of several waves or parts normalises them first.
__device__ __forceinline__ u32x4 tame(u32x4 v, const u32x4& keep, uint32_t& odd) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t u = v[e] & keep[e];
    // the top bit of each half whose exponent is all ones, then that whole half
    const uint32_t m = ((u & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    odd |= m;
    v[e] = u & ~((m << 1) - (m >> 15));
  }
  return v;
}

// Which halves of 8 values (keys k0 + 0 .. 3 and 8 .. 11) are of keys in [lo, hi).
__device__ __forceinline__ u32x4 inside(int k0, int lo, int hi) {
  u32x4 keep;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int k = k0 + 8 * (e / 2) + 2 * (e % 2);
    keep[e] = (k >= lo && k < hi ? 0xFFFFu : 0u) | (k + 1 >= lo && k + 1 < hi ? 0xFFFF0000u : 0u);
  }
  return keep;
}

// Ones where a value is of a kind: 1 and 2 the infinities, 3 NaN.
__device__ __forceinline__ u32x4 of_kind(u32x4 v, int kind) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t out = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t x = v[e] >> (16 * b) & 0xFFFFu, size = x & 0x7FFFu;
      const int of = size < 0x7F80u ? 0 : size > 0x7F80u ? 3 : x == 0x7F80u ? 1 : 2;
      if (of == kind) out |= 0x3F80u << (16 * b);
    }
    v[e] = out;
  }
  return v;
}

// Blocks first .. last of those whose values were not all finite.
struct Odd {
  int first, last;
};

// A block of 32 keys from kb on: x holds their products with the lane's query.  ALL:
// every row sees all of them.  TAME: infinities and NaN are held back, weights are times
// kLess.  hidden: the block has no page.
template <int D, int MODE, bool ALL, bool TAME, typename V>
__device__ __forceinline__ void take(const AttendArgs& a, const Seq& s, const Row& r, const Range& g, float sc, int kb,
                                     int half, f32x16& x, bool hidden, Sums<D>& c, Odd& odd, const V& value) {
  scores<MODE, ALL, 16>(a, s, r, kb, 4 * half, x);
  if (!ALL && hidden) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = kNone;
  }
  float top = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, x[i]);
  top = larger_half(top) * sc;
  if (__ballot(top > c.m + kSlack)) {
    const float m = __builtin_fmaxf(c.m, top);
    const float f = __builtin_amdgcn_exp2f(c.m - (m == kNone ? 0.f : m));
    c.m = m;
    c.l *= f;
#pragma unroll
    for (int t = 0; t < D / 32; ++t) c.o[t] *= f;
  }
  const float m = c.m == kNone ? 0.f : c.m;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i], sc, -m));
    const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i + 1], sc, -m));
    c.l += p0 + p1;
    w[i / 2] = TAME ? pack(p0 * kLess, p1 * kLess) : pack(p0, p1);
  }
  const bf16x8 p[2] = {as_bf16x8(w[0], w[1], w[2], w[3]), as_bf16x8(w[4], w[5], w[6], w[7])};
  const int lo = hidden ? 1 << 30 : g.lo;
  if (ALL || (!TAME && kb >= lo && kb + 32 <= g.hi)) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
        c.o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value(u, t), p[u], c.o[t], 0, 0, 0);
    return;
  }
  uint32_t found = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const u32x4 keep = inside(kb + 16 * u + 4 * half, lo, g.hi);
#pragma unroll
    for (int t = 0; t < D / 32; ++t) {
      u32x4 v = __builtin_bit_cast(u32x4, value(u, t));
      v = TAME ? tame(v, keep, found) : v & keep;
      c.o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(v), p[u], c.o[t], 0, 0, 0);
    }
  }
  if (TAME && __ballot(found != 0)) {
    const int blk = kb >> 5;
    odd.first = blk < odd.first ? blk : odd.first;
    odd.last = blk > odd.last ? blk : odd.last;
  }
}

__device__ __forceinline__ int page_of(const AttendArgs& a, const Seq& s, int kb) {
  return scalar(s.table, kb >> a.page_log2);
}

// Where a block of a page stands in the keys and in the values (elements); false: the
// page is none of the cache's.
__device__ __forceinline__ bool block_at(const AttendArgs& a, const Seq& s, int kvh, int blk, int dim, int64_t& at) {
  const int kb = blk << 5, page = 1 << a.page_log2;
  const int pg = page_of(a, s, kb);
  const bool ok = (uint32_t)pg < (uint32_t)a.pages;
  at = (((int64_t)(ok ? pg : 0) * a.kv_heads + kvh) * page + (kb & (page - 1))) * dim;
  return ok;
}

// The infinities and NaN that tame() held back, added to the rows that see them.  (In
// blocks between, too, that hold none.)
template <int D, int MODE>
__device__ __forceinline__ void settle(const AttendArgs& a, const Seq& s, const Row& r, const Range& g, int kvh,
                                       int half, const Odd& odd, int step, Sums<D>& c) {
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int blk = odd.first; blk <= odd.last; blk += step) {
    const int kb = blk << 5;
    int64_t at;
    if (!block_at(a, s, kvh, blk, D, at)) continue;
    f32x16 x = {};
    scores<MODE, false, 16>(a, s, r, kb, 4 * half, x);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 16; i += 2) w[i / 2] = (x[i] == kNone ? 0u : 0x3F80u) | (x[i + 1] == kNone ? 0u : 0x3F800000u);
    const bf16x8 p[2] = {as_bf16x8(w[0], w[1], w[2], w[3]), as_bf16x8(w[4], w[5], w[6], w[7])};
#pragma unroll 1
    for (int kind = 1; kind < 4; ++kind) {
      const float add = kind == 1 ? INFINITY : kind == 2 ? -INFINITY : NAN;
      uint32_t from = 0;
      asm volatile("" : "+v"(from));  // (the values are loaded for each kind: they would fill the registers)
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        f32x16 on = {};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x4 keep = inside(kb + 16 * u + 4 * half, g.lo, g.hi);
          const u32x4 v = *(const u32x4*)(a.vc + at + from + (u * 2 + half) * 8 * D + (t * 32 + (lane & 31)) * 8) & keep;
          on = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(of_kind(v, kind)), p[u], on, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) c.o[t][i] += on[i] != 0.f ? add : 0.f;
      }
    }
  }
}

// Whether some row's sums are not finite.
template <int N, typename O>
__device__ __forceinline__ bool not_finite(const O (&o)[N], int each) {
  float v = 0.f;  // (a value less itself is not zero then; so neither is the sum of such)
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int i = 0; i < each; ++i) v += o[t][i] - o[t][i];
  return __ballot(v != 0.f) != 0;
}

// The lane's query as the second operand: 8 elements from 16 t + 8 (lane / 32) on.
template <int D>
__device__ __forceinline__ void load_query(const AttendArgs& a, const Row& r, int half, bf16x8 (&q)[D / 16]) {
  const uint16_t* p = a.q + (int64_t)r.token * a.ldq + r.head * D + 8 * half;
#pragma unroll
  for (int t = 0; t < D / 16; ++t) q[t] = *(const bf16x8*)(p + 16 * t);
}

// Four elements (d .. d + 3) of a row, normalised: to y where the keys are not split, else
// to the part's place.
__device__ __forceinline__ void put(const AttendArgs& a, const Row& r, int z, int d, f32x4 o, float weight) {
  if (a.splits > 1) {
    if (weight != 0.f)  // (else the join passes it by)
      *(f32x4*)(a.part + (((int64_t)z * a.tokens + r.token) * a.heads + r.head) * a.dim + d) = o;
    return;
  }
  if (weight == 0.f) o = f32x4{};
  const int64_t at = (int64_t)r.token * a.ldy + r.head * a.dim + d;
  if (a.y_bf16)
    *(u32x2*)((uint16_t*)a.y + at) = u32x2{pack(o.x, o.y), pack(o.z, o.w)};
  else
    *(f32x4*)((float*)a.y + at) = o;
}

__device__ __forceinline__ void put_row(const AttendArgs& a, const Row& r, int z, float m, float weight) {
  if (a.splits > 1) {
    float* p = a.part + (int64_t)a.splits * a.tokens * a.heads * a.dim;
    *(f32x2*)(p + (((int64_t)z * a.tokens + r.token) * a.heads + r.head) * 2) = f32x2{m, weight};
  } else if (a.lse) {
    a.lse[(int64_t)r.token * a.heads + r.head] = weight == 0.f ? kNone : (m + __builtin_log2f(weight)) * kLn2;
  }
}

// A wave's rows (row0 .. row0 + 31 of sequence b and head kvh) done again, over blocks
// w, w + step, ... of the parts of the keys that begin at `first` and lie `stride` apart,
// each `chunk` long, up to block last.  A function of its own that is told as little as
// possible: it is hardly ever called, and its registers are not the kernels'.  Its sums
// (not their weight) are times kLess.
template <int D, int MODE>
__device__ __attribute__((noinline)) void careful(const AttendArgs* args, int b, int kvh, int row0, int first, int chunk,
                                                  int stride, int last, int w, int step, Sums<D>* out) {
  const AttendArgs& a = *args;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const Seq s = sequence(a, b);
  const Row r = row_of(a, s, kvh, row0 + (lane & 31));
  const Range g = range_of(a, s, r);
  const float sc = MODE ? 1.f : a.scale * kLog2e;
  bf16x8 q[D / 16];
  load_query<D>(a, r, half, q);
  Sums<D> c;
  clear(c);
  for (int p0 = first; p0 < last; p0 += stride) {
    Odd odd{1 << 30, -1};
    const int p1 = p0 + chunk < last ? p0 + chunk : last;
    for (int blk = p0 + w; blk < p1; blk += step) {
      int64_t at;
      if (!block_at(a, s, kvh, blk, D, at)) continue;
      f32x16 x = {};
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
        x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*(const bf16x8*)(a.kc + at + t * 512 + lane * 8), q[t], x, 0, 0, 0);
      take<D, MODE, false, true>(a, s, r, g, sc, blk << 5, half, x, false, c, odd, [&](int u, int t) {
        return *(const bf16x8*)(a.vc + at + (u * 2 + half) * 8 * D + (t * 32 + (lane & 31)) * 8);
      });
    }
    if (odd.last >= 0) settle<D, MODE>(a, s, r, g, kvh, half, odd, step, c);
  }
  *out = c;
}

// A wave's sums times a factor, normalised, to their places.
template <int D>
__device__ __forceinline__ void put_all(const AttendArgs& a, const Row& r, int z, int half, Sums<D>& c, float times) {
  c.l += other_half(c.l);
  if (!r.live) return;
  const float f = c.l == 0.f ? 0.f : 1.f / c.l * times;
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      put(a, r, z, t * 32 + 8 * i + 4 * half,
          f32x4{c.o[t][4 * i], c.o[t][4 * i + 1], c.o[t][4 * i + 2], c.o[t][4 * i + 3]} * f, c.l);
  if (half == 0) put_row(a, r, z, c.m, c.l);
}

// (of a kernel, whose only argument an AttendArgs is)
__device__ __forceinline__ const AttendArgs* kernel_args() {
  return (const AttendArgs*)(uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
}

}  // namespace
}  // namespace uw
