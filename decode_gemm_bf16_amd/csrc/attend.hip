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
// The weights go to the second product as bf16, the values' own type (an error of 2^-9
// a weight, on average over the keys less than the rounding of a bf16 y); scores,
// maxima, sums, and outputs until their end are float32.
#include "attention.h"
#include "recon.h"

namespace uw {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -INFINITY;
constexpr int kWaves = 4;
// A row's maximum moves only when a score is this far above it (in powers of two):
// weights stay below 2^8, and most blocks leave the sums as they are.
constexpr float kSlack = 8.f;

__device__ __forceinline__ uint32_t pack(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, 64); }

// Key of register i of S^T, less 4 (lane / 32).
__device__ __forceinline__ constexpr int key_of(int i) { return 8 * (i / 4) + i % 4; }

struct Seq {
  int t0, count, length, keys, start;  // first token, tokens, length, keys in reach of the table, length - tokens
  int prefix;
  const int32_t* table;
};

__device__ __forceinline__ int token_at(const AttendArgs& a, int t) { return t < 0 ? 0 : t > a.tokens ? a.tokens : t; }

__device__ __forceinline__ Seq sequence(const AttendArgs& a, int b) {
  Seq s;
  const int t0 = token_at(a, a.offsets[b]);
  int t1 = token_at(a, a.offsets[b + 1]);
  if (t1 < t0) t1 = t0;
  int len = a.lengths[b];
  len = len < 0 ? 0 : len > (1 << 30) ? (1 << 30) : len;
  s.t0 = __builtin_amdgcn_readfirstlane(t0);
  s.count = __builtin_amdgcn_readfirstlane(t1 - t0);
  s.length = __builtin_amdgcn_readfirstlane(len);
  const int64_t reach = (int64_t)a.max_pages << a.page_log2;
  s.keys = s.length < reach ? s.length : (int)reach;
  s.start = s.length - s.count;
  s.prefix = a.prefix ? __builtin_amdgcn_readfirstlane(a.prefix[b]) : 0;
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
  o.slope = a.slopes ? a.slopes[o.head] * kLog2e : 0.f;
  return o;
}

// Over a wave's rows: no row sees a key outside [lo, hi), every row sees all of
// [lo_all, hi_all).
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

__device__ __forceinline__ Range range_of(const AttendArgs& a, const Seq& s, const Row& r) {
  // (of a tree, drafted keys below the lower bound of the context may be seen: their
  // distance goes by their depth)
  const int top = a.mask ? s.start : r.upper;
  const int low = a.mask && r.lower > s.start ? s.start : r.lower;
  const bool any = low < r.upper;
  Range g;
  g.lo = wave_min(any ? low : 1 << 30);
  g.hi = -wave_min(any ? -r.upper : 0);
  g.lo_all = -wave_min(-r.lower);
  g.hi_all = wave_min(top);
  if (g.lo < 0) g.lo = 0;
  return g;
}

// Every row sees all keys of a block.
__device__ __forceinline__ bool whole(const Range& g, int kb) { return kb >= g.lo_all && kb + 32 <= g.hi_all; }

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

// Scores of a block in powers of two (EXTRA kernels; without them they stay products,
// which a factor turns into such).  x of keys that the row does not see becomes -inf.
template <bool EXTRA>
__device__ __forceinline__ void scores(const AttendArgs& a, const Seq& s, const Row& r, int kb, int half, bool all,
                                       f32x16& x) {
  if (EXTRA) {
    if (a.cap > 0.f) {
      const float in = a.scale / a.cap * (2.f * kLog2e), out = a.cap * kLog2e;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        x[i] = out - 2.f * out * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x[i] * in));  // cap tanh
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= a.scale * kLog2e;
    }
  }
  const int k0 = kb + 4 * half;
  if (EXTRA && a.mask && kb + 32 > s.start) {  // a block of drafted keys
    const uint32_t bits = mask_bits(a, r.token, kb - s.start) >> (4 * half);
    const bool far = a.window > 0 || a.slopes;
    const int pos = far ? key_pos(a, s, kb + (int)(threadIdx.x & 31)) : 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = k0 + key_of(i);
      bool in = k < r.upper && (k < s.start ? k >= r.lower : (bits >> key_of(i) & 1) && k >= r.first);
      if (far) {
        const int d = r.pos - __shfl(pos, 4 * half + key_of(i), 64);
        in = in && (a.window == 0 || d < a.window);
        x[i] -= r.slope * __builtin_fabsf((float)d);
      }
      if (!in) x[i] = kNone;
    }
    return;
  }
  if (EXTRA && a.slopes) {
    const float d = (float)(r.pos - k0);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] -= r.slope * __builtin_fabsf(d - (float)key_of(i));
  }
  if (!all) {
    const int lower = r.lower - k0, upper = r.upper - k0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (key_of(i) < lower || key_of(i) >= upper) x[i] = kNone;
  }
}

// Values of keys that a row does not see must not reach it, and zero times an
// infinity would.  In a block that some rows see in part, values of keys outside
// [lo, hi), infinities and NaN are set to zero; blocks with such inside are remembered
// (odd) and settled after the sums.
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

// NB blocks of 32 keys from kb on: x holds their products with the lane's query.  Bit
// n of hidden: block n has no page.
template <int D, bool EXTRA, int NB, typename V>
__device__ __forceinline__ void take(const AttendArgs& a, const Seq& s, const Row& r, const Range& g, float sc, int kb,
                                     int half, f32x16 (&x)[NB], uint32_t hidden, Sums<D>& c, Odd& odd,
                                     const V& value) {
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    scores<EXTRA>(a, s, r, kb + 32 * n, half, whole(g, kb + 32 * n), x[n]);
    if (hidden >> n & 1) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[n][i] = kNone;
    }
  }
  float top = x[0][0];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, x[n][i]);
  top = __builtin_fmaxf(top, other_half(top)) * sc;
  if (__ballot(top > c.m + kSlack)) {
    const float m = __builtin_fmaxf(c.m, top);
    const float f = __builtin_amdgcn_exp2f(c.m - (m == kNone ? 0.f : m));
    c.m = m;
    c.l *= f;
#pragma unroll
    for (int t = 0; t < D / 32; ++t) c.o[t] *= f;
  }
  const float m = c.m == kNone ? 0.f : c.m;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][i], sc, -m));
      const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][i + 1], sc, -m));
      c.l += p0 + p1;
      w[i / 2] = pack(p0, p1);
    }
    const bf16x8 p[2] = {as_bf16x8(w[0], w[1], w[2], w[3]), as_bf16x8(w[4], w[5], w[6], w[7])};
    if (!(hidden >> n & 1) && whole(g, kb + 32 * n)) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
          c.o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value(2 * n + u, t), p[u], c.o[t], 0, 0, 0);
    } else {
      uint32_t found = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const u32x4 keep = inside(kb + 32 * n + 16 * u + 4 * half, hidden >> n & 1 ? 1 << 30 : g.lo, g.hi);
#pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          const u32x4 v = tame(__builtin_bit_cast(u32x4, value(2 * n + u, t)), keep, found);
          c.o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(v), p[u], c.o[t], 0, 0, 0);
        }
      }
      if (__ballot(found != 0)) {
        const int blk = (kb >> 5) + n;
        odd.first = blk < odd.first ? blk : odd.first;
        odd.last = blk > odd.last ? blk : odd.last;
      }
    }
  }
}

__device__ __forceinline__ int page_of(const AttendArgs& a, const Seq& s, int kb) {
  return __builtin_amdgcn_readfirstlane(s.table[kb >> a.page_log2]);
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

// The infinities and NaN that tame() held back, added to the rows that see them.
template <int D, bool EXTRA>
__device__ __forceinline__ void settle(const AttendArgs& a, const Seq& s, const Row& r, const Range& g, int kvh,
                                       int half, const Odd& odd, Sums<D>& c) {
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int blk = odd.first; blk <= odd.last; ++blk) {
    const int kb = blk << 5;
    int64_t at;
    if (!block_at(a, s, kvh, blk, D, at) || whole(g, kb)) continue;
    f32x16 x = {};
    scores<EXTRA>(a, s, r, kb, half, false, x);
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

// The lane's query as the second operand: 8 elements from 16 t + 8 (lane / 32) on.
template <int D>
__device__ __forceinline__ void load_query(const AttendArgs& a, const Row& r, int half, bf16x8 (&q)[D / 16]) {
  const uint16_t* p = a.q + (int64_t)r.token * a.ldq + r.head * D + 8 * half;
#pragma unroll
  for (int t = 0; t < D / 16; ++t) q[t] = *(const bf16x8*)(p + 16 * t);
}

// Four sums of a row (elements d .. d + 3): to y where the keys are not split, else to
// the part's place.
__device__ __forceinline__ void put(const AttendArgs& a, const Row& r, int z, int d, f32x4 o, float weight) {
  if (a.splits > 1) {
    *(f32x4*)(a.part + (((int64_t)z * a.tokens + r.token) * a.heads + r.head) * a.dim + d) = o;
    return;
  }
  const float f = weight == 0.f ? 0.f : 1.f / weight;
  o = weight == 0.f ? f32x4{} : o * f;
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

// Sequence and tile of `rows` rows of the idx-th such tile of the call; false behind
// the last.
__device__ __forceinline__ bool tile_of(const AttendArgs& a, int rows, int idx, int& seq, int& tile) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += 64) {
    const int b = b0 + lane;
    int n = 0;
    if (b < a.seqs) {
      const int t0 = token_at(a, a.offsets[b]), t1 = token_at(a, a.offsets[b + 1]);
      n = t1 > t0 ? ((t1 - t0) * a.group + rows - 1) / rows : 0;
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    const uint64_t past = __ballot(before + sum > idx);
    if (past) {
      const int at = __builtin_ctzll(past);
      seq = b0 + at;
      tile = idx - before - __builtin_amdgcn_readlane(sum - n, at);
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

// ---- few rows: the waves of a workgroup share 32 rows and divide the keys ----
//
// Bound by HBM: each key and value is read once, from memory straight into the
// registers of the products (1 KB a load instruction, in order).  A wave takes every
// fourth block of 32 keys; the keys of the next block are on their way during the
// softmax, its values during the next product.
template <int D, bool EXTRA>
__global__ __launch_bounds__(64 * kWaves, D > 128 ? 1 : 2) void attend_few_kernel(AttendArgs a) {
  constexpr int kRound = D / 32 < 4 ? D / 32 : 4;  // blocks of 32 elements joined at once
  __shared__ __attribute__((aligned(16))) f32x4 join[kWaves][kRound][4][64];
  __shared__ float share[2][kWaves][32];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
  const int kvh = blockIdx.x, z = blockIdx.z;
  const Seq s = sequence(a, blockIdx.y);
  const float sc = EXTRA ? 1.f : a.scale * kLog2e;
  for (int rt = 0; rt * 32 < s.count * a.group; ++rt) {
    const Row r = row_of(a, s, kvh, rt * 32 + (lane & 31));
    const Range g = range_of(a, s, r);
    bf16x8 q[D / 16];
    load_query<D>(a, r, half, q);
    Sums<D> c;
    clear(c);
    Odd odd{1 << 30, -1};
    const int b0 = g.lo >> 5, b1 = (g.hi + 31) >> 5;  // (empty where nothing is seen)
    for (int p0 = b0 + z * a.chunk; p0 < b1; p0 += a.splits * a.chunk) {
      const int p1 = p0 + a.chunk < b1 ? p0 + a.chunk : b1;
      bf16x8 kx[D / 16], vx[2][D / 32];
      bool bad = false;
      auto where = [&](int blk, bool& off) {
        int64_t at;
        off = !block_at(a, s, kvh, blk < p1 ? blk : p1 - 1, D, at) || blk >= p1;
        return at;
      };
      auto load_k = [&](int64_t at, bool off) {
        const rsrc_t b = make_rsrc(a.kc + at, off ? 0 : 64 * D);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) kx[t] = as_bf16x8(ld16s(b, lane * 16, t * 1024));
      };
      auto load_v = [&](int64_t at, bool off) {
        const rsrc_t b = make_rsrc(a.vc + at, off ? 0 : 64 * D);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < D / 32; ++t)
            vx[u][t] = as_bf16x8(ld16s(b, (half * D + (lane & 31)) * 16, u * 32 * D + t * 512));
      };
      int64_t at = where(p0 + w, bad);
      load_k(at, bad);
      load_v(at, bad);
      for (int blk = p0 + w; blk < p1; blk += kWaves) {
        bool next_bad;
        const int64_t next = where(blk + kWaves, next_bad);
        f32x16 x[1] = {};
#pragma unroll
        for (int t = 0; t < D / 16; ++t) x[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kx[t], q[t], x[0], 0, 0, 0);
        load_k(next, next_bad);
        take<D, EXTRA, 1>(a, s, r, g, sc, blk << 5, half, x, bad ? 1u : 0u, c, odd, [&](int u, int t) { return vx[u][t]; });
        load_v(next, next_bad);
        bad = next_bad;
      }
    }
    if (odd.last >= 0) settle<D, EXTRA>(a, s, r, g, kvh, half, odd, c);
    // the waves' sums, brought to one maximum
    c.l += other_half(c.l);
    if (half == 0) {
      share[0][w][lane] = c.m;
      share[1][w][lane] = c.l;
    }
    __syncthreads();
    float m = kNone, weight = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) m = __builtin_fmaxf(m, share[0][i][lane & 31]);
    const float ref = m == kNone ? 0.f : m;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const float l = share[1][i][lane & 31];
      weight += l == 0.f ? 0.f : l * __builtin_amdgcn_exp2f(share[0][i][lane & 31] - ref);
    }
    const float f = __builtin_amdgcn_exp2f(c.m - ref);
#pragma unroll
    for (int t0 = 0; t0 < D / 32; t0 += kRound) {
      if (t0) __syncthreads();
#pragma unroll
      for (int t = 0; t < kRound; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x16 o = c.o[t0 + t < D / 32 ? t0 + t : 0] * f;
          if (r.live) join[w][t][i][lane] = f32x4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
        }
      __syncthreads();
      if (w < kRound && t0 + w < D / 32 && r.live) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 o = join[0][w][i][lane];
#pragma unroll
          for (int k = 1; k < kWaves; ++k) o += join[k][w][i][lane];
          put(a, r, z, (t0 + w) * 32 + 8 * i + 4 * half, o, weight);
        }
      }
    }
    if (w == 0 && half == 0 && r.live) put_row(a, r, z, m, weight);
    __syncthreads();
  }
}

// ---- many rows: 128 of them a workgroup, 32 a wave, keys and values shared in LDS ----
template <int D, bool EXTRA>
__global__ __launch_bounds__(64 * kWaves, D > 128 ? 1 : 2) void attend_many_kernel(AttendArgs a) {
  constexpr int kBlocks = D > 128 ? 1 : 2;  // of 32 keys at a time
  constexpr int kBytes = 64 * D;            // of a block's keys, or values
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2 * kBlocks][kBytes];
  __shared__ int range[2][kWaves];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
  const int kvh = (int)(gridDim.x - 1 - blockIdx.x) % a.kv_heads, z = blockIdx.y;
  int b, rt;
  // the last rows of a sequence see the most keys: they go first
  if (!tile_of(a, 32 * kWaves, (int)(gridDim.x - 1 - blockIdx.x) / a.kv_heads, b, rt)) return;
  const Seq s = sequence(a, b);
  const float sc = EXTRA ? 1.f : a.scale * kLog2e;
  {
    const int r0 = (rt * kWaves + w) * 32;
    const Row r = row_of(a, s, kvh, r0 + (lane & 31));
    const Range g = range_of(a, s, r);
    if (lane == 0) {
      range[0][w] = g.lo;
      range[1][w] = g.hi;
    }
    bf16x8 q[D / 16];
    load_query<D>(a, r, half, q);
    Sums<D> c;
    clear(c);
    Odd odd{1 << 30, -1};
    __syncthreads();
    int lo = range[0][0], hi = range[1][0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
      lo = range[0][i] < lo ? range[0][i] : lo;
      hi = range[1][i] > hi ? range[1][i] : hi;
    }
    const int b0 = __builtin_amdgcn_readfirstlane(lo) >> 5, b1 = (__builtin_amdgcn_readfirstlane(hi) + 31) >> 5;
    for (int p0 = b0 + z * a.chunk; p0 < b1; p0 += a.splits * a.chunk) {
      const int p1 = p0 + a.chunk < b1 ? p0 + a.chunk : b1;
      // blocks without a page in the cache are hidden (bit n of the result)
      auto fetch = [&](int blk, int buf) {
        uint32_t off = 0;
#pragma unroll
        for (int n = 0; n < kBlocks; ++n) {
          int64_t at;
          const bool bad = !block_at(a, s, kvh, blk + n < p1 ? blk + n : p1 - 1, D, at) || blk + n >= p1;
          off |= bad ? 1u << n : 0u;
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // keys, values
            const rsrc_t b = make_rsrc((i ? a.vc : a.kc) + at, bad ? 0 : kBytes);
#pragma unroll
            for (int t = 0; t < kBytes / 1024; t += kWaves) {
              if (t + w < kBytes / 1024)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    b, (__attribute__((address_space(3))) void*)(&lds[buf][i * kBlocks + n][(t + w) * 1024]), 16,
                    lane * 16, (t + w) * 1024, 0, 0);
            }
          }
        }
        return off;
      };
      uint32_t hidden = fetch(p0, 0), next = 0;
      int buf = 0;
      for (int blk = p0; blk < p1; blk += kBlocks, buf ^= 1) {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (blk + kBlocks < p1) next = fetch(blk + kBlocks, buf ^ 1);
        const int kb = blk << 5;
        if (kb < g.hi && kb + 32 * kBlocks > g.lo) {
          f32x16 x[kBlocks] = {};
#pragma unroll
          for (int n = 0; n < kBlocks; ++n)
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
              x[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*(const bf16x8*)&lds[buf][n][t * 1024 + lane * 16], q[t],
                                                             x[n], 0, 0, 0);
          take<D, EXTRA, kBlocks>(a, s, r, g, sc, kb, half, x, hidden, c, odd, [&](int u, int t) {
            return *(const bf16x8*)&lds[buf][kBlocks + u / 2][u % 2 * 32 * D + (half * D + t * 32 + (lane & 31)) * 16];
          });
        }
        hidden = next;
      }
      __syncthreads();
    }
    if (odd.last >= 0) settle<D, EXTRA>(a, s, r, g, kvh, half, odd, c);
    c.l += other_half(c.l);
    if (r.live) {
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          put(a, r, z, t * 32 + 8 * i + 4 * half, f32x4{c.o[t][4 * i], c.o[t][4 * i + 1], c.o[t][4 * i + 2], c.o[t][4 * i + 3]},
              c.l);
      if (half == 0) put_row(a, r, z, c.m, c.l);
    }
    __syncthreads();
  }
}

// ---- the parts of split keys, joined ----
//
// A workgroup joins 8 rows, or one row whose parts its 8 groups of 32 lanes divide
// (ONE), 4 elements of 32 columns a lane.
template <bool ONE>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
  __shared__ __attribute__((aligned(16))) float red[8][256];
  const int grp = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.tokens * a.heads;
  const int first = a.offsets[0], last = a.offsets[a.seqs];
  const float* const ml = a.part + (int64_t)a.splits * rows * a.dim;
  for (int64_t r0 = blockIdx.x; r0 * (ONE ? 1 : 8) < rows; r0 += gridDim.x) {
    const int64_t row = ONE ? r0 : r0 * 8 + grp;
    const int t = (int)(row / a.heads), h = (int)(row - (int64_t)t * a.heads);
    const bool live = row < rows && t >= first && t < last;
    float m = kNone, weight = 0.f;
    f32x4 o[2] = {};
    if (live) {
      for (int z = 0; z < a.splits; ++z) m = __builtin_fmaxf(m, ml[((int64_t)z * rows + row) * 2]);
      const float ref = m == kNone ? 0.f : m;
      for (int z = 0; z < a.splits; ++z) {
        const f32x2 e = *(const f32x2*)(ml + ((int64_t)z * rows + row) * 2);
        if (e.y == 0.f) continue;
        const float f = __builtin_amdgcn_exp2f(e.x - ref);
        weight += e.y * f;
        if (ONE && (z & 7) != grp) continue;
        const float* p = a.part + ((int64_t)z * rows + row) * a.dim;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int d = i * 128 + l * 4;
          if (d < a.dim) o[i] += f * *(const f32x4*)(p + d);
        }
      }
    }
    if (ONE) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = i * 128 + l * 4;
        if (d < a.dim) *(f32x4*)&red[grp][d] = o[i];
      }
      __syncthreads();
      if (grp) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = i * 128 + l * 4;
        if (d < a.dim)
          for (int k = 1; k < 8; ++k) o[i] += *(const f32x4*)&red[k][d];
      }
    }
    if (!live) continue;
    const float f = weight == 0.f ? 0.f : 1.f / weight;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = i * 128 + l * 4;
      if (d >= a.dim) continue;
      const f32x4 v = weight == 0.f ? f32x4{} : o[i] * f;
      const int64_t at = (int64_t)t * a.ldy + h * a.dim + d;
      if (a.y_bf16)
        *(u32x2*)((uint16_t*)a.y + at) = u32x2{pack(v.x, v.y), pack(v.z, v.w)};
      else
        *(f32x4*)((float*)a.y + at) = v;
    }
    if (a.lse && l == 0) a.lse[row] = weight == 0.f ? kNone : (m + __builtin_log2f(weight)) * kLn2;
  }
}

template <int D, bool EXTRA>
void launch(const AttendArgs& a, bool wide, hipStream_t s) {
  if (wide) {
    const int64_t tiles = (int64_t)a.tokens * a.group / (32 * kWaves) + a.seqs;  // at most
    hipLaunchKernelGGL((attend_many_kernel<D, EXTRA>), dim3((unsigned)(tiles * a.kv_heads), (unsigned)a.splits),
                       dim3(64 * kWaves), 0, s, a);
  } else {
    hipLaunchKernelGGL((attend_few_kernel<D, EXTRA>), dim3((unsigned)a.kv_heads, (unsigned)a.seqs, (unsigned)a.splits),
                       dim3(64 * kWaves), 0, s, a);
  }
}

}  // namespace

// Parts of the keys: enough workgroups to fill the chip, of at least so many keys.
AttendPlan attend_plan(int64_t tokens, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim, int64_t max_tokens,
                       int64_t max_length) {
  AttendPlan p;
  const int64_t group = heads / kv_heads, per = 32 * kWaves;
  p.wide = max_tokens * group > 32;
  int64_t tiles = seqs;
  if (p.wide) {
    const int64_t most = tokens * group / per + seqs;
    tiles *= (max_tokens * group + per - 1) / per;
    if (tiles > most) tiles = most;
  }
  const int64_t groups = tiles * kv_heads, blocks = (max_length + 31) / 32;
  const int64_t want = p.wide ? 512 : 2048, least = p.wide ? 16 : 8;  // workgroups; blocks of a part
  int64_t splits = (want + groups - 1) / groups;
  const int64_t most = blocks / least > 1 ? blocks / least : 1;
  if (splits > most) splits = most;
  if (splits > 256) splits = 256;
  int64_t chunk = (blocks + splits - 1) / splits;
  chunk = (chunk + kWaves - 1) / kWaves * kWaves;
  p.chunk = (int32_t)chunk;
  p.splits = (int32_t)((blocks + chunk - 1) / chunk);
  p.bytes = p.splits > 1 ? size_t(p.splits) * size_t(tokens) * heads * (dim + 2) * 4 : 0;
  return p;
}

hipError_t launch_attend(const AttendArgs& args, const AttendPlan& p, hipStream_t s) {
  AttendArgs a = args;
  a.splits = p.splits;
  a.chunk = p.chunk;
  const bool extra = a.cap > 0.f || a.slopes || a.mask;
  switch (a.dim) {
    case 64: extra ? launch<64, true>(a, p.wide, s) : launch<64, false>(a, p.wide, s); break;
    case 96: extra ? launch<96, true>(a, p.wide, s) : launch<96, false>(a, p.wide, s); break;
    case 128: extra ? launch<128, true>(a, p.wide, s) : launch<128, false>(a, p.wide, s); break;
    default: extra ? launch<256, true>(a, p.wide, s) : launch<256, false>(a, p.wide, s); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.tokens * a.heads, groups = a.splits > 16 ? rows : (rows + 7) / 8;
  const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
  if (a.splits > 16)
    hipLaunchKernelGGL(attend_join_kernel<true>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(attend_join_kernel<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace uw
