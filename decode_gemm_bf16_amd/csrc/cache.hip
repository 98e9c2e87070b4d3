// Rows of a paged cache of keys and values: written with their rotary positions,
// copied by whole pages, and moved when drafted tokens are accepted.
#include "attention.h"
#include "recon.h"

namespace uw {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack(float a, float b) {  // to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ float low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if (BF16) {
    const u32x4 u = *(const u32x4*)((const uint16_t*)p + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = low(u[e]);
      x[2 * e + 1] = high(u[e]);
    }
  } else {
    const f32x4 a = *(const f32x4*)((const float*)p + at), b = *(const f32x4*)((const float*)p + at + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = a[e];
      x[4 + e] = b[e];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  return BF16 ? low(((const uint16_t*)p)[at]) : ((const float*)p)[at];
}

// ---- rotary positions and the cache's rows ----
//
// One workgroup: a tile of tokens, and some heads of the queries, of the keys or of
// the values.  Cosines and sines of the tile's tokens are computed once for its heads:
// the angle, position times frequency, is formed and brought into one turn in 64 bits
// (32 would lose 0.06 of a turn's radians at a position of 10^6), the functions are
// float32.  A lane has 8 elements of a token's heads (and, where pairs lie apart, their
// partners).  Each row is read and written once (8191 tokens, 32 and 8 heads of 128 in bf16,
// 201 MB: 48.5 us, 4.2 TB/s, where a copy reaches 5.6): waves wait for memory 83 % of their time,
// with nothing in flight from a head of the values to the next, and the one round of
// workgroups leaves the CUs idle for a fifth of it.  One token by the launch (3.0 us).

// cos and sin of the tile's tokens and pairs: table[i * pairs + j].
__device__ __forceinline__ void turns(const CacheWriteArgs& a, int64_t t0, int n, f32x2* table) {
  int log = 0;  // pairs, rounded up to a power of two
  while ((1 << log) < a.pairs) ++log;
  const int j = threadIdx.x & ((1 << log) - 1);
  if (j >= a.pairs) return;
  const int axis = a.axis ? a.axis[j] : 0;
  const bool turns = (uint32_t)axis < (uint32_t)a.axes;
  const int32_t* const at = a.positions + (turns ? axis : 0) * a.tokens + t0;
  const double freq = a.freqs[j];
  for (int i = threadIdx.x >> log; i < n; i += 256 >> log) {
    f32x2 cs = {1.f, 0.f};
    if (turns) {
      const double angle = (double)at[i] * freq;
      const double turn = 6.283185307179586476925;
      const double r = __builtin_fma(-__builtin_rint(angle * (1.0 / turn)), turn, angle);
      float s, c;
      sincospif((float)(r * (2.0 / turn)), &s, &c);
      cs = f32x2{c, s};
    }
    table[i * a.pairs + j] = cs;
  }
}

// How a lane's 8 elements (8 c .. 8 c + 7 of a head) are turned: pairs within them,
// partners 8 further on or back in whole, partners anywhere, or not at all.
enum Kind { kStay, kWithin, kBehind, kAhead, kAnywhere };
__device__ __forceinline__ Kind kind_of(const CacheWriteArgs& a, int c) {
  if (8 * c >= 2 * a.pairs) return kStay;
  if (a.adjacent) return kWithin;
  if (a.pairs % 8) return kAnywhere;
  return 8 * c < a.pairs ? kBehind : kAhead;
}

template <bool BF16>
struct Piece {
  float x[8], z[8];  // elements and partners
  __device__ __forceinline__ void load(const CacheWriteArgs& a, Kind kind, const void* p, int64_t at, int c) {
    load8<BF16>(p, at + 8 * c, x);
    if (kind == kBehind || kind == kAhead) load8<BF16>(p, at + 8 * c + (kind == kBehind ? a.pairs : -a.pairs), z);
    if (kind == kAnywhere) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = 8 * c + e;
        z[e] = d < a.pairs ? load1<BF16>(p, at + d + a.pairs) : d < 2 * a.pairs ? load1<BF16>(p, at + d - a.pairs) : 0.f;
      }
    }
  }
};

// The cosines and sines of a lane's elements, signs included.
struct Factors {
  float c[8], s[8];
  __device__ __forceinline__ void load(const CacheWriteArgs& a, Kind kind, const f32x2* cs, int chunk) {
    if (kind == kStay) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = 8 * chunk + e;
      const bool first = kind == kWithin ? e % 2 == 0 : kind == kAnywhere ? d < a.pairs : kind == kBehind;
      const int j = kind == kWithin ? d / 2 : first ? d : d - a.pairs;
      const f32x2 t = j < a.pairs ? cs[j] : f32x2{1.f, 0.f};
      c[e] = t.x;
      s[e] = first ? -t.y : t.y;
    }
  }
};

// The first `turn` of 8 elements are turned (8 and more: all); the others stay, infinities, NaN
// and signs of zero included.
template <bool BF16>
__device__ __forceinline__ u32x4 turned(Kind kind, int turn, const Piece<BF16>& p, const Factors& f) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    y[e] = kind == kStay || e >= turn ? p.x[e] : p.x[e] * f.c[e] + (kind == kWithin ? p.x[e ^ 1] : p.z[e]) * f.s[e];
  return u32x4{pack(y[0], y[1]), pack(y[2], y[3]), pack(y[4], y[5]), pack(y[6], y[7])};
}

// C: chunks of 8 elements of a head.  ONE: one token a workgroup, whose lanes have
// its heads.
template <bool BF16, int C, bool ONE>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheWriteArgs a, int tile, int per) {
  constexpr int kDim = 8 * C, kAtOnce = 256 / C;  // rows that the lanes take at once
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int n = a.tokens - t0 < tile ? (int)(a.tokens - t0) : tile;
  const int nq = (a.heads + per - 1) / per, nk = (a.kv_heads + per - 1) / per;
  const int job = blockIdx.y, page = 1 << a.page_log2;
  const int64_t places = (int64_t)a.pages << a.page_log2;
  const int c = threadIdx.x % C, first = threadIdx.x / C;
  const bool idle = first >= kAtOnce;
  if (job < nq + nk) {
    const bool keys = job >= nq;
    const int h0 = (keys ? job - nq : job) * per, all = keys ? a.kv_heads : a.heads;
    const int hs = all - h0 < per ? all - h0 : per;
    const void* const from = keys ? a.k : a.q;
    const int64_t ld = keys ? a.ldk : a.ldq;
    const Kind kind = kind_of(a, c);
    const int turn = 2 * a.pairs - 8 * c;
    f32x2* const table = (f32x2*)lds;
    auto place = [&](int i) { return keys ? a.slots[t0 + i] : 0; };
    auto put = [&](int i, int h, int slot, const u32x4& v) {
      if (!keys) {
        *(u32x4*)(a.qo + (t0 + i) * a.ldqo + h * kDim + 8 * c) = v;
      } else if ((uint64_t)(int64_t)slot < (uint64_t)places) {
        const int64_t at = ((int64_t)(slot >> a.page_log2) * a.kv_heads + h) * page * kDim;
        *(u32x4*)(a.kc + at + key_at(slot & (page - 1), 8 * c, kDim)) = v;
      }
    };
    Piece<BF16> p;
    Factors f;
    if (ONE) {
      // the first row's loads before the table
      if (!idle && first < hs) p.load(a, kind, from, t0 * ld + (h0 + first) * kDim, c);
      const int slot = place(0);
      turns(a, t0, 1, table);
      __syncthreads();
      if (idle) return;
      f.load(a, kind, table, c);
      for (int h = first; h < hs; h += kAtOnce) {
        if (h != first) p.load(a, kind, from, t0 * ld + (h0 + h) * kDim, c);
        put(0, h0 + h, slot, turned(kind, turn, p, f));
      }
    } else {
      turns(a, t0, n, table);
      __syncthreads();
      if (idle) return;
      for (int i = first; i < n; i += kAtOnce) {
        const int slot = place(i);
        f.load(a, kind, table + i * a.pairs, c);
#pragma unroll 2
        for (int h = 0; h < hs; ++h) {
          p.load(a, kind, from, (t0 + i) * ld + (h0 + h) * kDim, c);
          put(i, h0 + h, slot, turned(kind, turn, p, f));
        }
      }
    }
    return;
  }
  const int h0 = (job - nq - nk) * per, hs = a.kv_heads - h0 < per ? a.kv_heads - h0 : per;
  if (ONE) {
    const int slot = a.slots[t0];
    if (idle || (uint64_t)(int64_t)slot >= (uint64_t)places) return;
    for (int h = first; h < hs; h += kAtOnce) {
      float v[8];
      load8<BF16>(a.v, t0 * a.ldv + (h0 + h) * kDim + 8 * c, v);
      uint16_t* to = a.vc + ((int64_t)(slot >> a.page_log2) * a.kv_heads + h0 + h) * page * kDim +
                     value_at(slot & (page - 1), 8 * c, kDim);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint32_t two = pack(v[e], v[e + 1]);
        to[8 * e] = (uint16_t)two;
        to[8 * e + 8] = (uint16_t)(two >> 16);
      }
    }
    return;
  }
  // values: through LDS, so that 16 tokens that fill 16 places in order, or 4 that fill
  // 4, are written in whole pieces (16 and 8 bytes; else 2)
  uint16_t* rows = (uint16_t*)lds;                        // [tile][dim]
  int* slots = (int*)(lds + (size_t)tile * kDim * 2);     // [tile]
  int* piece = slots + tile;                              // [tile]: tokens written from here on
  for (int i = threadIdx.x; i < n; i += 256) {
    const int slot = a.slots[t0 + i];
    slots[i] = (uint64_t)(int64_t)slot < (uint64_t)places ? slot : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 256) {
    auto run = [&](int size) {  // whether this token lies in a whole run of that many
      const int from = i - (slots[i] & (size - 1)), first = slots[i] & ~(size - 1);
      if (from < 0 || from + size > n) return false;
      for (int k = 0; k < size; ++k)
        if (slots[from + k] != first + k) return false;
      return true;
    };
    piece[i] = slots[i] < 0 ? 0 : run(16) ? (slots[i] & 15 ? 0 : 16) : run(4) ? (slots[i] & 3 ? 0 : 4) : 1;
  }
  for (int h = h0; h < h0 + hs; ++h) {
    __syncthreads();
    if (!idle)
      for (int i = first; i < n; i += kAtOnce) {
        float v[8];
        load8<BF16>(a.v, (t0 + i) * a.ldv + h * kDim + 8 * c, v);
        *(u32x4*)(rows + i * kDim + 8 * c) = u32x4{pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7])};
      }
    __syncthreads();
    for (int x = threadIdx.x; x < n * kDim; x += 256) {
      const int i = x / kDim, d = x - i * kDim, size = piece[i];
      if (size == 0) continue;
      const int slot = slots[i];
      uint16_t* to = a.vc + ((int64_t)(slot >> a.page_log2) * a.kv_heads + h) * page * kDim +
                     value_at(slot & (page - 1), d, kDim);
      const uint16_t* from = rows + i * kDim + d;
      auto two = [&](int k) { return from[k * kDim] | (uint32_t)from[(k + 1) * kDim] << 16; };
      if (size == 1) {
        *to = *from;
      } else if (size == 4) {
        *(u32x2*)to = u32x2{two(0), two(2)};
      } else {
        *(u32x4*)to = u32x4{two(0), two(2), two(8), two(10)};
        *(u32x4*)(to + 8 * kDim) = u32x4{two(4), two(6), two(12), two(14)};
      }
    }
  }
}

template <bool BF16, int C>
void launch_write(const CacheWriteArgs& a, hipStream_t s) {
  // Tiles of tokens fill the lines of the values (8191 tokens by 16, 32, 64: 61.5, 49.6, 67.7
  // us), as long as there are workgroups enough; fewer heads each where there are few tokens
  // (2000 tokens with 16 and 4: 25.8 and 17.4 us).
  const int tile = a.tokens >= 1024 ? 32 : a.tokens >= 512 ? 8 : 1, per = tile > 1 && a.tokens < 6000 ? 4 : 16;
  const unsigned jobs = (unsigned)((a.heads + per - 1) / per + 2 * ((a.kv_heads + per - 1) / per));
  const dim3 grid((unsigned)((a.tokens + tile - 1) / tile), jobs);
  const size_t table = size_t(tile) * a.pairs * 8, rows = size_t(tile) * (a.dim * 2 + 8);
  const size_t lds = table > rows ? table : rows;
  if (tile == 1)
    hipLaunchKernelGGL((cache_write_kernel<BF16, C, true>), grid, dim3(256), lds, s, a, tile, per);
  else
    hipLaunchKernelGGL((cache_write_kernel<BF16, C, false>), grid, dim3(256), lds, s, a, tile, per);
}

template <bool BF16>
void launch_write(const CacheWriteArgs& a, hipStream_t s) {
  switch (a.dim) {
    case 64: launch_write<BF16, 8>(a, s); break;
    case 96: launch_write<BF16, 12>(a, s); break;
    case 128: launch_write<BF16, 16>(a, s); break;
    default: launch_write<BF16, 32>(a, s); break;
  }
}

// ---- pages ----
//
// 16 KB of a page a workgroup, 64 bytes a lane.  Bound by HBM (160 pages of 64 tokens, 8
// heads of 128, 32 layers, 2.7 GB read and written: 510 us, 5.3 TB/s; one page of 16
// layers 3.2 us).
constexpr int kCopyBytes = 16384;
__global__ __launch_bounds__(256) void cache_copy_kernel(uint8_t* kc, uint8_t* vc, int64_t pages, int64_t page_bytes,
                                                         const int32_t* src, const int32_t* dst, int64_t n) {
  const int64_t layer = blockIdx.z >> 1;
  uint8_t* const m = (blockIdx.z & 1 ? vc : kc) + layer * pages * page_bytes;
  const int64_t at = (int64_t)blockIdx.x * kCopyBytes + threadIdx.x * 16;
  for (int64_t i = blockIdx.y; i < n; i += gridDim.y) {
    const int32_t from = src[i], to = dst[i];
    if ((uint64_t)(int64_t)from >= (uint64_t)pages || (uint64_t)(int64_t)to >= (uint64_t)pages || from == to) continue;
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k * 4096 < page_bytes) v[k] = *(const u32x4*)(m + from * page_bytes + at + k * 4096);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k * 4096 < page_bytes) *(u32x4*)(m + to * page_bytes + at + k * 4096) = v[k];
  }
}

// ---- accepted drafts ----
//
// One workgroup: one sequence and some heads of all layers.  A lane moves one
// element of the values, or 8 of the keys, of every row of the list in order: entries
// rise, so that row i's place is read by no later row, and 8 rows are in flight.  Bound by
// latency: a workgroup is one chain of list, table, places and rows, and its waves wait for
// memory 87 % of their time; each works out its sequence's places again (256 times a
// sequence here), and 144 of its 256 lanes have rows to move.  64 sequences, up to 7 rows each,
// 32 layers of 8 heads of 128: 84 us.  The traffic is less: 144 to 188 MB for the 68 of the rows
// (which are 16 bytes of each 128 of the keys, 2 of each 16 of the values), 26 to 33 us at a
// copy's rate.  1, 2, 4 and 8 heads a workgroup in an earlier form: 95, 100, 108 and 120 us; one
// sequence 4 us.
template <int C>
__global__ __launch_bounds__(256) void cache_keep_kernel(CacheKeepArgs a, int per) {
  constexpr int kDim = 8 * C, kEach = kDim + C;  // a head's lanes: its values' elements, then its keys' chunks
  // first element of the values' and the keys' row in its page's first head; < 0: none
  __shared__ int64_t from[2][kKeepMost], to[2][kKeepMost];
  __shared__ int count;
  const int b = blockIdx.x, page = 1 << a.page_log2;
  const int start = a.starts[b];
  const int32_t* table = a.tables + (int64_t)b * a.ldt;
  const int32_t* kept = a.kept + (int64_t)b * a.most;
  if (threadIdx.x == 0) count = a.most;
  __syncthreads();
  auto place = [&](int64_t at, int64_t& value, int64_t& key) {
    value = key = -1;
    if (at < 0 || at >= (int64_t)a.max_pages << a.page_log2) return;
    const int pg = table[at >> a.page_log2], o = (int)(at & (page - 1));
    if ((uint32_t)pg >= (uint32_t)a.pages) return;
    const int64_t first = (int64_t)pg * a.kv_heads * page * kDim;
    value = first + value_at(o, 0, kDim);
    key = first + key_at(o, 0, kDim);
  };
  const int i = threadIdx.x;
  if (i < a.most) {
    const int k = kept[i];
    if (k < 0 || (i > 0 && k <= kept[i - 1])) atomicMin(&count, i);
    place((int64_t)start + k, from[0][i], from[1][i]);
    place((int64_t)start + i, to[0][i], to[1][i]);
    if (to[0][i] < 0 || k == i) from[0][i] = from[1][i] = -1;  // (a row that stays where it is)
  }
  __syncthreads();
  const int n = count;
  if (blockIdx.y == 0 && i == 0) a.lengths[b] = start + n;
  const int64_t all = (int64_t)a.layers * a.kv_heads, h0 = (int64_t)blockIdx.y * per;
  const int hs = all - h0 < per ? (int)(all - h0) : per;
  const int64_t layer_size = (int64_t)a.pages * a.kv_heads * page * kDim;
  for (int x = i; x < hs * kEach; x += 256) {
    const int e = x % kEach;
    const int64_t lh = h0 + x / kEach, layer = lh / a.kv_heads, head = lh - layer * a.kv_heads;
    const int64_t base = layer * layer_size + head * page * kDim;
    const bool keys = e >= kDim;
    // (a chunk of a key is 32 * 8 elements from the next, an element of a value 8)
    uint16_t* const m = (keys ? a.kc + (e - kDim) * 256 : a.vc + e * 8) + base;
    const int64_t* const f = from[keys];
    const int64_t* const t = to[keys];
    for (int j0 = 0; j0 < n; j0 += 8) {
      if (!keys) {
        uint16_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < n && f[j0 + j] >= 0) v[j] = m[f[j0 + j]];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < n && f[j0 + j] >= 0) m[t[j0 + j]] = v[j];
      } else {
        u32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < n && f[j0 + j] >= 0) v[j] = *(const u32x4*)(m + f[j0 + j]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < n && f[j0 + j] >= 0) *(u32x4*)(m + t[j0 + j]) = v[j];
      }
    }
  }
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t s) {
  a.bf16 ? launch_write<true>(a, s) : launch_write<false>(a, s);
  return hipGetLastError();
}

hipError_t launch_cache_copy(uint8_t* kc, uint8_t* vc, int64_t layers, int64_t pages, int64_t page_bytes,
                             const int32_t* src, const int32_t* dst, int64_t n, hipStream_t s) {
  const dim3 grid((unsigned)((page_bytes + kCopyBytes - 1) / kCopyBytes), (unsigned)(n < 65535 ? n : 65535),
                  (unsigned)(2 * layers));
  hipLaunchKernelGGL(cache_copy_kernel, grid, dim3(256), 0, s, kc, vc, pages, page_bytes, src, dst, n);
  return hipGetLastError();
}

hipError_t launch_cache_keep(const CacheKeepArgs& a, hipStream_t s) {
  const int64_t heads = (int64_t)a.layers * a.kv_heads;
  // one head a workgroup: 64 sequences of 256 heads, 260 rows, 95 us; 2 heads 100, 4 108, 8 120
  int64_t per = 1;
  if (heads > per * 65535) per = (heads + 65534) / 65535;
  const dim3 grid((unsigned)a.seqs, (unsigned)((heads + per - 1) / per));
  switch (a.dim) {
    case 64: hipLaunchKernelGGL(cache_keep_kernel<8>, grid, dim3(256), 0, s, a, (int)per); break;
    case 96: hipLaunchKernelGGL(cache_keep_kernel<12>, grid, dim3(256), 0, s, a, (int)per); break;
    case 128: hipLaunchKernelGGL(cache_keep_kernel<16>, grid, dim3(256), 0, s, a, (int)per); break;
    default: hipLaunchKernelGGL(cache_keep_kernel<32>, grid, dim3(256), 0, s, a, (int)per); break;
  }
  return hipGetLastError();
}

}  // namespace uw
