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
// float32.  Bound by HBM: each row is read and written once.

// cos and sin of the tile's tokens and pairs: table[i * pairs + j].
__device__ __forceinline__ void turns(const CacheWriteArgs& a, int64_t t0, int n, f32x2* table) {
  for (int x = threadIdx.x; x < n * a.pairs; x += 256) {
    const int i = x / a.pairs, j = x - i * a.pairs;
    const int axis = a.axis ? a.axis[j] : 0;
    f32x2 cs = {1.f, 0.f};
    if ((uint32_t)axis < (uint32_t)a.axes) {
      const double angle = (double)a.positions[axis * a.tokens + t0 + i] * (double)a.freqs[j];
      const double turn = 6.283185307179586476925;
      const float r = (float)__builtin_fma(-__builtin_rint(angle * (1.0 / turn)), turn, angle);
      float s, c;
      sincosf(r, &s, &c);
      cs = f32x2{c, s};
    }
    table[x] = cs;
  }
}

// Elements 8 c .. 8 c + 7 of one head, turned.  at: the head's first element.
template <bool BF16>
__device__ __forceinline__ u32x4 turned(const CacheWriteArgs& a, const void* p, int64_t at, int c, const f32x2* cs) {
  float x[8], y[8];
  load8<BF16>(p, at + 8 * c, x);
  if (a.adjacent) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 t = 4 * c + e < a.pairs ? cs[4 * c + e] : f32x2{1.f, 0.f};
      y[2 * e] = x[2 * e] * t.x - x[2 * e + 1] * t.y;
      y[2 * e + 1] = x[2 * e] * t.y + x[2 * e + 1] * t.x;
    }
  } else if (8 * c >= 2 * a.pairs) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e];
  } else if (a.pairs % 8 == 0) {
    const bool first = 8 * c < a.pairs;
    float z[8];
    load8<BF16>(p, at + 8 * c + (first ? a.pairs : -a.pairs), z);
    const f32x2* t = cs + 8 * c - (first ? 0 : a.pairs);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * t[e].x + (first ? -z[e] : z[e]) * t[e].y;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = 8 * c + e;
      if (d < a.pairs)
        y[e] = x[e] * cs[d].x - load1<BF16>(p, at + d + a.pairs) * cs[d].y;
      else if (d < 2 * a.pairs)
        y[e] = x[e] * cs[d - a.pairs].x + load1<BF16>(p, at + d - a.pairs) * cs[d - a.pairs].y;
      else
        y[e] = x[e];
    }
  }
  return u32x4{pack(y[0], y[1]), pack(y[2], y[3]), pack(y[4], y[5]), pack(y[6], y[7])};
}

template <bool BF16>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheWriteArgs a, int tile, int per) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int64_t t0 = (int64_t)blockIdx.x * tile;
  const int n = a.tokens - t0 < tile ? (int)(a.tokens - t0) : tile;
  const int nq = (a.heads + per - 1) / per, nk = (a.kv_heads + per - 1) / per;
  const int job = blockIdx.y, chunks = a.dim / 8, page = 1 << a.page_log2;
  const int64_t places = (int64_t)a.pages << a.page_log2;
  if (job < nq + nk) {
    f32x2* table = (f32x2*)lds;
    turns(a, t0, n, table);
    __syncthreads();
    const bool keys = job >= nq;
    const int h0 = (keys ? job - nq : job) * per, all = keys ? a.kv_heads : a.heads;
    const int hs = all - h0 < per ? all - h0 : per;
    for (int x = threadIdx.x; x < n * hs * chunks; x += 256) {
      if (!keys) {
        const int c = x % chunks, h = h0 + x / chunks % hs, i = x / chunks / hs;
        *(u32x4*)(a.qo + (t0 + i) * a.ldqo + h * a.dim + 8 * c) =
            turned<BF16>(a, a.q, (t0 + i) * a.ldq + h * a.dim, c, table + i * a.pairs);
      } else {
        const int i = x % n, c = x / n % chunks, h = h0 + x / n / chunks;
        const int slot = a.slots[t0 + i];
        if ((uint64_t)(int64_t)slot >= (uint64_t)places) continue;
        const int64_t at = ((int64_t)(slot >> a.page_log2) * a.kv_heads + h) * page * a.dim;
        *(u32x4*)(a.kc + at + key_at(slot & (page - 1), 8 * c, a.dim)) =
            turned<BF16>(a, a.k, (t0 + i) * a.ldk + h * a.dim, c, table + i * a.pairs);
      }
    }
    return;
  }
  // values: through LDS, so that 16 tokens that fill 16 places in order, or 4 that fill
  // 4, are written in whole pieces (16 and 8 bytes; else 2)
  uint16_t* rows = (uint16_t*)lds;                          // [tile][dim]
  int* slots = (int*)(lds + (size_t)tile * a.dim * 2);      // [tile]
  int* piece = slots + tile;                                // [tile]: tokens written from here on
  const int h0 = (job - nq - nk) * per, hs = a.kv_heads - h0 < per ? a.kv_heads - h0 : per;
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
    for (int x = threadIdx.x; x < n * chunks; x += 256) {
      const int i = x / chunks, c = x - i * chunks;
      float v[8];
      load8<BF16>(a.v, (t0 + i) * a.ldv + h * a.dim + 8 * c, v);
      *(u32x4*)(rows + i * a.dim + 8 * c) = u32x4{pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7])};
    }
    __syncthreads();
    for (int x = threadIdx.x; x < n * a.dim; x += 256) {
      const int i = x / a.dim, d = x - i * a.dim, size = piece[i];
      if (size == 0) continue;
      const int slot = slots[i];
      uint16_t* to = a.vc + ((int64_t)(slot >> a.page_log2) * a.kv_heads + h) * page * a.dim +
                     value_at(slot & (page - 1), d, a.dim);
      const uint16_t* from = rows + i * a.dim + d;
      auto two = [&](int k) { return from[k * a.dim] | (uint32_t)from[(k + 1) * a.dim] << 16; };
      if (size == 1) {
        *to = *from;
      } else if (size == 4) {
        *(u32x2*)to = u32x2{two(0), two(2)};
      } else {
        *(u32x4*)to = u32x4{two(0), two(2), two(8), two(10)};
        *(u32x4*)(to + 8 * a.dim) = u32x4{two(4), two(6), two(12), two(14)};
      }
    }
  }
}

// ---- pages ----
//
// 16 KB of a page a workgroup, 64 bytes a lane.  Bound by HBM.
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
// rise, so that row i's place is read by no later row, and 8 rows are in flight.
__global__ __launch_bounds__(256) void cache_keep_kernel(CacheKeepArgs a, int per) {
  __shared__ int from[kKeepMost], to[kKeepMost];  // places of the cache, -1: none
  __shared__ int count;
  const int b = blockIdx.x, page = 1 << a.page_log2;
  const int start = a.starts[b];
  const int32_t* table = a.tables + (int64_t)b * a.ldt;
  const int32_t* kept = a.kept + (int64_t)b * a.most;
  if (threadIdx.x == 0) count = a.most;
  __syncthreads();
  auto place = [&](int64_t at) {
    if (at < 0 || at >= (int64_t)a.max_pages << a.page_log2) return -1;
    const int pg = table[at >> a.page_log2];
    return (uint32_t)pg < (uint32_t)a.pages ? pg * page + (int)(at & (page - 1)) : -1;
  };
  const int i = threadIdx.x;
  if (i < a.most) {
    const int k = kept[i];
    if (k < 0 || (i > 0 && k <= kept[i - 1])) atomicMin(&count, i);
    from[i] = place((int64_t)start + k);
    to[i] = place((int64_t)start + i);
  }
  __syncthreads();
  const int n = count;
  if (blockIdx.y == 0 && i == 0) a.lengths[b] = start + n;
  const int each = a.dim + a.dim / 8;
  const int64_t all = (int64_t)a.layers * a.kv_heads, h0 = (int64_t)blockIdx.y * per;
  const int hs = all - h0 < per ? (int)(all - h0) : per;
  for (int x = i; x < hs * each; x += 256) {
    const int64_t lh = h0 + x / each;
    const int e = x % each;
    const int64_t layer = lh / a.kv_heads, h = lh - layer * a.kv_heads;
    const int64_t base = layer * a.pages * a.kv_heads;
    auto head = [&](int at) { return (base + (int64_t)(at >> a.page_log2) * a.kv_heads + h) * page * a.dim; };
    for (int j0 = 0; j0 < n; j0 += 8) {
      const int m = n - j0 < 8 ? n - j0 : 8;
      if (e < a.dim) {
        uint16_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = j < m ? from[j0 + j] : -1;
          if (at >= 0) v[j] = a.vc[head(at) + value_at(at & (page - 1), e, a.dim)];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = j < m && from[j0 + j] >= 0 ? to[j0 + j] : -1;
          if (at >= 0) a.vc[head(at) + value_at(at & (page - 1), e, a.dim)] = v[j];
        }
      } else {
        const int d = (e - a.dim) * 8;
        u32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = j < m ? from[j0 + j] : -1;
          if (at >= 0) v[j] = *(const u32x4*)(a.kc + head(at) + key_at(at & (page - 1), d, a.dim));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = j < m && from[j0 + j] >= 0 ? to[j0 + j] : -1;
          if (at >= 0) *(u32x4*)(a.kc + head(at) + key_at(at & (page - 1), d, a.dim)) = v[j];
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t s) {
  const int tile = a.tokens >= 1024 ? 32 : a.tokens >= 256 ? 8 : 1, per = tile == 1 ? 16 : 4;
  const unsigned jobs = (unsigned)((a.heads + per - 1) / per + 2 * ((a.kv_heads + per - 1) / per));
  const dim3 grid((unsigned)((a.tokens + tile - 1) / tile), jobs);
  const size_t table = size_t(tile) * a.pairs * 8, rows = size_t(tile) * (a.dim * 2 + 8);
  const size_t lds = table > rows ? table : rows;
  if (a.bf16)
    hipLaunchKernelGGL(cache_write_kernel<true>, grid, dim3(256), lds, s, a, tile, per);
  else
    hipLaunchKernelGGL(cache_write_kernel<false>, grid, dim3(256), lds, s, a, tile, per);
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
  const int per = heads <= 2 * 65535 ? 2 : (int)((heads + 65534) / 65535);
  const dim3 grid((unsigned)a.seqs, (unsigned)((heads + per - 1) / per));
  hipLaunchKernelGGL(cache_keep_kernel, grid, dim3(256), 0, s, a, per);
  return hipGetLastError();
}

}  // namespace uw
