// Rows grouped by an index (a token's experts, a request's adapter), copied to
// their groups and combined on the way back.
#include "recon.h"
#include "routing.h"

namespace uw {
namespace {

__device__ __forceinline__ uint16_t to_bf16(float f) {  // round to nearest even, NaN stays NaN
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + (((u >> 16) & 1u) + 0x7FFFu)) >> 16);
}

// ---- grouping: a stable counting sort ----
//
// The entries are cut into one section per wave, in order.  Each wave counts
// its section's labels (label = group, or `groups` for ungrouped entries) into
// its own row of LDS counters; a prefix sum over the waves and then over the
// labels turns the counters into each (wave, label)'s first position; each
// wave then walks its section again, 64 entries at a time, and an entry's
// position is its counter plus its rank among the equal labels of the 64.  No
// position depends on the order in which atomics are served.
//
// A lane reads kKept entries at once and keeps its section's first kKept from the
// counting to the placing, so that most sections are read once.
//
// Up to kOneBlock entries one workgroup does all of it (in a graph, 8 and 256
// groups: 1024 entries 4.1 and 4.8 us against 6.3 and 7.2 in two launches, 4096 6.1
// and 7.6 against 7.1 and 7.9, 8192 9.1 and 12.0 against 7.2 and 8.1).  Beyond, a
// first kernel writes each workgroup's counts and in the second each workgroup sums
// the counts of those before it by itself (65536 entries 8.4 and 9.6 us, 2^21 20.9
// and 29).

constexpr int64_t kOneBlock = 4096;
constexpr int kMaxBlocks = 256;
constexpr int kKept = 4;

// Waves of a workgroup: their counters and the labels' totals stay within 64 KB of LDS.
int waves_of(int32_t groups) { return groups < 900 ? 16 : groups < 1700 ? 8 : groups < 3000 ? 4 : 2; }

// Waves of the single workgroup: one for each 64 entries, up to waves_of.
int waves_one(int64_t n, int32_t groups) {
  const int64_t want = (n + 63) / 64, most = waves_of(groups);
  return (int)(want < most ? want : most);
}

// Entries per workgroup, a multiple of 64 per wave.  64 workgroups, because each
// reads the counts of all; with that at least one entry a lane (16384 of 256 groups
// 8.2 us against 9.0 with two) and at most the kKept that are read once (2^19
// entries 15.5 us against 17.8 with two), as far as kMaxBlocks workgroups do.
int64_t chunk_of(int64_t n, int waves) {
  const int64_t step = 64 * waves;
  if (n <= kOneBlock) return (n + step - 1) / step * step;
  const int64_t want = (n + 63) / 64, most = (n + kMaxBlocks - 1) / kMaxBlocks;
  const int64_t c = most > kKept * step ? most : want > kKept * step ? kKept * step : want;
  return (c + step - 1) / step * step;
}

__device__ __forceinline__ int label_of(const GroupArgs& a, int64_t i) {
  const int32_t v = a.index[i];
  return (uint32_t)v < (uint32_t)a.groups ? v : a.groups;
}

// Labels of entries lo + t, lo + t + step, ... < hi (-1 past them).  The loads are
// not under a condition, so that they are in flight together.
template <int KEPT>
__device__ __forceinline__ void labels_of(const GroupArgs& a, int64_t lo, int64_t hi, int t, int step, int (&g)[KEPT]) {
#pragma unroll
  for (int k = 0; k < KEPT; ++k) {
    const int64_t i = lo + t + k * step;
    g[k] = label_of(a, i < hi ? i : a.n - 1);
  }
#pragma unroll
  for (int k = 0; k < KEPT; ++k)
    if (lo + t + k * step >= hi) g[k] = -1;
}

// Counts them.  Entries of one label stand together in many batches (a request's
// tokens): a wave whose entries are equal adds them at once instead of one after the
// other.
template <int KEPT>
__device__ __forceinline__ void count(int* ctr, const int (&labels)[KEPT]) {
  int g[KEPT];
#pragma unroll
  for (int k = 0; k < KEPT; ++k) g[k] = labels[k];
#pragma unroll 1
  for (int k = 0; k < KEPT; ++k) {
    const uint64_t there = __ballot(g[0] >= 0);
    if (there == 0) break;
    const int from = __builtin_ctzll(there), first = __builtin_amdgcn_readlane(g[0], from);
    if (__ballot(g[0] == first) != there) {
      if (g[0] >= 0) atomicAdd(&ctr[g[0]], 1);
    } else if ((int)(threadIdx.x & 63) == from) {
      atomicAdd(&ctr[first], (int)__popcll(there));
    }
#pragma unroll
    for (int m = 1; m < KEPT; ++m) g[m - 1] = g[m];
  }
}

__global__ __launch_bounds__(1024) void group_count_kernel(GroupArgs a, int64_t chunk) {
  extern __shared__ int ctr[];  // [groups + 1]
  const int labels = a.groups + 1;
  for (int g = threadIdx.x; g < labels; g += blockDim.x) ctr[g] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < a.n ? lo + chunk : a.n;
  for (int64_t i0 = lo; i0 < hi; i0 += kKept * blockDim.x) {
    int g[kKept];
    labels_of(a, i0, hi, threadIdx.x, blockDim.x, g);
    count(ctr, g);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < labels; g += blockDim.x) a.work[(int64_t)blockIdx.x * labels + g] = ctr[g];
}

// Exclusive sum of v over the workgroup's threads; wsum: LDS for 16 waves.
__device__ __forceinline__ int block_scan(int v, int* wsum) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nw = blockDim.x >> 6;
  int x = v;
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) wsum[w] = x;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < nw; ++i) before += i < w ? wsum[i] : 0;
  return before + x - v;
}

template <bool MULTI, int KEPT>
__global__ __launch_bounds__(1024) void group_place_kernel(GroupArgs a, int64_t chunk) {
  extern __shared__ int ctr[];  // [waves][groups + 1], then each label's total, later its first position
  __shared__ int wsum[16];
  const int labels = a.groups + 1, nw = blockDim.x >> 6, w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int* const base = ctr + nw * labels;
  for (int i = threadIdx.x; i < nw * labels; i += blockDim.x) ctr[i] = 0;
  __syncthreads();
  const int64_t sec = chunk / nw;
  const int64_t lo = blockIdx.x * chunk + w * sec, hi = lo + sec < a.n ? lo + sec : a.n;
  int* const mine = ctr + w * labels;
  int kept[KEPT];  // the section's first entries; the rest is read twice
  labels_of(a, lo, hi, lane, 64, kept);
  count(mine, kept);
  for (int64_t i0 = lo + KEPT * 64; i0 < hi; i0 += KEPT * 64) {
    int g[KEPT];
    labels_of(a, i0, hi, lane, 64, g);
    count(mine, g);
  }
  __syncthreads();
  // this thread's labels: their counts over all entries and in the workgroups before
  const int per = (labels + blockDim.x - 1) / blockDim.x;
  const int g0 = threadIdx.x * per, g1 = g0 + per < labels ? g0 + per : labels;
  int sum = 0, tiles = 0;
  for (int g = g0; g < g1; ++g) {
    int all = 0, run = 0;
    if (MULTI) {
      const int32_t* h = a.work + g;
      const int blocks = gridDim.x;
      auto add = [&](int b, int v) {
        all += v;
        run += b < (int)blockIdx.x ? v : 0;
      };
      int b = 0;
      for (; b + 16 <= blocks; b += 16) {
        int v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = h[(int64_t)(b + k) * labels];
#pragma unroll
        for (int k = 0; k < 16; ++k) add(b + k, v[k]);
      }
      for (; b < blocks; b += 8) {  // as many loads in flight, also where fewer are left
        int v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = h[(int64_t)(b + k < blocks ? b + k : blocks - 1) * labels];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (b + k < blocks) add(b + k, v[k]);
      }
    }
    for (int i = 0; i < nw; ++i) {
      const int v = ctr[i * labels + g];
      ctr[i * labels + g] = run;
      run += v;
    }
    if (!MULTI) all = run;
    base[g] = all;
    sum += all;
    tiles += (all + kPlanTile - 1) / kPlanTile;
  }
  int first = block_scan(sum, wsum);
  const bool plan = a.header && blockIdx.x == 0;
  int tile = plan ? block_scan(tiles, wsum) : 0;
  for (int g = g0; g < g1; ++g) {
    const int c = base[g];
    base[g] = first;
    if (blockIdx.x == 0 && a.offsets) a.offsets[g] = first;
    if (plan) {
      for (int r = 0; r < c; r += kPlanTile)
        a.tiles[tile++] = PlanTile{first + r, c - r < kPlanTile ? c - r : kPlanTile, g < a.groups ? g : -1, 0};
      if (g == labels - 1) *a.header = PlanHeader{(int32_t)a.n, a.groups, tile, 0};
    }
    first += c;
  }
  __syncthreads();
  int bits = 0;
  while ((1 << bits) < labels) ++bits;
  auto place = [&](int64_t i, int label) {
    const bool there = label >= 0;
    const int g = there ? label : 0;
    uint64_t same = __ballot(there);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((g >> b) & 1);
      same &= (g >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (there) {
      const int at = base[g] + mine[g] + rank;
      a.order[at] = (int32_t)i;
      if (a.slot) a.slot[i] = g < a.groups ? at : -1;
    }
    __builtin_amdgcn_wave_barrier();
    if (there && rank == 0) mine[g] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
  };
  for (int64_t i0 = lo; i0 < hi; i0 += KEPT * 64) {
    if (i0 > lo) labels_of(a, i0, hi, lane, 64, kept);
#pragma unroll 1
    for (int64_t i = i0; i < hi && i < i0 + KEPT * 64; i += 64) {
      place(i + lane, kept[0]);
#pragma unroll
      for (int m = 1; m < KEPT; ++m) kept[m - 1] = kept[m];
    }
  }
}

// ---- dispatch and combine ----

// One workgroup copies 2048 columns of one token's row to its top_k places:
// the row is read once, whatever top_k is.  Bound by HBM.  STREAM: the stores
// pass the caches by, for copies that would not fit them before they are read
// (8191 tokens x 8 of 2048 columns: 51.4 us, 5.7 TB/s; 59.4 without).
template <bool STREAM>
__global__ __launch_bounds__(256) void dispatch_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                       const int32_t* __restrict__ slot, int64_t tokens, int top_k,
                                                       int64_t cols, uint16_t* __restrict__ xs, uint32_t rows) {
  const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= cols) return;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    const u32x4 v = *(const u32x4*)(x + t * ldx + c);
    for (int j = 0; j < top_k; ++j) {
      const int32_t at = slot[t * top_k + j];
      if ((uint32_t)at >= rows) continue;
      u32x4* to = (u32x4*)(xs + at * cols + c);
      if (STREAM)
        __builtin_nontemporal_store(v, to);
      else
        *to = v;
    }
  }
}

// One workgroup: 1024 columns of one token.  y may be base (each element is
// read before it is written, by one lane).  Sums in float32, top_k terms in
// order; entries without a row (slot outside 0..rows-1) add nothing (their load
// goes to row 0, so that kBatch loads are in flight without a branch between).
// Bound by HBM: 8191 tokens x 8 of 2048 columns to bf16 99 us, 5.6 TB/s, the
// rate of a large copy (108 us with loads that keep ys, read once, in the caches).
constexpr int kBatch = 4;
template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ ys, const int32_t* __restrict__ slot,
                                                      const float* __restrict__ weight, int64_t tokens, int top_k,
                                                      int64_t cols, uint32_t rows, const float* base, void* y) {
  const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
  if (c >= cols) return;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < top_k; j0 += kBatch) {
      f32x4 v[kBatch];
      uint32_t at[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        at[j] = j0 + j < top_k ? (uint32_t)slot[t * top_k + j0 + j] : rows;
        v[j] = __builtin_nontemporal_load((const f32x4*)(ys + (int64_t)(at[j] < rows ? at[j] : 0) * cols + c));
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (at[j] < rows) s += weight[t * top_k + j0 + j] * v[j];
    }
    if (base) s += *(const f32x4*)(base + t * cols + c);
    if (BF16)
      *(u32x2*)((uint16_t*)y + t * cols + c) =
          u32x2{to_bf16(s.x) | (uint32_t)to_bf16(s.y) << 16, to_bf16(s.z) | (uint32_t)to_bf16(s.w) << 16};
    else
      *(f32x4*)((float*)y + t * cols + c) = s;
  }
}

// A grid of at most 2^20 workgroups along the tokens (HIP bounds a grid to
// 2^32 threads); the kernels stride over the rest.
unsigned token_blocks(int64_t tokens) { return (unsigned)(tokens < (1 << 20) ? tokens : (1 << 20)); }

}  // namespace

size_t group_work_bytes(int64_t n, int32_t groups) {
  if (n <= kOneBlock) return 0;
  const int64_t chunk = chunk_of(n, waves_of(groups));
  return size_t((n + chunk - 1) / chunk) * size_t(groups + 1) * 4;
}

hipError_t launch_group_rows(const GroupArgs& a, hipStream_t s) {
  const bool one = a.n <= kOneBlock;
  const int waves = one ? waves_one(a.n, a.groups) : waves_of(a.groups), labels = a.groups + 1;
  const int64_t chunk = chunk_of(a.n, waves);
  const size_t lds = size_t(waves + 1) * labels * 4;
  if (one) {
    if (chunk == 64 * waves)
      hipLaunchKernelGGL((group_place_kernel<false, 1>), dim3(1), dim3(64 * waves), lds, s, a, chunk);
    else
      hipLaunchKernelGGL((group_place_kernel<false, kKept>), dim3(1), dim3(64 * waves), lds, s, a, chunk);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.n + chunk - 1) / chunk));
  hipLaunchKernelGGL(group_count_kernel, grid, dim3(64 * waves), size_t(labels) * 4, s, a, chunk);
  hipLaunchKernelGGL((group_place_kernel<true, kKept>), grid, dim3(64 * waves), lds, s, a, chunk);
  return hipGetLastError();
}

hipError_t launch_dispatch_rows(const uint16_t* x, int64_t ldx, const int32_t* slot, int64_t tokens, int32_t top_k,
                                int64_t cols, uint16_t* xs, int64_t rows, hipStream_t s) {
  const dim3 grid(token_blocks(tokens), (unsigned)((cols + 2047) / 2048));
  // half of the 256 MB Infinity Cache
  if (tokens * top_k * cols * 2 >= (int64_t(128) << 20))
    hipLaunchKernelGGL(dispatch_kernel<true>, grid, dim3(256), 0, s, x, ldx, slot, tokens, (int)top_k, cols, xs,
                       (uint32_t)rows);
  else
    hipLaunchKernelGGL(dispatch_kernel<false>, grid, dim3(256), 0, s, x, ldx, slot, tokens, (int)top_k, cols, xs,
                       (uint32_t)rows);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const float* ys, const int32_t* slot, const float* weight, int64_t tokens,
                               int32_t top_k, int64_t cols, int64_t rows, const float* base, void* y, bool y_bf16,
                               hipStream_t s) {
  const dim3 grid(token_blocks(tokens), (unsigned)((cols + 1023) / 1024));
  if (y_bf16)
    hipLaunchKernelGGL(combine_kernel<true>, grid, dim3(256), 0, s, ys, slot, weight, tokens, (int)top_k, cols,
                       (uint32_t)rows, base, y);
  else
    hipLaunchKernelGGL(combine_kernel<false>, grid, dim3(256), 0, s, ys, slot, weight, tokens, (int)top_k, cols,
                       (uint32_t)rows, base, y);
  return hipGetLastError();
}

}  // namespace uw
