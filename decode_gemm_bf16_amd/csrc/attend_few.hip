// Attention with few rows: single tokens, short runs of them, small calls.
#include "attend_core.h"

namespace uw {
namespace {

// A value's largest over the four lanes that hold one row's scores.
__device__ __forceinline__ float largest_of_row(float v) {
  const auto two = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return larger_half(__builtin_fmaxf(__uint_as_float(two[0]), __uint_as_float(two[1])));
}
__device__ __forceinline__ float sum_of_row(float v) {
  const auto two = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float w = __uint_as_float(two[0]) + __uint_as_float(two[1]);
  return w + other_half(w);
}

// The waves of a workgroup share up to 16 R rows and divide the keys.
//
// On v_mfma_f32_16x16x32_bf16, with the same arrangement: lane group g (of 16 lanes)
// takes as rows 4 g .. 4 g + 3 of the first and second product of a block the keys
// 16 (g / 2) + 4 (g % 2) + 0 .. 3 and 8 more, which are the eight that the values' order
// has for it; a row's scores lie in the four lanes of its column.
//
// Bound by HBM: each key and value is read once, from memory straight into the
// registers of the products (lines of 128 bytes whole).  A wave takes every eighth block
// of 32 keys; the keys of the next block are on their way during the softmax, its
// values during the next product.  64 sequences of up to 8192 keys, 32 heads of 128 on 8:
// 194 us (5.7 TB/s; with four waves 216, with cached loads 262 against 234); two of up to 131072
// 162 us (6.4 TB/s; four waves 184).  Heads of 256 fill 512 registers and have four waves
// (32 sequences of 8192 keys 315 us, 6.8 TB/s, against 366 with eight; two tiles of rows 194
// against 479).
//
// A workgroup has up to 32 rows of a sequence and key head (R = 2; up to 16 one tile of
// them), others the next ones; keys are read again for those, out of the L2.
template <int D, int MODE, int R>
__global__ __launch_bounds__(64 * few_waves(D), D > 128 ? 1 : 2) void attend_few_kernel(AttendArgs a) {
  constexpr int kAcross = few_waves(D);
  constexpr int kTiles = D / 16, kRound = kTiles < 8 ? kTiles : 8;  // of 16 elements; joined at once
  __shared__ __attribute__((aligned(16))) f32x4 join[kAcross][kRound][64];
  __shared__ float share[2][kAcross][16];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  const int kvh = (int)blockIdx.x % a.kv_heads, z = blockIdx.z;
  const int row0 = (int)blockIdx.x / a.kv_heads * 16 * R, row_step = (int)gridDim.x / a.kv_heads * 16 * R;
  const int lane_key = 16 * (grp >> 1) + 4 * (grp & 1);
  const Seq s = sequence(a, blockIdx.y);
  const float sc = MODE ? 1.f : a.scale * kLog2e;
  for (int r0 = row0; r0 < s.count * a.group; r0 += row_step) {
    Row r[R];
    bf16x8 q[R][D / 32];
#pragma unroll
    for (int n = 0; n < R; ++n) {
      r[n] = row_of(a, s, kvh, r0 + 16 * n + col);
      const uint16_t* p = a.q + (int64_t)r[n].token * a.ldq + r[n].head * D + 8 * grp;
#pragma unroll
      for (int t = 0; t < D / 32; ++t) q[n][t] = *(const bf16x8*)(p + 32 * t);
    }
    const Range g = range_of<R>(a, s, r);
    f32x4 o[R * kTiles];
    float m[R], l[R];
    bool again = false;  // sums that are not finite are done again with what is not finite held back
    Odd odd{1 << 30, -1};
    const int b0 = g.lo >> 5, b1 = (g.hi + 31) >> 5;  // (empty where nothing is seen)
  from_the_start:
#pragma unroll
    for (int i = 0; i < R * kTiles; ++i) o[i] = f32x4{};
#pragma unroll
    for (int n = 0; n < R; ++n) {
      m[n] = kNone;
      l[n] = 0.f;
    }
    for (int p0 = b0 + z * a.chunk; p0 < b1; p0 += a.splits * a.chunk) {
      const int p1 = p0 + a.chunk < b1 ? p0 + a.chunk : b1;
      bf16x8 kx[2][D / 32], vx[kTiles];
      auto where = [&](int blk, bool& off) {
        int64_t at;
        off = !block_at(a, s, kvh, blk < p1 ? blk : p1 - 1, D, at) || blk >= p1;
        return at;
      };
      // key lane_row (+ 8) of the block is this lane's row of the products
      const int lane_row = 16 * (col >> 3) + (col & 7);
      auto load_k = [&](int64_t at, bool off) {
        const rsrc_t b = make_rsrc(a.kc + at, off ? 0 : 64 * D);
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            kx[i][t] = as_bf16x8(ld16s(b, (grp * 32 + lane_row) * 16, t * 2048 + i * 128));
        __builtin_amdgcn_sched_barrier(0);  // (loads in one order, so that a wait for some leaves the others in flight)
      };
      auto load_v = [&](int64_t at, bool off) {
        const rsrc_t b = make_rsrc(a.vc + at, off ? 0 : 64 * D);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) vx[t] = as_bf16x8(ld16s(b, (grp * D + col) * 16, t * 256));
        __builtin_amdgcn_sched_barrier(0);
      };
      bool bad = false;
      int64_t at = where(p0 + w, bad);
      load_k(at, bad);
      load_v(at, bad);
      for (int blk = p0 + w; blk < p1; blk += kAcross) {
        bool next_bad;
        const int64_t next = where(blk + kAcross, next_bad);
        const int kb = blk << 5;
        float x[R][8];
        f32x4 product[R][2] = {};
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < R; ++n)
              product[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kx[i][t], q[n][t], product[n][i], 0, 0, 0);
#pragma unroll
        for (int n = 0; n < R; ++n)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[n][e] = product[n][e / 4][e % 4];
        __builtin_amdgcn_sched_barrier(0);
        load_k(next, next_bad);
        if (!bad && kb >= g.lo_all && kb + 32 <= g.hi_all) {
#pragma unroll
          for (int n = 0; n < R; ++n) scores<MODE, true, 8>(a, s, r[n], kb, lane_key, x[n]);
        } else {
#pragma unroll
          for (int n = 0; n < R; ++n) {
            scores<MODE, false, 8>(a, s, r[n], kb, lane_key, x[n]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (bad) x[n][i] = kNone;
          }
          if (bad || again || kb < g.lo || kb + 32 > g.hi) {  // values of places that no row sees
            const u32x4 keep = inside(kb + lane_key, bad ? 1 << 30 : g.lo, g.hi);
            uint32_t found = 0;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              u32x4 v = __builtin_bit_cast(u32x4, vx[t]) & keep;
              if (again) v = tame(v, keep, found);
              vx[t] = as_bf16x8(v);
            }
            if (__ballot(found != 0)) {
              odd.first = blk < odd.first ? blk : odd.first;
              odd.last = blk;
            }
          }
        }
#pragma unroll
        for (int n = 0; n < R; ++n) {
          float top = x[n][0];
#pragma unroll
          for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, x[n][i]);
          top = largest_of_row(top) * sc;
          if (__ballot(top > m[n] + kSlack)) {
            const float mm = __builtin_fmaxf(m[n], top);
            const float f = __builtin_amdgcn_exp2f(m[n] - (mm == kNone ? 0.f : mm));
            m[n] = mm;
            l[n] *= f;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) o[n * kTiles + t] *= f;
          }
          const float ref = m[n] == kNone ? 0.f : m[n];
          uint32_t p[4];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][i], sc, -ref));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][i + 1], sc, -ref));
            l[n] += p0 + p1;
            p[i / 2] = again ? pack(p0 * kLess, p1 * kLess) : pack(p0, p1);
          }
          const bf16x8 weights = as_bf16x8(p[0], p[1], p[2], p[3]);
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            o[n * kTiles + t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vx[t], weights, o[n * kTiles + t], 0, 0, 0);
        }
        load_v(next, next_bad);
        bad = next_bad;
      }
    }
    if (!again && not_finite(o, 4)) {
      again = true;
      goto from_the_start;
    }
    for (int blk = odd.first; blk <= odd.last; blk += kAcross) {  // what was held back, to the rows that see it
      int64_t at;
      if (!block_at(a, s, kvh, blk, D, at)) continue;
#pragma unroll
      for (int n = 0; n < R; ++n) {
        float x[8] = {};
        scores<MODE, false, 8>(a, s, r[n], blk << 5, lane_key, x);
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) p[i / 2] = (x[i] == kNone ? 0u : 0x3F80u) | (x[i + 1] == kNone ? 0u : 0x3F800000u);
        const bf16x8 seen = as_bf16x8(p[0], p[1], p[2], p[3]);
        const u32x4 keep = inside((blk << 5) + lane_key, g.lo, g.hi);
#pragma unroll 1
        for (int kind = 1; kind < 4; ++kind) {
          const float add = kind == 1 ? INFINITY : kind == 2 ? -INFINITY : NAN;
          uint32_t from = 0;
          asm volatile("" : "+v"(from));  // (the values are loaded for each kind: they would fill the registers)
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const u32x4 v = *(const u32x4*)(a.vc + at + from + (grp * D + t * 16 + col) * 8) & keep;
            const f32x4 on = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(of_kind(v, kind)), seen, f32x4{}, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n * kTiles + t][i] += on[i] != 0.f ? add : 0.f;
          }
        }
      }
    }
    // the waves' sums, brought to one maximum and normalised
#pragma unroll
    for (int n = 0; n < R; ++n) {
      l[n] = sum_of_row(l[n]);
      __syncthreads();
      if (grp == 0) {
        share[0][w][col] = m[n];
        share[1][w][col] = l[n];
      }
      __syncthreads();
      float all = kNone, weight = 0.f;
#pragma unroll
      for (int i = 0; i < kAcross; ++i) all = __builtin_fmaxf(all, share[0][i][col]);
      const float ref = all == kNone ? 0.f : all;
#pragma unroll
      for (int i = 0; i < kAcross; ++i) {
        const float e = share[1][i][col];
        weight += e == 0.f ? 0.f : e * __builtin_amdgcn_exp2f(share[0][i][col] - ref);
      }
      const float f = weight == 0.f ? 0.f : __builtin_amdgcn_exp2f(m[n] - ref) * (1.f / weight) * (again ? kMore : 1.f);
#pragma unroll
      for (int t0 = 0; t0 < kTiles; t0 += kRound) {
        if (t0) __syncthreads();
#pragma unroll
        for (int t = 0; t < kRound; ++t)
          if (t0 + t < kTiles && r[n].live) join[w][t][lane] = o[n * kTiles + t0 + t] * f;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < kRound; t += kAcross)
          if (t + w < kRound && t0 + t + w < kTiles && r[n].live) {
            f32x4 sum = join[0][t + w][lane];
#pragma unroll
            for (int k = 1; k < kAcross; ++k) sum += join[k][t + w][lane];
            put(a, r[n], z, (t0 + t + w) * 16 + 4 * grp, sum, weight);
          }
      }
      if (w == 0 && grp == 0 && r[n].live) put_row(a, r[n], z, all, weight);
    }
    __syncthreads();
  }
}

template <int D, int MODE>
void launch(const AttendArgs& a, hipStream_t s) {
  const int each = a.rows <= 16 ? 16 : 32;
  const dim3 grid((unsigned)(a.kv_heads * ((a.rows + each - 1) / each)), (unsigned)a.seqs, (unsigned)a.splits);
  if (each == 16)
    hipLaunchKernelGGL((attend_few_kernel<D, MODE, 1>), grid, dim3(64 * few_waves(D)), 0, s, a);
  else
    hipLaunchKernelGGL((attend_few_kernel<D, MODE, 2>), grid, dim3(64 * few_waves(D)), 0, s, a);
}

template <int D>
void launch_mode(const AttendArgs& a, hipStream_t s) {
  with_mode(a, [&](auto mode) { launch<D, mode.value>(a, s); });
}

}  // namespace

hipError_t launch_attend_few(const AttendArgs& a, hipStream_t s) {
  switch (a.dim) {
    case 64: launch_mode<64>(a, s); break;
    case 96: launch_mode<96>(a, s); break;
    case 128: launch_mode<128>(a, s); break;
    default: launch_mode<256>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace uw
