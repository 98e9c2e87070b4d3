// Attention with few rows a sequence: single tokens and short runs of them.
#include "attend_core.h"

namespace uw {
namespace {

// ---- few rows: the waves of a workgroup share 32 rows and divide the keys ----
//
// Bound by HBM: each key and value is read once, from memory straight into the
// registers of the products (1 KB a load instruction, in order).  A wave takes every
// fourth block of 32 keys; the keys of the next block are on their way during the
// softmax, its values during the next product.
template <int D, int MODE>
__global__ __launch_bounds__(64 * kWaves, D > 128 ? 1 : 2) void attend_few_kernel(AttendArgs a) {
  constexpr int kRound = D / 32 < 4 ? D / 32 : 4;  // blocks of 32 elements joined at once
  __shared__ __attribute__((aligned(16))) f32x4 join[kWaves][kRound][4][64];
  __shared__ float share[2][kWaves][32];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
  const int kvh = blockIdx.x, z = blockIdx.z;
  const Seq s = sequence(a, blockIdx.y);
  const float sc = MODE ? 1.f : a.scale * kLog2e;
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
        f32x16 x = {};
#pragma unroll
        for (int t = 0; t < D / 16; ++t) x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kx[t], q[t], x, 0, 0, 0);
        load_k(next, next_bad);
        auto value = [&](int u, int t) { return vx[u][t]; };
        const int kb = blk << 5;
        if (!bad && kb >= g.lo_all && kb + 32 <= g.hi_all)
          take<D, MODE, true, false>(a, s, r, g, sc, kb, half, x, false, c, odd, value);
        else
          take<D, MODE, false, false>(a, s, r, g, sc, kb, half, x, bad, c, odd, value);
        load_v(next, next_bad);
        bad = next_bad;
      }
    }
    if (not_finite(c)) {
      Sums<D> again;
      careful<D, MODE>(kernel_args(), blockIdx.y, kvh, rt * 32, b0 + z * a.chunk, a.chunk, a.splits * a.chunk, b1, w, kWaves,
                       &again);
      c = again;
    }
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

template <int D, int MODE>
void launch(const AttendArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((attend_few_kernel<D, MODE>), dim3((unsigned)a.kv_heads, (unsigned)a.seqs, (unsigned)a.splits),
                     dim3(64 * kWaves), 0, s, a);
}

template <int D>
void launch_mode(const AttendArgs& a, hipStream_t s) {
  const int mode = (a.cap > 0.f ? kCap : 0) | (a.slopes ? kSlopes : 0);
  mode == 0 ? launch<D, 0>(a, s) : mode == 1 ? launch<D, 1>(a, s) : mode == 2 ? launch<D, 2>(a, s) : launch<D, 3>(a, s);
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
