// The sums of split keys, joined; and the rule that splits them.
#include "attend_core.h"

namespace uw {
namespace {

// ---- the parts of split keys, joined ----
//
// A workgroup joins 8 rows, 32 lanes each, or one row whose parts its 8 groups of 32
// lanes divide (ONE).  Up to 8 parts, and 256: a lane has each part's maximum and weight;
// then 4 elements of 32 columns a lane (H: twice, of long heads), the loads of
// several parts in flight.
__device__ __forceinline__ float max32(float v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ float sum32(float v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <bool ONE, int H>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
  constexpr int kJoinAtOnce = ONE ? 4 : 2;
  __shared__ __attribute__((aligned(16))) float red[8][256];
  __shared__ float factor[256], tops[8], weights[8];
  const int grp = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.tokens * a.heads;
  const int first = a.offsets[0], last = a.offsets[a.seqs];
  const float* const ml = a.part + (int64_t)a.splits * rows * a.dim;
  for (int64_t r0 = blockIdx.x; r0 * (ONE ? 1 : 8) < rows; r0 += gridDim.x) {
    const int64_t row = ONE ? r0 : r0 * 8 + grp;
    const int t = (int)(row / a.heads), h = (int)(row - (int64_t)t * a.heads);
    const bool live = row < rows && t >= first && t < last;
    if (ONE && !live) continue;  // (the whole workgroup)
    const int mine = ONE ? threadIdx.x : l;
    f32x2 e = {kNone, 0.f};
    if (live && mine < a.splits) e = *(const f32x2*)(ml + ((int64_t)mine * rows + row) * 2);
    float m = max32(e.x), f = 0.f, weight;
    if (ONE) {
      if (l == 0) tops[grp] = m;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) m = __builtin_fmaxf(m, tops[k]);
    }
    // a part's share; one without weight has written nothing (-1)
    f = e.y == 0.f ? 0.f : e.y * __builtin_amdgcn_exp2f(e.x - (m == kNone ? 0.f : m));
    weight = sum32(f);
    if (e.y == 0.f) f = -1.f;
    if (ONE) {
      factor[mine] = f;
      if (l == 0) weights[grp] = weight;
      __syncthreads();
      weight = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) weight += weights[k];
    }
    const float inv = weight == 0.f ? 0.f : 1.f / weight;
    f32x4 o[H] = {};
    const float* const part = a.part + row * a.dim;
    const int step = ONE ? 8 : 1;
    if (live) {
      for (int z0 = ONE ? grp : 0; z0 < a.splits; z0 += step * kJoinAtOnce) {
        f32x4 v[kJoinAtOnce][H];
        float g[kJoinAtOnce];
#pragma unroll
        for (int k = 0; k < kJoinAtOnce; ++k) {
          const int z = z0 + k * step;
          if (ONE)
            g[k] = z < a.splits ? factor[z] : -1.f;
          else
            g[k] = __shfl(f, (threadIdx.x & 32) + z, 64);
          if (z >= a.splits) g[k] = -1.f;
#pragma unroll
          for (int i = 0; i < H; ++i) {
            const int d = i * 128 + l * 4;
            v[k][i] = f32x4{};
            if (d < a.dim && !(g[k] < 0.f)) v[k][i] = *(const f32x4*)(part + (int64_t)z * rows * a.dim + d);
          }
        }
#pragma unroll
        for (int k = 0; k < kJoinAtOnce; ++k)
#pragma unroll
          for (int i = 0; i < H; ++i)
            if (!(g[k] < 0.f)) o[i] += g[k] * inv * v[k][i];
      }
    }
    if (ONE) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const int d = i * 128 + l * 4;
        if (d < a.dim) *(f32x4*)&red[grp][d] = o[i];
      }
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const int d = i * 128 + l * 4;
          if (d < a.dim)
            for (int k = 1; k < 8; ++k) o[i] += *(const f32x4*)&red[k][d];
        }
      }
    }
    if (live && (!ONE || grp == 0)) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const int d = i * 128 + l * 4;
        if (d >= a.dim) continue;
        const f32x4 v = o[i];
        const int64_t at = (int64_t)t * a.ldy + h * a.dim + d;
        if (a.y_bf16)
          *(u32x2*)((uint16_t*)a.y + at) = u32x2{pack(v.x, v.y), pack(v.z, v.w)};
        else
          *(f32x4*)((float*)a.y + at) = v;
      }
      if (a.lse && l == 0) a.lse[row] = weight == 0.f ? kNone : (m + __builtin_log2f(weight)) * kLn2;
    }
    if (ONE) __syncthreads();
  }
}

template <bool ONE, int H>
void join(const AttendArgs& a, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((attend_join_kernel<ONE, H>), grid, dim3(256), 0, s, a);
}

// The plan for sequences of so many blocks of 32 keys.
//
// Few rows a sequence, up to 32, take the kernel that streams keys past them.  So do more
// of them where the whole call is up to 256 workgroups of 32 rows and the keys are short:
// eight waves divide a workgroup's keys there, which takes less time from the first key to
// the last than 128 rows that walk them all (one sequence of 24 tokens, 32 heads of 128 on 8:
// 200 keys 16.6 -> 12.4 us, 600 19.2 -> 13.1; 61 tokens, 6000 keys 29.7 -> 28.4; four of 61
// over 2000 29.9 -> 27.1; but 30000 keys 39 -> 73, and 24 keys 10.8 -> 11.3).  The bounds are not
// the best everywhere: 240 tokens over 5000 keys, 240 workgroups, lose (43 -> 56), and heads of
// 256 would gain past theirs (24 tokens over 2000 keys 43 -> 33).
//
// Parts of the keys: enough workgroups to fill the chip, two a unit of the kernel for many
// rows and one of the other, of at least so many keys that joining them is worth it.  Few rows
// over up to 48 blocks stay in one part: the join's launch costs more than it gives one sequence
// (700 keys 11.0 us, in parts 14.0; 1500 keys 12.2 and 13.7; but eight of 1500 19.7 and 16.7).
// Parts go by the call's sizes alone: where 256 workgroups are reached without them, one long
// context among short ones is walked by one workgroup a key head (63 sequences of 500 keys and
// one of 131072: 1110 us), and a last round of few workgroups costs a whole one (32 sequences of
// 8192 keys 161 us, 40 of them 238, 64 315).
AttendPlan plan_for(int64_t tokens, int64_t seqs, int64_t group, int64_t kv_heads, int64_t dim, int64_t max_tokens,
                    int64_t blocks) {
  AttendPlan p;
  const int64_t rows = max_tokens * group;
  p.rows = (int32_t)rows;
  int64_t tiles = seqs * ((rows + 31) / 32);
  const bool short_keys = blocks >= 4 && blocks <= (dim > 128 ? 48 : 192);
  p.wide = rows > 32 && !(short_keys && tiles * kv_heads <= 256);
  if (p.wide) {
    const int64_t most = tokens * group / kAttendRows + seqs;
    tiles = seqs * ((rows + kAttendRows - 1) / kAttendRows);
    if (tiles > most) tiles = most;
  }
  const int64_t groups = tiles * kv_heads, want = p.wide ? 512 : 256, least = p.wide ? 16 : 8, whole = p.wide ? 4 : 8;
  int64_t splits = (want + groups - 1) / groups;
  const int64_t most = blocks / least > 1 ? blocks / least : 1;
  if (splits > most) splits = most;
  if (!p.wide && blocks <= 48) splits = 1;
  if (splits > 256) splits = 256;
  int64_t chunk = (blocks + splits - 1) / splits;
  chunk = (chunk + whole - 1) / whole * whole;
  p.chunk = (int32_t)chunk;
  p.splits = (int32_t)((blocks + chunk - 1) / chunk);
  p.bytes = p.splits > 1 ? size_t(p.splits) * size_t(tokens) * kv_heads * group * (dim + 2) * 4 : 0;
  return p;
}

}  // namespace

// A window leaves fewer keys to see, and so fewer parts; the workspace is sized without it.
AttendPlan attend_plan(int64_t tokens, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim, int64_t max_tokens,
                       int64_t max_length, int64_t window) {
  const int64_t blocks = (max_length + 31) / 32, seen = (window + max_tokens + 31) / 32 + 1;
  const AttendPlan all = plan_for(tokens, seqs, heads / kv_heads, kv_heads, dim, max_tokens, blocks);
  if (window <= 0 || seen >= blocks) return all;
  AttendPlan p = plan_for(tokens, seqs, heads / kv_heads, kv_heads, dim, max_tokens, seen);
  if (p.splits > all.splits) p.splits = all.splits;
  p.bytes = all.bytes;
  return p;
}

hipError_t launch_attend(const AttendArgs& args, const AttendPlan& p, hipStream_t s) {
  AttendArgs a = args;
  a.rows = p.rows;
  a.splits = p.splits;
  a.chunk = p.chunk;
  const hipError_t e = p.wide ? launch_attend_many(a, s) : launch_attend_few(a, s);
  if (e != hipSuccess || a.splits == 1) return e;
  const bool one = a.splits > 8;
  const int64_t rows = (int64_t)a.tokens * a.heads, groups = one ? rows : (rows + 7) / 8;
  const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
  if (a.dim > 128)
    one ? join<true, 2>(a, grid, s) : join<false, 2>(a, grid, s);
  else
    one ? join<true, 1>(a, grid, s) : join<false, 1>(a, grid, s);
  return hipGetLastError();
}

}  // namespace uw
