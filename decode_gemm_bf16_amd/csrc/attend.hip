// The sums of split keys, joined; and the rule that splits them.
#include "attend_core.h"

namespace uw {
namespace {

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

}  // namespace

// Parts of the keys: enough workgroups to fill the chip, of at least so many keys.
AttendPlan attend_plan(int64_t tokens, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim, int64_t max_tokens,
                       int64_t max_length) {
  AttendPlan p;
  const int64_t group = heads / kv_heads, per = kAttendRows;
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
  const hipError_t e = p.wide ? launch_attend_many(a, s) : launch_attend_few(a, s);
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
