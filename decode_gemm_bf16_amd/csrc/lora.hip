// Low-rank adapters of many requests beside a projection that they share:
//   y[t] = base[t] + scale_i * B_i (A_i x[t])   for the token's adapter i,
// and y[t] = base[t] where it has none.  A_i is [rank, cols], B_i [rows, rank].
//
// Two kernels per call, both walking the plan's tiles (up to 64 tokens of one
// adapter, in the plan's order):
//   shrink: v = A_i x, [tokens, rank] in float32, split along cols over
//           workgroups when tiles are few (their partial sums lie apart and
//           are added by the second kernel, in order);
//   expand: y = base + (scale_i v) B_i^T.  Both products run on the bf16
//           matrix cores.  v is float32 there too: scale_i v is cut into three
//           bf16 parts (8 + 8 + 8 bits of the 24), whose products with the
//           bf16 B are exact in float32, so that nothing is rounded to bf16.
// What bounds it: few tokens, the adapters' bytes; many, base and y (8 bytes
// an output element against 2 * rank bf16 operations).
#include "recon.h"
#include "routing.h"

namespace uw {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kSub = kPlanTile / 16;  // 16-token subtiles of a tile
constexpr int kRankBlock = 64;        // ranks per shrink workgroup

// ---- shrink ----
//
// One workgroup: one tile, up to 64 ranks, one of ksplit parts of cols.  Its 4
// waves take every fourth 32-column step; each holds all 16 x 16 blocks of
// the tile (4 x 4), so that a step's loads (16 bytes a lane) feed 16 matrix
// instructions.  The waves' sums are added in LDS.
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs a) {
  __shared__ float red[4][16][kRankBlock + 1];
  const LoraProj& p = a.proj[blockIdx.z % a.nproj];
  const int rblock = blockIdx.z / a.nproj;
  if (a.header->tokens != a.tokens || a.header->slots != a.slots || (int)blockIdx.x >= a.header->tiles) return;
  const PlanTile tile = a.tiles[blockIdx.x];
  if (tile.slot < 0) return;
  const int rank = p.table[tile.slot].rank - rblock * kRankBlock;
  if (rank <= 0) return;
  const int nr = rank >= kRankBlock ? kRankBlock / 16 : (rank + 15) / 16;
  const int ns = (tile.len + 15) / 16;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int steps = a.cols / 32, per = (steps + a.ksplit - 1) / a.ksplit;
  const int s0 = blockIdx.y * per, s1 = s0 + per < steps ? s0 + per : steps;
  const uint16_t* ar = p.a + ((int64_t)tile.slot * p.rank16 + rblock * kRankBlock + r) * a.cols + q * 8;
  const uint16_t* xr[kSub];
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    const int k = i * 16 + r;  // rows past the tile's end read its first row; they are not stored
    xr[i] = a.x + (int64_t)a.order[tile.start + (k < tile.len ? k : 0)] * a.ldx + q * 8;
  }
  f32x4 acc[kSub][4] = {};
  for (int s = s0 + w; s < s1; s += 4) {
    bf16x8 xv[kSub], av[4];
#pragma unroll
    for (int i = 0; i < kSub; ++i)
      if (i < ns) xv[i] = *(const bf16x8*)(xr[i] + s * 32);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < nr) av[j] = *(const bf16x8*)(ar + (int64_t)j * 16 * a.cols + s * 32);
#pragma unroll
    for (int i = 0; i < kSub; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i < ns && j < nr) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[i], av[j], acc[i][j], 0, 0, 0);
  }
  // block (i, j): token 4 q + k of subtile i, rank 16 j + r
  float* out = p.part + ((int64_t)blockIdx.y * a.tokens + tile.start) * p.rank16 + rblock * kRankBlock;
  const int ranks = nr * 16;
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    if (i >= ns) break;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) red[w][4 * q + k][16 * j + r] = acc[i][j][k];
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * ranks; e += 256) {
      const int tk = e / ranks, rk = e - tk * ranks;
      if (i * 16 + tk < tile.len)
        out[(int64_t)(i * 16 + tk) * p.rank16 + rk] =
            (red[0][tk][rk] + red[1][tk][rk]) + (red[2][tk][rk] + red[3][tk][rk]);
    }
  }
}

// ---- expand ----

// The leading 8 bits of v as bf16, which are taken off it.  An infinity or NaN
// is one part, and zero remains.
__device__ __forceinline__ uint16_t bf16_part(float& v) {
  uint32_t u = __float_as_uint(v);
  const bool special = (u & 0x7F800000u) == 0x7F800000u;
  if (special && (u & 0x007FFFFFu)) u |= 0x00400000u;  // a NaN stays one without its low bits
  u &= 0xFFFF0000u;
  v = special ? 0.f : v - __uint_as_float(u);
  return (uint16_t)(u >> 16);
}

// One workgroup: one tile, 256 rows of B, 64 per wave.  B is the A operand (16
// rows x 16 ranks), so that a lane's 4 results are 4 neighbouring columns of
// one token's y.
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a) {
  // scale * v in three bf16 parts: [part][token][rank], one 16-rank block at a time
  __shared__ __attribute__((aligned(16))) uint16_t parts[3][kPlanTile][16 + 4];
  const LoraProj& p = a.proj[blockIdx.z];
  if (a.header->tokens != a.tokens || a.header->slots != a.slots || (int)blockIdx.x >= a.header->tiles) return;
  if ((int)blockIdx.y * 256 >= p.rows) return;
  const PlanTile tile = a.tiles[blockIdx.x];
  const LoraSlot entry = tile.slot >= 0 ? p.table[tile.slot] : LoraSlot{0, 0.f};
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.y * 256 + w * 64;
  const int nr = (entry.rank + 15) / 16, ns = (tile.len + 15) / 16;
  if (nr == 0 && p.base == p.y && p.ldbase == p.ldy) return;  // in place, nothing to add
  f32x4 acc[kSub][4];
  int64_t tok[kSub];
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    const int k = i * 16 + r;
    tok[i] = k < tile.len ? a.order[tile.start + k] : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 16 * j + 4 * q;
      acc[i][j] = p.base && tok[i] >= 0 && n < p.rows ? *(const f32x4*)(p.base + tok[i] * p.ldbase + n)
                                                      : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  const uint16_t* b = p.b + (int64_t)(tile.slot < 0 ? 0 : tile.slot) * p.rank16 * p.rows;
  for (int rb = 0; rb < nr; ++rb) {
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * tile.len; e += 256) {
      const int k = e >> 4, c = e & 15;
      const float* src = p.part + (int64_t)(tile.start + k) * p.rank16 + rb * 16 + c;
      float v = 0.f;
      for (int s = 0; s < a.ksplit; ++s) v += src[(int64_t)s * a.tokens * p.rank16];
      // ranks past the adapter's own: an infinity in x makes NaN of them
      v = rb * 16 + c < entry.rank ? v * entry.scale : 0.f;
      parts[0][k][c] = bf16_part(v);
      parts[1][k][c] = bf16_part(v);
      parts[2][k][c] = bf16_part(v);
    }
    __syncthreads();
    s16x4 bv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 16 * j + r;
      bv[j] = n < p.rows ? *(const s16x4*)(b + ((int64_t)rb * p.rows + n) * 16 + 4 * q) : s16x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      if (i >= ns) break;
#pragma unroll
      for (int h = 2; h >= 0; --h) {  // the smallest part first
        // tokens past the tile's end: stale LDS, in columns of the result that are not stored
        const s16x4 vv = *(const s16x4*)&parts[h][i * 16 + r][4 * q];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(bv[j], vv, acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    if (tok[i] < 0) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 16 * j + 4 * q;
      if (n < p.rows) *(f32x4*)(p.y + tok[i] * p.ldy + n) = acc[i][j];
    }
  }
}

// ---- loading an adapter into a slot ----
__global__ __launch_bounds__(256) void lora_load_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
                                                        int64_t rows, int64_t cols, int rank, float scale,
                                                        uint16_t* __restrict__ a_slot, uint16_t* __restrict__ b_slot,
                                                        LoraSlot* __restrict__ entry) {
  const int64_t ranks = (rank + 15) / 16 * 16, na = ranks * cols, nb = ranks * rows;
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = first; i < na; i += stride) a_slot[i] = i < rank * cols ? a[i] : 0;
  for (int64_t i = first; i < nb; i += stride) {
    const int64_t rb = i / (rows * 16), n = i / 16 % rows, c = rb * 16 + i % 16;
    b_slot[i] = c < rank ? b[n * rank + c] : 0;
  }
  if (first == 0) *entry = LoraSlot{rank, scale};
}

}  // namespace

int64_t lora_tiles_max(int64_t tokens, int32_t slots) {
  const int64_t t = (tokens + kPlanTile - 1) / kPlanTile + slots;  // each label's last tile may be short
  return t < tokens ? t : tokens;
}

int lora_ksplit(int64_t tokens, int32_t slots, int64_t cols, int nproj) {
  const int64_t blocks = lora_tiles_max(tokens, slots) * nproj, steps = cols / 32;
  int64_t k = 512 / blocks, most = steps / 16;  // at least 4 steps a wave
  k = k < most ? k : most;
  return (int)(k < 1 ? 1 : k > 16 ? 16 : k);
}

hipError_t launch_lora_apply(const LoraArgs& a, hipStream_t s) {
  int rank16 = 0, rows = 0;
  for (int i = 0; i < a.nproj; ++i) {
    rank16 = a.proj[i].rank16 > rank16 ? a.proj[i].rank16 : rank16;
    rows = a.proj[i].rows > rows ? a.proj[i].rows : rows;
  }
  const unsigned rblocks = (rank16 + kRankBlock - 1) / kRankBlock;
  hipLaunchKernelGGL(lora_shrink_kernel, dim3(a.tiles_max, a.ksplit, rblocks * a.nproj), dim3(256), 0, s, a);
  hipLaunchKernelGGL(lora_expand_kernel, dim3(a.tiles_max, (rows + 255) / 256, a.nproj), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_lora_load(const uint16_t* a, const uint16_t* b, int64_t rows, int64_t cols, int32_t rank,
                            float scale, uint16_t* a_slot, uint16_t* b_slot, LoraSlot* entry, hipStream_t s) {
  const int64_t n = (rank + 15) / 16 * 16 * (rows > cols ? rows : cols), blocks = n / 1024 + 1;  // rank 0: the entry
  hipLaunchKernelGGL(lora_load_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a, b, rows,
                     cols, (int)rank, scale, a_slot, b_slot, entry);
  return hipGetLastError();
}

}  // namespace uw
