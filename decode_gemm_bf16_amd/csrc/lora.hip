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
#include <type_traits>

#include "recon.h"
#include "routing.h"

namespace uw {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kRankBlock = 64;        // ranks per shrink workgroup and per staging of v
constexpr int kShrinkWaves = 8;
constexpr int kLoraMaxSplit = 8;
// A of at most this size a workgroup of lora_one_kernel reads for itself.  One
// launch against two, gate and up of 14336 x 4096 in a graph: 16 ranks (128 KB)
// 5.5 against 6.9 us at one token and 7.5 against 7.7 at four, 32 ranks (256 KB) 7.1
// against 8.1 and 9.4 against 9.4; above, 16 ranks of 14336 columns (448 KB) 9.6
// against 8.0 and 64 of 4096 (512 KB) 11.9 against 9.6.  (Not captured, the launch
// saved is 2.3 us of host time more.)
constexpr int64_t kLoraOneBytes = 256 << 10;

template <typename Args>
__device__ __forceinline__ bool plan_has(const Args& a, int tile) {
  return a.header->tokens == a.tokens && a.header->slots == a.slots && tile < a.header->tiles;
}

union ShrinkLds {
  u32x4 turn[kShrinkWaves][512];  // a wave's 64 tokens x 64 columns
  float red[kShrinkWaves][16][kRankBlock];
};

// ---- shrink ----
//
// One workgroup: one tile, or 32 tokens of it (`halves`) where there are tiles
// enough to fill the CUs so, up to 64 ranks, one of ksplit parts of cols, whose
// batches of 64 columns its 8 waves take in turn (together 1 KB of each row at a
// time).  A wave holds all NS x NR blocks of 16 tokens x 16 ranks.  A lies in the
// order of the operands (1 KB for 16 ranks x 32 columns).  x goes from memory to
// the wave's part of LDS 128 bytes of a row at a time and is read from there in
// that order: loads of 64 bytes of 16 rows, as the operands have it, waste most
// of a memory page's activation.  The waves' sums are added in LDS.
// A wave waits for a batch's loads before its products and has nothing in flight
// during them, so a CU takes in about 22 GB/s: one batch's bytes per memory latency.
// That bounds it, and the work is spread over all CUs before anything else.  (128
// registers, two of them spilled: 12 bytes of scratch a lane.)
template <int NS, int NR, typename Args>
__device__ __forceinline__ void shrink_tile(const Args& a, const LoraProj& p, const PlanTile& tile, int kpart,
                                            int ksplit, int rblock, int nr, ShrinkLds& lds, float* out, int64_t ldout) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int batches = a.cols / 64, per = (batches + ksplit - 1) / ksplit;
  const int b0 = kpart * per, b1 = b0 + per < batches ? b0 + per : batches;
  // a slot's A is less than 2^32 bytes: one address for the wave, 32-bit offsets
  const uint16_t* const abase = p.a + ((int64_t)tile.slot * p.rank16 + rblock * kRankBlock) * a.cols;
  // Load i: tokens 8 i + lane / 8, 16 bytes of each 128 a lane.  A lane takes the
  // piece (lane ^ token) % 8, so that the pieces that a read of the operands takes
  // at once lie in different banks.
  int tok[2 * NS];
#pragma unroll
  for (int i = 0; i < 2 * NS; ++i) {
    const int k = 8 * i + (lane >> 3);  // rows past the tile's end repeat its last
    tok[i] = a.order[tile.start + (k < tile.len ? k : tile.len - 1)];
  }
  const int piece = ((lane ^ (lane >> 3)) & 7) * 8;
  u32x4* const turn = lds.turn[w];
  f32x4 acc[NS][NR] = {};
  for (int b = b0 + w; b < b1; b += kShrinkWaves) {
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(a.x + ((int64_t)tok[i] * a.ldx + b * 64 + piece)),
          (__attribute__((address_space(3))) void*)(turn + i * 64), 16, 0, 0);
    bf16x8 av[2][NR];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < NR; ++j)  // blocks past the adapter's ranks repeat the first; they are not stored
        av[u][j] = *(const bf16x8*)(abase + (uint32_t)((j < nr ? j : 0) * 16 * a.cols + (b * 2 + u) * 512 + lane * 8));
    __builtin_amdgcn_s_waitcnt(0);  // all of it in flight, then all of it there
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const u32x4 xf = turn[(i * 16 + r) * 8 + ((4 * u + q) ^ (r & 7))];
#pragma unroll
        for (int j = 0; j < NR; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(xf), av[u][j], acc[i][j], 0, 0, 0);
      }
    // the reads have left LDS before the next batch's loads write it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  __syncthreads();  // the waves' parts of LDS become the sums'
  float(&red)[kShrinkWaves][16][kRankBlock] = lds.red;
  // block (i, j): token 4 q + k of subtile i, rank 16 j + r
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    if (i) __syncthreads();
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) red[w][4 * q + k][16 * j + r] = acc[i][j][k];
    __syncthreads();
    const int rk = threadIdx.x % (NR * 16);
    for (int tk = threadIdx.x / (NR * 16); tk < 16 && i * 16 + tk < tile.len; tk += 64 * kShrinkWaves / (NR * 16)) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kShrinkWaves; ++k) v += red[k][tk][rk];
      if (rk < nr * 16) out[(i * 16 + tk) * ldout + rk] = v;
    }
  }
}

template <int N>
__global__ __launch_bounds__(64 * kShrinkWaves, 4) void lora_shrink_kernel(LoraArgsOf<N> a) {
  __shared__ __attribute__((aligned(16))) ShrinkLds lds;
  const LoraProj& p = a.proj[blockIdx.z % a.nproj];
  const int rblock = blockIdx.z / a.nproj, kpart = blockIdx.x;
  const int at = a.halves ? blockIdx.y >> 1 : blockIdx.y, i0 = a.halves ? (blockIdx.y & 1) * 32 : 0;
  if (!plan_has(a, at)) return;
  PlanTile tile = a.tiles[at];
  tile.slot = __builtin_amdgcn_readfirstlane(tile.slot);
  tile.start = __builtin_amdgcn_readfirstlane(tile.start) + i0;
  tile.len = __builtin_amdgcn_readfirstlane(tile.len) - i0;
  if (tile.slot < 0 || tile.len <= 0) return;
  if (a.halves && tile.len > 32) tile.len = 32;
  const int rank = p.table[tile.slot].rank - rblock * kRankBlock;
  if (rank <= 0) return;
  const int nr = __builtin_amdgcn_readfirstlane(rank >= kRankBlock ? kRankBlock / 16 : (rank + 15) / 16);
  float* out = p.part + ((int64_t)kpart * a.tokens + tile.start) * p.rank16 + rblock * kRankBlock;
  auto run = [&](auto ns) {
    constexpr int NS = decltype(ns)::value;
    if (nr == 1)
      shrink_tile<NS, 1>(a, p, tile, kpart, a.ksplit, rblock, nr, lds, out, p.rank16);
    else if (nr == 2)
      shrink_tile<NS, 2>(a, p, tile, kpart, a.ksplit, rblock, nr, lds, out, p.rank16);
    else
      shrink_tile<NS, 4>(a, p, tile, kpart, a.ksplit, rblock, nr, lds, out, p.rank16);
  };
  if (tile.len <= 16)
    run(std::integral_constant<int, 1>());
  else if (tile.len <= 32)
    run(std::integral_constant<int, 2>());
  else
    run(std::integral_constant<int, 4>());
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

// For a B that holds infinities: zero times one is NaN, so that no part of a value
// other than zero may be zero.  A part with none behind it gives a step of its own to
// the next, and an infinity is all three.  The sum stays the same, which is why this
// does no harm to a B without infinities in a slot that has held such a one.  (Done
// only where a slot's entry says so: for all, 64 adapters of one token take 17.2 us
// instead of 16.5.)
__device__ __forceinline__ void fill_parts(uint16_t& h0, uint16_t& h1, uint16_t& h2) {
  auto fill = [](uint16_t& h, uint16_t& next) {
    if ((h & 0x7FFF) == 0 || (next & 0x7FFF) != 0) return;
    const uint32_t u = (uint32_t)h << 16;
    const bool finite = (u & 0x7F800000u) != 0x7F800000u;
    next = finite ? __float_as_uint(__uint_as_float(u) - __uint_as_float(u - 0x10000u)) >> 16 : h;
    if (finite) h -= 1;
  };
  fill(h0, h1);
  fill(h1, h2);
}

// scale * v in three bf16 parts: [part][token][rank]; 8 ranks of padding keep
// the lanes' 8-byte reads of 16 tokens apart in the banks
typedef uint16_t LoraParts[3][kPlanTile][kRankBlock + 8];

// Where the products with A stand: [ksplit][token of the tile][ranks].
struct LoraSource {
  const float* v;
  int64_t ld, next;
  int ksplit;
};

// Thread t: token t / 4, ranks 4 (t % 4) .. + 3 of each 16-rank block.
__device__ __forceinline__ void stage_parts(const LoraSource& from, int len, const LoraSlot& entry, int r0, int blocks,
                                            LoraParts& parts) {
  const int k = threadIdx.x >> 2, c = (threadIdx.x & 3) * 4;
  if (k >= len) return;
  const float* src = from.v + k * from.ld + r0 + c;
  f32x4 v[kRankBlock / 16] = {};
  for (int s = 0; s < from.ksplit; ++s) {
#pragma unroll
    for (int i = 0; i < kRankBlock / 16; ++i)  // blocks past the last repeat it
      v[i] += *(const f32x4*)(src + s * from.next + (i < blocks ? i : blocks - 1) * 16);
  }
#pragma unroll
  for (int i = 0; i < kRankBlock / 16; ++i) {
    if (i >= blocks) break;
    uint16_t h[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // ranks past the adapter's own: an infinity in x makes NaN of them
      float f = r0 + i * 16 + c + j < entry.rank ? v[i][j] * entry.scale : 0.f;
#pragma unroll
      for (int m = 0; m < 3; ++m) h[m][j] = bf16_part(f);
    }
#pragma unroll
    for (int m = 0; m < 3; ++m)
      *(u32x2*)&parts[m][k][i * 16 + c] =
          u32x2{h[m][0] | (uint32_t)h[m][1] << 16, h[m][2] | (uint32_t)h[m][3] << 16};
  }
  if (entry.special)  // what this thread has written, from there: no registers more for the rest
#pragma unroll 1
    for (int at = c; at < blocks * 16; at += (at & 3) == 3 ? 13 : 1)
      fill_parts(parts[0][k][at], parts[1][k][at], parts[2][k][at]);
}

// One workgroup: one tile; each of its 4 waves takes one group of 64 rows of B,
// `reps` times over, and 32 tokens at a time (64 at a time hold 164 registers instead
// of 120, three waves a SIMD instead of four: 777 tokens on 4096 x 14336 18.4
// against 15.7 us, 3999 on 4096 x 4096 33.1 against 29.1, 8192 on 14336 173 against 172;
// 16 at a time 777 tokens of 128 ranks 54 against 37).  v is the A operand (16 tokens x
// 16 ranks) and B the B operand; row 4 r + j of a group is column r of its j-th
// 16-column product, so that a lane's results of the four products are 4
// neighbouring columns of y, and a load or store of 16 bytes a lane covers 256
// bytes of each of 4 tokens.  Row 4 q + k of the A operand is token q + 4 k of 16.
// B lies in the order of the operands: a lane's 4 x 4 values of a group and rank
// block are 32 bytes.
template <bool STREAM, typename Args>
__device__ __forceinline__ void expand_tile(const Args& a, const LoraProj& p, const PlanTile& tile,
                                            const LoraSource& from, int reps, LoraParts& parts) {
  constexpr int NS = 2;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int groups = (p.rows + 63) / 64;
  const uint16_t* b = p.b + (int64_t)(tile.slot < 0 ? 0 : tile.slot) * p.rank16 * groups * 64 + lane * 16;
  const LoraSlot entry = tile.slot >= 0 ? p.table[tile.slot] : LoraSlot{0, 0.f, 0, 0};
  if (entry.rank == 0 && p.base == p.y && p.ldbase == p.ldy) return;  // in place, nothing to add
  const int nr = (entry.rank + 15) / 16;
  for (int rep = 0; rep < reps; ++rep)
    for (int i0 = 0; i0 < tile.len; i0 += 16 * NS) {
      const int g = (blockIdx.x * reps + rep) * 4 + w;
      // columns past the last row of B read the last four: no branch between the loads
      const int n = g * 64 + 4 * r, nc = n < p.rows ? n : p.rows - 4, gc = g < groups ? g : groups - 1;
      int tok[NS][4];
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = i0 + i * 16 + q + 4 * k;  // past the tile's end: its last token, not stored
          tok[i][k] = a.order[tile.start + (t < tile.len ? t : tile.len - 1)];
        }
      u32x4 bv[2];
      auto load_b = [&](int rb) {
        const u32x4* src = (const u32x4*)(b + ((int64_t)rb * groups + gc) * 1024);
        bv[0] = src[0];
        bv[1] = src[1];
      };
      if (nr > 0) load_b(0);
      f32x4 acc[NS][4] = {};
      if (p.base) {
        f32x4 v[NS][4];
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[i][k] = __builtin_nontemporal_load((const f32x4*)(p.base + (int64_t)tok[i][k] * p.ldbase + nc));
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j][k] = v[i][k][j];
      }
      for (int r0 = 0; r0 < nr; r0 += kRankBlock / 16) {
        const int blocks = nr - r0 < kRankBlock / 16 ? nr - r0 : kRankBlock / 16;
        if ((rep == 0 && i0 == 0) || nr > kRankBlock / 16) {  // else the parts of all ranks are there
          if (rep || i0 || r0) __syncthreads();
          stage_parts(from, tile.len, entry, r0 * 16, blocks, parts);
          __syncthreads();
        }
        for (int rb = 0; rb < blocks; ++rb) {
          s16x4 now[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            now[j] = __builtin_bit_cast(s16x4, u32x2{bv[j >> 1][(j & 1) * 2], bv[j >> 1][(j & 1) * 2 + 1]});
          if (r0 + rb + 1 < nr) load_b(r0 + rb + 1);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
#pragma unroll
            for (int h = 2; h >= 0; --h) {  // the smallest part first
              // tokens past the tile's end: stale LDS, in rows of the result that are not stored
              const s16x4 vv = *(const s16x4*)&parts[h][i0 + i * 16 + (r >> 2) + 4 * (r & 3)][rb * 16 + 4 * q];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(vv, now[j], acc[i][j], 0, 0, 0);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i0 + i * 16 + q + 4 * k < tile.len && n < p.rows) {
            const f32x4 v = {acc[i][0][k], acc[i][1][k], acc[i][2][k], acc[i][3][k]};
            f32x4* to = (f32x4*)(p.y + (int64_t)tok[i][k] * p.ldy + n);
            if constexpr (STREAM)
              __builtin_nontemporal_store(v, to);
            else
              *to = v;
          }
    }
}

// The same for a tile of at most 4 tokens, whose token t is row 4 t of the A
// operand, by WAVES waves with C groups (WAVES apart) at once.  Each wave cuts v
// into its parts by itself, in the registers of that operand, and waits for no
// other: 64 adapters of one token, gate and up of 14336 rows, 16.3 us against 17.8
// with the parts in LDS.  (Of 4 groups a wave, 2 at once: 4 at once take 27.6 us,
// one after the other 19.5.)
template <int C, bool STREAM, int WAVES, typename Args>
__device__ __forceinline__ void expand_few(const Args& a, const LoraProj& p, const PlanTile& tile,
                                           const LoraSource& from, int reps) {
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int groups = (p.rows + 63) / 64;
  const uint16_t* b = p.b + (int64_t)(tile.slot < 0 ? 0 : tile.slot) * p.rank16 * groups * 64 + lane * 16;
  const LoraSlot entry = tile.slot >= 0 ? p.table[tile.slot] : LoraSlot{0, 0.f, 0, 0};
  if (entry.rank == 0 && p.base == p.y && p.ldbase == p.ldy) return;  // in place, nothing to add
  const int nr = (entry.rank + 15) / 16;
  // results: lane (q, r) has columns 4 r .. + 3 of a group for token q (past the tile's end: its last, not stored)
  const int tok = a.order[tile.start + (q < tile.len ? q : tile.len - 1)];
  const int mine = (r & 3) == 0 && (r >> 2) < tile.len ? r >> 2 : -1;  // the operand's token
  const float* v0 = from.v + (mine < 0 ? 0 : mine) * from.ld + 4 * q;
  for (int rep = 0; rep < reps; ++rep) {
    const int g0 = (blockIdx.x * reps + rep) * WAVES * C + w;
    u32x4 bv[C][2];
    f32x4 v;
    auto load = [&](int rb) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int g = g0 + WAVES * c < groups ? g0 + WAVES * c : groups - 1;
        const u32x4* src = (const u32x4*)(b + ((int64_t)rb * groups + g) * 1024);
        bv[c][0] = src[0];
        bv[c][1] = src[1];
      }
      v = *(const f32x4*)(v0 + rb * 16);
      for (int s = 1; s < from.ksplit; ++s) v += *(const f32x4*)(v0 + rb * 16 + s * from.next);
    };
    f32x4 acc[C][4] = {};
    if (p.base) {
      // columns past the last row of B read the last four: no branch between the loads
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int n = (g0 + WAVES * c) * 64 + 4 * r, nc = n < p.rows ? n : p.rows - 4;
        const f32x4 y = __builtin_nontemporal_load((const f32x4*)(p.base + (int64_t)tok * p.ldbase + nc));
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[c][j][0] = y[j];
      }
    }
    if (nr > 0) load(0);
    for (int rb = 0; rb < nr; ++rb) {
      uint16_t h[3][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // ranks past the adapter's own: an infinity in x makes NaN of them
        float f = mine >= 0 && rb * 16 + 4 * q + j < entry.rank ? v[j] * entry.scale : 0.f;
#pragma unroll
        for (int m = 0; m < 3; ++m) h[m][j] = bf16_part(f);
      }
      s16x4 now[C][4];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          now[c][j] = __builtin_bit_cast(s16x4, u32x2{bv[c][j >> 1][(j & 1) * 2], bv[c][j >> 1][(j & 1) * 2 + 1]});
      if (rb + 1 < nr) load(rb + 1);
      if (__builtin_expect(entry.special != 0, 0)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) fill_parts(h[0][j], h[1][j], h[2][j]);
      }
#pragma unroll
      for (int m = 2; m >= 0; --m) {  // the smallest part first
        const s16x4 vv = __builtin_bit_cast(s16x4, u32x2{h[m][0] | (uint32_t)h[m][1] << 16, h[m][2] | (uint32_t)h[m][3] << 16});
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[c][j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(vv, now[c][j], acc[c][j], 0, 0, 0);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int n = (g0 + WAVES * c) * 64 + 4 * r;
      if (q < tile.len && n < p.rows) {
        const f32x4 y = {acc[c][0][0], acc[c][1][0], acc[c][2][0], acc[c][3][0]};
        f32x4* to = (f32x4*)(p.y + (int64_t)tok * p.ldy + n);
        if constexpr (STREAM)
          __builtin_nontemporal_store(y, to);
        else
          *to = y;
      }
    }
  }
}

// C: groups of 64 rows per wave; two at once where the tile has at most 4
// tokens.  STREAM: y passes the caches by.
template <int N, int C, bool STREAM>
__global__ __launch_bounds__(256, 4) void lora_expand_kernel(LoraArgsOf<N> a) {
  __shared__ __attribute__((aligned(16))) LoraParts parts;
  const LoraProj& p = a.proj[blockIdx.z];
  if (!plan_has(a, blockIdx.y)) return;
  if ((int)blockIdx.x * 256 * C >= p.rows) return;
  const PlanTile tile = a.tiles[blockIdx.y];
  constexpr int kFew = C > 2 ? 2 : C;
  const LoraSource from{p.part + (int64_t)tile.start * p.rank16, p.rank16, (int64_t)a.tokens * p.rank16, a.ksplit};
  if (tile.len <= 4)
    expand_few<kFew, STREAM, 4>(a, p, tile, from, C / kFew);
  else
    expand_tile<STREAM>(a, p, tile, from, C, parts);
}

// ---- both in one launch, for at most four tokens ----
//
// Each workgroup takes 512 rows of B and makes the products with A for itself:
// A is read rows / 512 times over, from L2 but for the first, and a launch is
// saved.
template <int N>
__global__ __launch_bounds__(64 * kShrinkWaves, 4) void lora_one_kernel(LoraArgsOf<N> a) {
  __shared__ __attribute__((aligned(16))) ShrinkLds lds;
  __shared__ __attribute__((aligned(16))) float v[4][kRankBlock];
  const LoraProj& p = a.proj[blockIdx.z];
  if (!plan_has(a, blockIdx.y)) return;
  if ((int)blockIdx.x * 512 >= p.rows) return;
  PlanTile tile = a.tiles[blockIdx.y];
  tile.slot = __builtin_amdgcn_readfirstlane(tile.slot);
  tile.start = __builtin_amdgcn_readfirstlane(tile.start);
  tile.len = __builtin_amdgcn_readfirstlane(tile.len);
  const int nr = tile.slot < 0 ? 0 : __builtin_amdgcn_readfirstlane((p.table[tile.slot].rank + 15) / 16);
  if (nr == 1)
    shrink_tile<1, 1>(a, p, tile, 0, 1, 0, nr, lds, v[0], kRankBlock);
  else if (nr == 2)
    shrink_tile<1, 2>(a, p, tile, 0, 1, 0, nr, lds, v[0], kRankBlock);
  else if (nr > 2)
    shrink_tile<1, 4>(a, p, tile, 0, 1, 0, nr, lds, v[0], kRankBlock);
  __syncthreads();
  expand_few<1, false, kShrinkWaves>(a, p, tile, LoraSource{v[0], kRankBlock, 0, 1}, 1);
}

template <int N, int C>
void launch_expand(const LoraArgsOf<N>& a, int rows, hipStream_t s) {
  const dim3 grid((rows + 256 * C - 1) / (256 * C), a.tiles_max, a.nproj);
  if (a.stream)
    hipLaunchKernelGGL((lora_expand_kernel<N, C, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((lora_expand_kernel<N, C, false>), grid, dim3(256), 0, s, a);
}

template <int N>
hipError_t launch_apply(const LoraArgs& all, hipStream_t s) {
  LoraArgsOf<N> a;
  int rank16 = 0, rows = 0;
  for (int i = 0; i < N; ++i) {
    a.proj[i] = all.proj[i];
    rank16 = a.proj[i].rank16 > rank16 ? a.proj[i].rank16 : rank16;  // (those past nproj are zeros)
    rows = a.proj[i].rows > rows ? a.proj[i].rows : rows;
  }
  a.header = all.header;
  a.tiles = all.tiles;
  a.order = all.order;
  a.x = all.x;
  a.ldx = all.ldx;
  a.tokens = all.tokens;
  a.slots = all.slots;
  a.cols = all.cols;
  a.nproj = all.nproj;
  a.ksplit = all.ksplit;
  a.tiles_max = all.tiles_max;
  a.halves = all.halves;
  a.stream = all.stream;
  if (a.tokens <= 4 && rank16 <= kRankBlock && (int64_t)rank16 * a.cols * 2 <= kLoraOneBytes) {
    hipLaunchKernelGGL(lora_one_kernel<N>, dim3((rows + 511) / 512, a.tiles_max, a.nproj), dim3(64 * kShrinkWaves), 0,
                       s, a);
    return hipGetLastError();
  }
  const unsigned rblocks = (rank16 + kRankBlock - 1) / kRankBlock;
  hipLaunchKernelGGL(lora_shrink_kernel<N>, dim3(a.ksplit, a.halves ? 2 * a.tiles_max : a.tiles_max, rblocks * a.nproj),
                     dim3(64 * kShrinkWaves), 0, s, a);
  // Few tokens a slot: mostly tiles of a token or a few, whose workgroups take 1024
  // columns, if there are workgroups enough (gate and up of 14336 rows: 64 adapters of
  // one token 16.3 us against 24.9 with 256, of four in a run 20.9 against 27.5, of
  // four on average 27.8 against 29.2).  The number of slots stands in for the number
  // of adapters in the batch, which is known on the device only: 256 tokens of one
  // adapter in 256 slots take 30.6 against 16.0.
  if (a.tokens <= 4 * a.slots && (int64_t)a.tiles_max * rows * a.nproj >= 256 * 2048)
    launch_expand<N, 4>(a, rows, s);
  else
    launch_expand<N, 1>(a, rows, s);
  return hipGetLastError();
}

// ---- loading an adapter into a slot ----
__global__ __launch_bounds__(256) void lora_load_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
                                                        int64_t rows, int64_t cols, int rank, float scale,
                                                        uint16_t* __restrict__ a_slot, uint16_t* __restrict__ b_slot,
                                                        LoraSlot* __restrict__ entry) {
  const int64_t rows64 = (rows + 63) / 64 * 64, ranks = (rank + 15) / 16 * 16, na = ranks * cols, nb = ranks * rows64;
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = first; i < na; i += stride) {
    // [rank / 16][col / 32][q][r][8]: rank r of a block, columns 8 q .. + 7 of a step
    const int64_t rb = i / (cols * 16), m = i % 512;
    const int64_t c = rb * 16 + m / 8 % 16, k = i / 512 % (cols / 32) * 32 + m / 128 * 8 + m % 8;
    a_slot[i] = c < rank ? a[c * cols + k] : 0;
  }
  for (int64_t i = first; i < nb; i += stride) {
    // [rank / 16][row / 64][q][r][j][4]: row 4 r + j of a group, ranks 4 q .. + 3 of a block
    const int64_t rb = i / (rows64 * 16), g = i / 1024 % (rows64 / 64), m = i % 1024;
    const int64_t n = g * 64 + m / 16 % 16 * 4 + m / 4 % 4, c = rb * 16 + m / 256 * 4 + m % 4;
    const uint16_t v = c < rank && n < rows ? b[n * rank + c] : 0;
    b_slot[i] = v;
    if ((v & 0x7F80) == 0x7F80) entry->special = 1;
  }
  if (first == 0) {
    entry->rank = rank;
    entry->scale = scale;
    // Emptying a slot takes it back.  A load does not, as that would have to come before
    // what the other workgroups do; with it a finite B gives the same sums up to their roundings.
    if (rank == 0) entry->special = 0;
  }
}

}  // namespace

int64_t lora_tiles_max(int64_t tokens, int32_t slots) {
  const int64_t t = (tokens + kPlanTile - 1) / kPlanTile + slots;  // each label's last tile may be short
  return t < tokens ? t : tokens;
}

// These rules see how many tiles a batch of this size can have at most, with every
// slot of the handle in use, and not how many it has: the host does not know the plan.
// A batch of few adapters in a handle of many slots runs with fewer workgroups than
// would suit it (plan and call, 512 tokens of one adapter of 16 ranks on 4096 x
// 14336: 23.5 us in 4 slots, 44 in 128 or 512).

// Whether the shrink takes 32 tokens a workgroup: 136 tiles of 4096 columns 20 +
// 172 us (shrink and expansion) against 19 + 175 with whole tiles in two parts.
bool lora_halves(int64_t tokens, int32_t slots, int nproj) { return lora_tiles_max(tokens, slots) * nproj >= 128; }

// Parts of cols: up to two workgroups a CU, and two batches for each wave.  (More
// parts cost the expansion, which reads all of them for every 256 columns of y:
// 777 tokens on 4096 x 14336 in 4 parts 19.0 + 14.5 us, in 8 15.3 + 15.7.)
int lora_ksplit(int64_t tokens, int32_t slots, int64_t cols, int nproj) {
  const int64_t tiles = lora_tiles_max(tokens, slots) * nproj, batches = cols / 64;
  const int64_t blocks = lora_halves(tokens, slots, nproj) ? 2 * tiles : tiles;
  int k = kLoraMaxSplit;
  while (k > 1 && (k * blocks > 512 || batches < 2 * k * kShrinkWaves)) k /= 2;
  return k;
}

hipError_t launch_lora_apply(const LoraArgs& a, hipStream_t s) {
  return a.nproj == 1 ? launch_apply<1>(a, s) : a.nproj == 2 ? launch_apply<2>(a, s) : launch_apply<kLoraMaxProj>(a, s);
}

hipError_t launch_lora_load(const uint16_t* a, const uint16_t* b, int64_t rows, int64_t cols, int32_t rank,
                            float scale, uint16_t* a_slot, uint16_t* b_slot, LoraSlot* entry, hipStream_t s) {
  const int64_t n = (rank + 15) / 16 * 16 * (rows > cols ? rows : cols), blocks = n / 1024 + 1;  // rank 0: the entry
  hipLaunchKernelGGL(lora_load_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a, b, rows,
                     cols, (int)rank, scale, a_slot, b_slot, entry);
  return hipGetLastError();
}

}  // namespace uw
