// Attention with many rows a sequence: prompts, chunks of them, trees of drafted tokens.
#include "attend_core.h"

namespace uw {
namespace {

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

constexpr int kManyRows = 32 * kWaves;
static_assert(kManyRows == kAttendRows, "the rule on sizes counts them");

typedef __attribute__((address_space(3))) uint8_t* lds_ptr;
typedef const __attribute__((address_space(3))) uint8_t* lds_cptr;
__device__ __forceinline__ bf16x8 lds16(lds_cptr p) { return *(const __attribute__((address_space(3))) bf16x8*)p; }

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the wave's last N vector loads have arrived
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Product i of a unit of work: the first kLead are of the values, while the softmax finds
// its maximum, then two of the keys and one of the values in turn.
template <int D>
struct UnitOrder {
  static constexpr int kAll = D / 8, kLead = kAll / 4;
  static constexpr int kAhead = D == 256 ? 8 : 4;  // operands are read so many products before theirs
  static_assert(kAll % 4 == 0 && kAll % kAhead == 0, "a quarter of the products leads; whole rounds of operands");
  static __device__ constexpr bool of_value(int i) { return i < kLead || (i - kLead) % 3 == 2; }
  static __device__ constexpr int number(int i) {
    return i < kLead ? i : (i - kLead) % 3 == 2 ? kLead + (i - kLead) / 3 : (i - kLead) / 3 * 2 + (i - kLead) % 3;
  }
};

// One unit of work of a wave.  S: products of kt's keys to xn.  W: x, the products of
// block kb, become weights.  P: the weights p times vt's values; p then holds the new
// ones.  FIRST: no operand is read yet.  NEXT: the next unit's are there, (kn, vn).
// EDGES: block kb may hold keys that rows do not see.
template <int D, int MODE, bool EDGES>
struct Unit {
  using Order = UnitOrder<D>;
  const AttendArgs& a;
  const Row& r;
  const Range& g;
  const bf16x8 (&q)[D / 16];
  const float sc;
  const int half, key_lane, value_lane;
  bf16x8 (&ring)[Order::kAhead];
  Sums<D>& c;

  __device__ __forceinline__ bf16x8 operand(int i, lds_cptr kt, lds_cptr vt) const {
    const int n = Order::number(i);
    return Order::of_value(i) ? lds16(vt + n / (D / 32) * 32 * D + n % (D / 32) * 512 + value_lane)
                              : lds16(kt + n * 1024 + key_lane);
  }
  template <bool S, bool P>
  static __device__ __forceinline__ bool there(int i) {
    return Order::of_value(i) ? P : S;
  }

  template <bool S, bool W, bool P, bool FIRST, bool NEXT>
  __device__ __forceinline__ void run(lds_cptr kt, lds_cptr vt, lds_cptr kn, lds_cptr vn, int kb, f32x16& x, f32x16& xn,
                                      bf16x8 (&p)[2]) const {
    constexpr int kAll = Order::kAll, kLead = Order::kLead, kAhead = Order::kAhead;
    if (FIRST) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (there<S, P>(i)) ring[i] = operand(i, kt, vt);
    }
    const Cap cap(a);
    FarCap far(a);
    if (W && (MODE & kFar) && far.passed<16>(x)) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = far.any(cap, x[e]);
      far.pass();
    }
    const float base = MODE & kSlopes ? -r.slope * (float)(r.pos - kb - 4 * half) : 0.f;
    float top = kNone, m = 0.f;
    bool moved = false;
    float f = 1.f;
    uint32_t wt[8];
    float last = 0.f;
    if (S) xn = f32x16{};
    if (W && EDGES && (kb < g.lo_all || kb + 32 > g.hi_all)) {
      const int lower = r.lower - kb - 4 * half, upper = r.upper - kb - 4 * half;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (key_of(e) < lower || key_of(e) >= upper) x[e] = kNone;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kAll; ++i) {
      const int n = Order::number(i);
      if (there<S, P>(i)) {
        if (Order::of_value(i))
          c.o[n % (D / 32)] =
              __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i % kAhead], p[n / (D / 32)], c.o[n % (D / 32)], 0, 0, 0);
        else
          xn = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i % kAhead], q[n], xn, 0, 0, 0);
      }
      const int j = i + kAhead;
      if (j < kAll) {
        if (there<S, P>(j)) ring[j % kAhead] = operand(j, kt, vt);
      } else if (NEXT) {
        if (there<S, P>(j - kAll)) ring[j % kAhead] = operand(j - kAll, kn, vn);
      }
      if (W) {
        if (i < kLead) {
#pragma unroll
          for (int e = 16 * i / kLead; e < 16 * (i + 1) / kLead; ++e) {
            if (MODE == (kCap | kSlopes)) x[e] = cap(x[e]);
            if (MODE == (kCap | kSlopes | kFar)) x[e] = far(x[e]);
            if (MODE & kSlopes)
              x[e] = __builtin_fmaf(x[e], MODE & kCap ? 1.f : a.scale * kLog2e,
                                    __builtin_fmaf(r.slope, (float)key_of(e), base));
            top = __builtin_fmaxf(top, x[e]);
          }
          if (i == kLead - 1) {
            top = larger_half(top);
            if (MODE == kCap) top = cap(top);
            if (MODE == (kCap | kFar)) top = far(top);
            if (MODE == 0) top *= sc;
            moved = __ballot(top > c.m + kSlack) != 0;
            const float was = c.m;
            if (moved) c.m = __builtin_fmaxf(c.m, top);
            m = c.m == kNone ? 0.f : c.m;
            f = moved ? __builtin_amdgcn_exp2f(was - m) : 1.f;
            c.l *= f;
            asm volatile("" : "+v"(c.l));  // (no fused sum: rows done again by careful() come out the same)
          }
        } else {
          constexpr int kRest = kAll - kLead;
#pragma unroll
          for (int e = 16 * (i - kLead) / kRest; e < 16 * (i - kLead + 1) / kRest; ++e) {
            const float y = MODE == 0 ? __builtin_fmaf(x[e], sc, -m)
                                      : (MODE == kCap ? cap(x[e]) : MODE == (kCap | kFar) ? far(x[e]) : x[e]) - m;
            const float now = __builtin_amdgcn_exp2f(y);
            if (e % 2) {
              c.l += last + now;
              wt[e / 2] = pack(last, now);
              asm volatile("" : "+v"(wt[e / 2]), "+v"(c.l));  // (here, not behind the branch below)
            }
            last = now;
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (W) {
      p[0] = as_bf16x8(wt[0], wt[1], wt[2], wt[3]);
      p[1] = as_bf16x8(wt[4], wt[5], wt[6], wt[7]);
      if (moved) {
#pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          // (the sums of long heads fill the accumulators' half of the registers and stay there)
          if (D > 128) asm volatile("" : "+a"(c.o[t]));
          c.o[t] *= f;
          if (D > 128) asm volatile("" : "+a"(c.o[t]));
        }
      }
    }
  }
};

// 128 rows a workgroup, 32 a wave; keys and values shared in LDS.
//
// Keys and values go from memory to LDS, 64 keys a tile, and stand there as in the
// cache (1 KB a load, and read from there in order); a tile is on its way while the one
// before it is used.  The tiles are LDS objects of their own, and page numbers scalar
// loads, so that the compiler's waits for what is used leave the loads in flight.
//
// Where every row sees every key (EDGES: up to a sequence's last block) a wave works on
// three blocks of 32 keys at once: the products of the keys of block u + 1, the softmax
// of block u, and the products with the values of block u - 1.  The three depend on
// nothing of each other's, and the vector instructions of one hide, with two waves a SIMD,
// behind half of the matrix instructions of the others (8 products of 32x32x16 131 ns, 96
// FMA 110, both 187).  That bounds it: a prompt of 8192 tokens, 32 heads of 128 on 8, 514 to 544
// us from card to card (1.01 to 1.07 PFLOP/s; the library's matrix product reaches 1.2), the
// matrix units at work for 57 % of the cycles, waves waiting for loads, LDS and barriers 22 %
// of theirs; with a cap, whose tanh is five more instructions a score, trees of 61 tokens over
// 6000 keys 0.59 PFLOP/s, without one 0.75.  64 rows a
// wave, which read LDS half as often, leave one wave a SIMD, and that issues vector
// instructions at half the rate (722 us against 613, under a profiler).
//
// Heads of 256 have one wave a SIMD all the same: their sums take half of its registers
// (prompt of 4096 tokens 328 us, 0.84 PFLOP/s).
template <int D, int MODE, bool EDGES>
__global__ __launch_bounds__(64 * kWaves, D > 128 ? 1 : 2) void attend_many_kernel(AttendArgs a) {
  constexpr int kBytes = 64 * D;               // of a block's keys, or values
  constexpr int kSteps = D / 16;               // products of a block's keys, and of its values
  constexpr int kChunks = 2 * kBytes / 1024;   // loads of a tile's keys, or values
  __shared__ __attribute__((aligned(1024))) uint8_t tk0[2 * kBytes], tk1[2 * kBytes], tv0[2 * kBytes], tv1[2 * kBytes];
  __shared__ int range[4][kWaves];
  const lds_ptr k0 = (lds_ptr)tk0, k1 = (lds_ptr)tk1, v0 = (lds_ptr)tv0, v1 = (lds_ptr)tv1;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
  const int kvh = (int)(gridDim.x - 1 - blockIdx.x) % a.kv_heads, z = blockIdx.y;
  int b, rt;
  // the last rows of a sequence see the most keys: they go first
  if (!tile_of(a, kManyRows, (int)(gridDim.x - 1 - blockIdx.x) / a.kv_heads, b, rt)) return;
  const Seq s = sequence(a, b);
  const float sc = MODE ? 1.f : a.scale * kLog2e;
  const Row r = row_of(a, s, kvh, rt * kManyRows + w * 32 + (lane & 31));
  const Range g = range_of(a, s, r);
  if (lane == 0) {
    range[0][w] = g.lo;
    range[1][w] = -g.hi;
    range[2][w] = -g.lo_all;
    range[3][w] = g.hi_all;
  }
  bf16x8 q[kSteps];
  load_query<D>(a, r, half, q);
  Sums<D> c;
  clear(c);
  Odd none{1 << 30, -1};
  __syncthreads();
  auto least = [&](int i) {
    int v = range[i][0];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v = range[i][k] < v ? range[i][k] : v;
    return __builtin_amdgcn_readfirstlane(v);
  };
  // blocks that some row of the workgroup sees, and those that every row sees all of
  const int b0 = least(0) >> 5, b1 = (31 - least(1)) >> 5;
  int f0 = (31 - least(2)) >> 5, f1 = least(3) >> 5;
  if (EDGES && !(a.slopes && a.prefix)) {  // (keys ahead of a row: as far off as those behind it)
    f0 = b0;
    f1 = (a.mask && s.start < s.keys ? s.start : s.keys) >> 5;  // (may be negative)
  }
  const int key_lane = lane * 16, value_lane = (half * D + (lane & 31)) * 16;
  bf16x8 ring[UnitOrder<D>::kAhead];
  const Unit<D, MODE, EDGES> unit{a, r, g, q, sc, half, key_lane, value_lane, ring, c};

  struct Place {
    int64_t at[2];
    uint32_t off;  // bit n: block n has no page in the cache, or lies behind the end
  };
  for (int p0 = b0 + z * a.chunk; p0 < b1; p0 += a.splits * a.chunk) {
    const int p1 = p0 + a.chunk < b1 ? p0 + a.chunk : b1;
    auto locate = [&](int blk) {
      Place p;
      p.off = 0;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const bool ok = block_at(a, s, kvh, blk + n < p1 ? blk + n : p1 - 1, D, p.at[n]) && blk + n < p1;
        p.off |= ok ? 0u : 1u << n;
      }
      return p;
    };
    auto fetch = [&](const uint16_t* cache, const Place& p, lds_ptr tile) {
      const rsrc_t b[2] = {make_rsrc(cache + p.at[0], p.off & 1 ? 0 : kBytes),
                           make_rsrc(cache + p.at[1], p.off & 2 ? 0 : kBytes)};
#pragma unroll
      for (int t = 0; t < kChunks; t += kWaves) {
        const int ch = t + w;
        const int n = ch / (kChunks / 2);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(n ? b[1] : b[0], (__attribute__((address_space(3))) void*)(tile + ch * 1024),
                                                 16, lane * 16, (ch - n * (kChunks / 2)) * 1024, 0, 0);
      }
    };
    // All that was fetched is there, every wave's part, and every wave has left the tiles
    // that are fetched next.
    auto arrive = [&]() {
      wait_loads<0>();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    int blk = p0, buf = 0;
    Place here = locate(p0), next = locate(p0 + 2);
    fetch(a.kc, here, k0);
    fetch(a.vc, here, v0);
    while (blk < p1) {
      Place third = locate(blk + 4);
      // three whole tiles at least: an odd number of them goes through the stages
      if (buf == 0 && blk >= f0 && blk + 6 <= f1 && (here.off | next.off | third.off) == 0) {
        arrive();
        fetch(a.kc, next, k1);
        f32x16 xa = {}, xb;
#pragma unroll
        for (int t = 0; t < kSteps; ++t)
          xa = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lds16(k0 + t * 1024 + key_lane), q[t], xa, 0, 0, 0);
        bf16x8 p[2] = {};
        unit.template run<true, true, false, true, false>(k0 + kBytes, v0, k0, v0, blk << 5, xa, xb, p);
        do {
          // (keys of the tile after blk's are there or on their way, its values not; third
          // is the tile after that)
          arrive();
          fetch(a.vc, next, v1);
          fetch(a.kc, third, k0);
          next = third;
          third = locate(blk + 6);
          unit.template run<true, true, true, true, true>(k1, v0, k1 + kBytes, v0 + kBytes, (blk + 1) << 5, xb, xa, p);
          unit.template run<true, true, true, false, false>(k1 + kBytes, v0 + kBytes, k0, v0, (blk + 2) << 5, xa, xb, p);
          blk += 2;
          arrive();
          fetch(a.vc, next, v0);
          fetch(a.kc, third, k1);
          next = third;
          third = locate(blk + 6);
          unit.template run<true, true, true, true, true>(k0, v1, k0 + kBytes, v1 + kBytes, (blk + 1) << 5, xb, xa, p);
          unit.template run<true, true, true, false, false>(k0 + kBytes, v1 + kBytes, k0, v0, (blk + 2) << 5, xa, xb, p);
          blk += 2;
        } while (blk + 6 <= f1 && (next.off | third.off) == 0);
        arrive();
        fetch(a.vc, next, v1);
        unit.template run<false, true, true, true, false>(k0, v0, k0, v0, (blk + 1) << 5, xb, xa, p);
        unit.template run<false, false, true, true, false>(k0, v0 + kBytes, k0, v0, 0, xb, xa, p);
        blk += 2;
        buf = 1;
        here = next;
        next = third;
      } else {
        arrive();
        const uint32_t off = here.off;
        here = next;
        next = third;
        fetch(a.kc, here, buf ? k0 : k1);
        fetch(a.vc, here, buf ? v0 : v1);
        const lds_cptr kt = buf ? k1 : k0, vt = buf ? v1 : v0;
#pragma unroll 1
        for (int n = 0; n < 2; ++n) {
          const int kb = (blk + n) << 5;
          if (kb >= g.hi || kb + 32 <= g.lo) continue;
          f32x16 x = {};
#pragma unroll
          for (int t = 0; t < kSteps; ++t)
            x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lds16(kt + n * kBytes + t * 1024 + key_lane), q[t], x, 0, 0, 0);
          auto value = [&](int u, int t) { return lds16(vt + n * kBytes + u * 32 * D + t * 512 + value_lane); };
          take<D, MODE, false, false>(a, s, r, g, sc, kb, half, x, off >> n & 1, c, none, value);
        }
        blk += 2;
        buf ^= 1;
      }
    }
    arrive();  // (of tiles behind the end, too: nothing is written to LDS later on)
  }
  float times = 1.f;
  if (not_finite(c.o, 16)) {
    Sums<D> again;
    careful<D, MODE>(kernel_args(), b, kvh, rt * kManyRows + w * 32, b0 + z * a.chunk, a.chunk, a.splits * a.chunk, b1, 0, 1,
                     &again);
    c = again;
    times = kMore;
  }
  put_all(a, r, z, half, c, times);
}

template <int D, int MODE, bool EDGES>
void launch_edges(const AttendArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)a.tokens * a.group / kManyRows + a.seqs;  // at most
  hipLaunchKernelGGL((attend_many_kernel<D, MODE, EDGES>), dim3((unsigned)(tiles * a.kv_heads), (unsigned)a.splits),
                     dim3(64 * kWaves), 0, s, a);
}

// EDGES where many blocks are seen in part: with documents, and with short heads, whose
// 128 rows are 128 tokens of one head as a rule (24 chunks of up to 700 tokens, heads of 64,
// a window: 95 -> 87 us, with slopes 116 -> 111; documents of 300 tokens 87 -> 77, heads of 64
// 59 -> 51; a prompt with heads of 64 pays 328 -> 338).  Elsewhere its branch gives little or
// takes some (chunks of 4 heads of 128 a key head 261 -> 260, with a window 204 -> 200; a prompt of
// 8192 tokens 514 -> 523), and the places of a cap's scores are hidden after it.
template <int D, int MODE>
void launch(const AttendArgs& a, hipStream_t s) {
  if constexpr (MODE & kCap)
    launch_edges<D, MODE, false>(a, s);
  else if constexpr (D < 128)
    launch_edges<D, MODE, true>(a, s);
  else
    a.first ? launch_edges<D, MODE, true>(a, s) : launch_edges<D, MODE, false>(a, s);
}

template <int D>
void launch_mode(const AttendArgs& a, hipStream_t s) {
  with_mode(a, [&](auto mode) { launch<D, mode.value>(a, s); });
}

}  // namespace

hipError_t launch_attend_many(const AttendArgs& a, hipStream_t s) {
  switch (a.dim) {
    case 64: launch_mode<64>(a, s); break;
    case 96: launch_mode<96>(a, s); break;
    case 128: launch_mode<128>(a, s); break;
    default: launch_mode<256>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace uw
