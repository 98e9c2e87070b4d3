// Launchers of the kernels that route rows to experts and back (route.hip,
// rows.hip) and of the low-rank adapters (lora.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace uw {

// ---- routing (route.hip) ----
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxGroups = 64;
constexpr int kRouteMaxTopK = 64;
struct RouteArgs {
  const void* logits;  // [tokens, ld] float32 or bf16
  const float* bias;   // [experts] or null
  int32_t* index;      // [tokens, top_k]
  float* weight;       // [tokens, top_k]
  int64_t ld, tokens;
  int32_t experts, top_k, groups, top_groups;
  bool bf16, sigmoid, pairs, renormalise;
  float scale;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

// ---- grouping of rows, their way out and back (rows.hip) ----
constexpr int kGroupMax = 4000;
// Rows per tile of a plan (lora.hip works a tile at a time).
constexpr int kPlanTile = 64;
struct PlanHeader {
  int32_t tokens, slots, tiles, unused;
};
struct PlanTile {
  int32_t start, len, slot, unused;  // slot: -1 for the rows without an adapter
};
struct GroupArgs {
  const int32_t* index;  // [n]; anything outside 0..groups-1 is ungrouped
  int64_t n;
  int32_t groups;
  int32_t* offsets;  // [groups + 1] or null
  int32_t* order;    // [n]
  int32_t* slot;     // [n] or null
  int32_t* work;     // group_work_bytes
  PlanHeader* header;  // null, or where the tiles' header goes
  PlanTile* tiles;
};
size_t group_work_bytes(int64_t n, int32_t groups);
hipError_t launch_group_rows(const GroupArgs& a, hipStream_t s);
hipError_t launch_dispatch_rows(const uint16_t* x, int64_t ldx, const int32_t* slot, int64_t tokens, int32_t top_k,
                                int64_t cols, uint16_t* xs, int64_t rows, hipStream_t s);
// rows: of xs and ys; a slot outside them has no row.  base may be null or y
// itself; y is float32 or bf16.
hipError_t launch_combine_rows(const float* ys, const int32_t* slot, const float* weight, int64_t tokens,
                               int32_t top_k, int64_t cols, int64_t rows, const float* base, void* y, bool y_bf16,
                               hipStream_t s);

// ---- low-rank adapters (lora.hip) ----
constexpr int kLoraMaxProj = 4;
struct LoraSlot {
  int32_t rank;
  float scale;
  int32_t special;  // not 0: B holds infinities or NaN, or has held some since the slot was last empty
  int32_t unused;
};
// One projection's adapters, both matrices in the order of the matrix
// operands.  Slot i's A is a + i * rank16 * cols, [rank16 / 16][cols / 32][4][16][8]
// bf16 with rank r of a block of 16 and column 8 q + i of a step of 32 at
// [q][r][i].  Its B is b + i * rank16 * rows64 (rows rounded up to 64),
// [rank16 / 16][rows64 / 64][4][16][4][4] bf16 with row 4 r + j of a group of 64
// and rank 4 q + i of a block of 16 at [q][r][j][i].  Ranks past the slot's own
// are zero up to the next multiple of 16.
struct LoraProj {
  const uint16_t* a;
  const uint16_t* b;
  const LoraSlot* table;
  const float* base;  // null: zero
  float* y;
  int64_t ldbase, ldy;
  int32_t rows, rank16;
  float* part;  // [ksplit][tokens][rank16] products with A
};
// N: projections that there is room for (a launch costs about 0.4 us of host time
// more per 100 bytes of arguments).
template <int N>
struct LoraArgsOf {
  LoraProj proj[N];
  const PlanHeader* header;
  const PlanTile* tiles;
  const int32_t* order;
  const uint16_t* x;
  int64_t ldx;
  int32_t tokens, slots, cols, nproj, ksplit, tiles_max;
  bool halves;  // the shrink takes 32 tokens a workgroup
  bool stream;  // y passes the caches by
};
using LoraArgs = LoraArgsOf<kLoraMaxProj>;
// Rules on sizes alone.
bool lora_halves(int64_t tokens, int32_t slots, int nproj);
int lora_ksplit(int64_t tokens, int32_t slots, int64_t cols, int nproj);
int64_t lora_tiles_max(int64_t tokens, int32_t slots);
hipError_t launch_lora_apply(const LoraArgs& a, hipStream_t s);
hipError_t launch_lora_load(const uint16_t* a, const uint16_t* b, int64_t rows, int64_t cols, int32_t rank,
                            float scale, uint16_t* a_slot, uint16_t* b_slot, LoraSlot* entry, hipStream_t s);

}  // namespace uw
