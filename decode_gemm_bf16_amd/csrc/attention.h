// Launchers of the kernels around a paged cache of keys and values: rows written
// to it and moved in it (cache.hip), attention over it (attend.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace uw {

// A cache is two bf16 arrays [pages, kv_heads, page * dim].  Within a page of one
// head, element d of place o stands, for the keys, at
//   ((o / 32 * dim / 8 + d / 8) * 32 + o % 32) * 8 + d % 8
// (a block of 32 keys is what 32x32x16 matrix instructions take as their first
// operand, 16 elements of 32 keys in 1 KB that the lanes read in order), and for
// the values at
//   ((o / 16 * 2 + o / 4 % 2) * dim + d) * 8 + o / 8 % 2 * 4 + o % 4
// (the first operand of the product with the weights, 16 keys a step, in the order
// in which the lanes hold the weights after the first product).
__host__ __device__ inline int64_t key_at(int64_t o, int d, int dim) {
  return ((o / 32 * (dim / 8) + d / 8) * 32 + o % 32) * 8 + d % 8;
}
__host__ __device__ inline int64_t value_at(int64_t o, int d, int dim) {
  return ((o / 16 * 2 + o / 4 % 2) * dim + d) * 8 + o / 8 % 2 * 4 + o % 4;
}

constexpr int kRotaryMaxAxes = 4;
struct CacheWriteArgs {
  const void *q, *k, *v;  // float32 or bf16 rows; q may be null
  int64_t ldq, ldk, ldv, ldqo;
  const int32_t* positions;  // [axes, tokens]
  const float* freqs;        // [pairs]
  const int32_t* axis;       // [pairs] or null
  const int32_t* slots;      // [tokens]
  uint16_t* qo;
  uint16_t *kc, *vc;
  int64_t tokens;
  int32_t heads, kv_heads, dim, page_log2, pages, axes, pairs;
  bool adjacent, bf16;
};
hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t s);

// Page src[i] of every layer to page dst[i]; page_bytes of one array's page.
hipError_t launch_cache_copy(uint8_t* kc, uint8_t* vc, int64_t layers, int64_t pages, int64_t page_bytes,
                             const int32_t* src, const int32_t* dst, int64_t n, hipStream_t s);

constexpr int kKeepMost = 256;
struct CacheKeepArgs {
  uint16_t *kc, *vc;
  const int32_t* tables;  // [seqs, ldt], max_pages entries each
  const int32_t* starts;
  const int32_t* kept;  // [seqs, most]
  int32_t* lengths;
  int64_t ldt;
  int32_t layers, seqs, most, max_pages, kv_heads, dim, page_log2, pages;
};
hipError_t launch_cache_keep(const CacheKeepArgs& a, hipStream_t s);

// Caps up to here take the form of tanh that is off by 4 * 2^-23 of the cap: 6e-5 of a weight at
// 128, a 64th of its rounding to bf16.
constexpr float kNearCap = 128.f;

struct AttendArgs {
  const uint16_t* q;
  const uint16_t *kc, *vc;
  const int32_t *offsets, *lengths, *tables;
  const float* slopes;
  const int32_t* prefix;
  const int32_t* first;
  const uint64_t* mask;
  void* y;
  float* lse;    // [tokens, heads] or null
  float* part;   // [splits][tokens * heads][dim] rows, then [splits][tokens * heads][2] maximum and weight
  int64_t ldq, ldy, ldt;
  int32_t tokens, seqs, heads, kv_heads, group, dim, page_log2, pages, max_pages, words, window;
  int32_t rows;    // of one sequence and head of the cache that the call is laid out for
  int32_t splits;  // parts of the keys
  int32_t chunk;   // blocks of 32 keys a part
  float scale, cap;
  float cap_in, cap_out;  // 2 scale / cap and the cap, both in powers of two, and finite
  bool y_bf16;
};
// Rows of a workgroup of the kernel for many rows.
constexpr int kAttendRows = 128;
// The rule on sizes that chooses kernel and parts.
struct AttendPlan {
  bool wide;  // kAttendRows a workgroup, else 32
  int32_t rows, splits, chunk;
  size_t bytes;  // of the workspace
};
AttendPlan attend_plan(int64_t tokens, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim, int64_t max_tokens,
                       int64_t max_length, int64_t window = 0);
hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, hipStream_t s);
hipError_t launch_attend_few(const AttendArgs& a, hipStream_t s);   // (with its parts set)
hipError_t launch_attend_many(const AttendArgs& a, hipStream_t s);

}  // namespace uw
