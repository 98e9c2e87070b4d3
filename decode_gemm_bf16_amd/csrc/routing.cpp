// C ABI (include/uw.h) of the routing of rows to experts and back and of the
// low-rank adapters: every argument is checked on the host before any launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/uw.h"
#include "routing.h"
#include "runtime_internal.h"

struct uw_adapters {
  int64_t rows = 0, cols = 0, rows64 = 0;
  int32_t slots = 0, max_rank = 0, rank16 = 0;
  int device = 0;
  void* mem = nullptr;
  uint16_t* a = nullptr;
  uint16_t* b = nullptr;
  uw::LoraSlot* table = nullptr;
};

namespace {

uw_status fail(uw_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return uw::set_error(st, buf);
}

#define UW_HIP(call)                                                                       \
  do {                                                                                     \
    hipError_t e_ = (call);                                                                \
    if (e_ != hipSuccess) return fail(UW_ERR_HIP, "%s: %s", #call, hipGetErrorString(e_)); \
  } while (0)

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxEntries = int64_t(1) << 30;
constexpr int64_t kMaxLoraTokens = int64_t(1) << 20;  // two halves of every tile within a grid dimension

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

// The same for two [rows, cols] float matrices with row strides: column windows
// of one wider matrix (one stride) do not overlap where their columns do not.
bool overlap_rows(const float* p, int64_t pcols, int64_t ldp, const float* q, int64_t qcols, int64_t ldq,
                  int64_t rows) {
  const size_t np = size_t((rows - 1) * ldp + pcols) * 4, nq = size_t((rows - 1) * ldq + qcols) * 4;
  if (!overlap(p, np, q, nq)) return false;
  if (ldp != ldq) return true;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) / 4;
  const int64_t m = ((d % ldp) + ldp) % ldp;  // q's first column in p's rows
  return m < pcols || m + qcols > ldp;
}

// Bytes from the first to past the last element of [rows, cols] with row stride ld.
size_t span(int64_t rows, int64_t cols, int64_t ld, size_t size) { return size_t((rows - 1) * ld + cols) * size; }

uw_status check_tokens(int64_t tokens, int64_t most = kMaxTokens) {
  if (tokens < 1) return fail(UW_ERR_INVALID_ARG, "tokens must be >= 1");
  if (tokens > most) return fail(UW_ERR_INVALID_ARG, "tokens too large");
  return UW_OK;
}

uw_status check_entries(int64_t tokens, int32_t top_k, int64_t cols, int64_t cols_multiple, int64_t rows) {
  uw_status st = check_tokens(tokens);
  if (st != UW_OK) return st;
  if (top_k < 1 || tokens * top_k > kMaxEntries) return fail(UW_ERR_INVALID_ARG, "top_k %d out of range", top_k);
  if (cols < 1 || cols > (int64_t(1) << 24) || cols % cols_multiple)
    return fail(UW_ERR_SHAPE, "cols = %lld must be a multiple of %lld", (long long)cols, (long long)cols_multiple);
  if (rows < 1 || rows > kMaxEntries) return fail(UW_ERR_INVALID_ARG, "rows out of range");
  return UW_OK;
}

// The plan's parts: header, tiles, offsets of the order, work of the grouping.
struct PlanParts {
  size_t tiles, order, work, total;
};
PlanParts plan_parts(int64_t tokens, int32_t slots) {
  PlanParts p;
  p.tiles = align256(sizeof(uw::PlanHeader));
  p.order = p.tiles + align256(size_t(uw::lora_tiles_max(tokens, slots)) * sizeof(uw::PlanTile));
  p.work = p.order + align256(size_t(tokens) * 4);
  p.total = p.work + align256(uw::group_work_bytes(tokens, slots));
  return p;
}

uw_status check_plan(const void* plan, size_t bytes, int64_t tokens, int32_t slots) {
  if (!plan) return fail(UW_ERR_INVALID_ARG, "null plan");
  if (!aligned(plan, 16)) return fail(UW_ERR_INVALID_ARG, "the plan must be 16-byte aligned");
  const size_t need = plan_parts(tokens, slots).total;
  if (bytes < need)
    return fail(UW_ERR_INVALID_ARG, "plan of %zu bytes, %lld tokens and %d slots need %zu", bytes, (long long)tokens,
                slots, need);
  return UW_OK;
}

uw_status check_slots(int32_t slots) {
  if (slots < 1 || slots > uw::kGroupMax) return fail(UW_ERR_INVALID_ARG, "slots must be 1..%d", uw::kGroupMax);
  return UW_OK;
}

}  // namespace

namespace uw {

uw_status route_check(const void* logits, int32_t type, int64_t ld, int64_t tokens, const float* bias,
                      const uw_route_config* c, const int32_t* experts, const float* weights) {
  if (!logits || !c || !experts || !weights) return fail(UW_ERR_INVALID_ARG, "null argument");
  uw_status st = check_tokens(tokens);
  if (st != UW_OK) return st;
  if (type != UW_F32 && type != UW_BF16) return fail(UW_ERR_INVALID_ARG, "unknown logit type %d", type);
  if (c->experts < 1 || c->experts > kRouteMaxExperts)
    return fail(UW_ERR_SHAPE, "experts = %d must be 1..%d", c->experts, kRouteMaxExperts);
  if (c->top_k < 1 || c->top_k > c->experts || c->top_k > kRouteMaxTopK)
    return fail(UW_ERR_INVALID_ARG, "top_k = %d must be 1..%d and at most the experts", c->top_k, kRouteMaxTopK);
  if (c->groups < 1 || c->groups > kRouteMaxGroups || c->experts % c->groups)
    return fail(UW_ERR_SHAPE, "groups = %d must be 1..%d and divide the experts", c->groups, kRouteMaxGroups);
  if (c->top_groups < 1 || c->top_groups > c->groups)
    return fail(UW_ERR_INVALID_ARG, "top_groups = %d must be 1..groups", c->top_groups);
  if (c->score != UW_SCORE_SOFTMAX && c->score != UW_SCORE_SIGMOID)
    return fail(UW_ERR_INVALID_ARG, "unknown score %d", c->score);
  if (c->group_score != UW_GROUP_MAX && c->group_score != UW_GROUP_TOP2)
    return fail(UW_ERR_INVALID_ARG, "unknown group score %d", c->group_score);
  if (!std::isfinite(c->scale)) return fail(UW_ERR_INVALID_ARG, "scale must be finite");
  if (ld < c->experts) return fail(UW_ERR_SHAPE, "row stride %lld below %d experts", (long long)ld, c->experts);
  const size_t size = type == UW_F32 ? 4 : 2;
  if (!aligned(logits, size) || (bias && !aligned(bias, 4)) || !aligned(experts, 4) || !aligned(weights, 4))
    return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
  const size_t in = span(tokens, c->experts, ld, size), out = size_t(tokens) * c->top_k * 4;
  const size_t nb = bias ? size_t(c->experts) * 4 : 0;
  if (overlap(logits, in, experts, out) || overlap(logits, in, weights, out) || overlap(experts, out, weights, out) ||
      (bias && (overlap(bias, nb, experts, out) || overlap(bias, nb, weights, out))))
    return fail(UW_ERR_INVALID_ARG, "outputs overlap an input or each other");
  return UW_OK;
}

uw_status route_launch(const void* logits, int32_t type, int64_t ld, int64_t tokens, const float* bias,
                       const uw_route_config* c, int32_t* experts, float* weights, hipStream_t s) {
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.index = experts;
  a.weight = weights;
  a.ld = ld;
  a.tokens = tokens;
  a.experts = c->experts;
  a.top_k = c->top_k;
  a.groups = c->groups;
  a.top_groups = c->top_groups;
  a.bf16 = type == UW_BF16;
  a.sigmoid = c->score == UW_SCORE_SIGMOID;
  a.pairs = c->group_score == UW_GROUP_TOP2;
  a.renormalise = c->renormalise != 0;
  a.scale = c->scale;
  UW_HIP(launch_route(a, s));
  return UW_OK;
}

}  // namespace uw

extern "C" {

uw_status uw_route(const void* logits_dev, int32_t type, int64_t ld, int64_t tokens, const float* bias_dev,
                   const uw_route_config* config, int32_t* experts_dev, float* weights_dev, void* stream) {
  uw_status st = uw::route_check(logits_dev, type, ld, tokens, bias_dev, config, experts_dev, weights_dev);
  if (st != UW_OK) return st;
  return uw::route_launch(logits_dev, type, ld, tokens, bias_dev, config, experts_dev, weights_dev,
                          static_cast<hipStream_t>(stream));
}

size_t uw_group_rows_workspace_bytes(int64_t n, int32_t groups) {
  if (n < 1 || n > kMaxEntries || groups < 1 || groups > uw::kGroupMax) return 0;
  return uw::group_work_bytes(n, groups);
}

uw_status uw_group_rows(const int32_t* index_dev, int64_t n, int32_t groups, int32_t* offsets_dev, int32_t* order_dev,
                        int32_t* slot_dev, void* work_dev, size_t work_bytes, void* stream) {
  if (!index_dev || !offsets_dev || !order_dev || !slot_dev) return fail(UW_ERR_INVALID_ARG, "null argument");
  if (n < 1 || n > kMaxEntries) return fail(UW_ERR_INVALID_ARG, "n must be 1..%lld", (long long)kMaxEntries);
  if (groups < 1 || groups > uw::kGroupMax) return fail(UW_ERR_INVALID_ARG, "groups must be 1..%d", uw::kGroupMax);
  const size_t need = uw::group_work_bytes(n, groups), nb = size_t(n) * 4, ob = size_t(groups + 1) * 4;
  if (need && (!work_dev || work_bytes < need))
    return fail(UW_ERR_INVALID_ARG, "workspace of %zu bytes, %lld entries need %zu", work_dev ? work_bytes : size_t(0),
                (long long)n, need);
  const void* const ps[5] = {index_dev, offsets_dev, order_dev, slot_dev, work_dev};
  const size_t bs[5] = {nb, ob, nb, nb, need};
  for (int i = 0; i < 5; ++i) {
    if (bs[i] && !aligned(ps[i], 4)) return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
    for (int j = 0; j < i; ++j)
      if (bs[i] && bs[j] && overlap(ps[i], bs[i], ps[j], bs[j]))
        return fail(UW_ERR_INVALID_ARG, "buffers overlap");
  }
  uw::GroupArgs a{index_dev, n, groups, offsets_dev, order_dev, slot_dev, static_cast<int32_t*>(work_dev), nullptr,
                  nullptr};
  UW_HIP(uw::launch_group_rows(a, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

uw_status uw_dispatch_rows(const uint16_t* x_dev, int64_t ldx, const int32_t* slot_dev, int64_t tokens, int32_t top_k,
                           int64_t cols, uint16_t* xs_dev, int64_t rows, void* stream) {
  if (!x_dev || !slot_dev || !xs_dev) return fail(UW_ERR_INVALID_ARG, "null argument");
  uw_status st = check_entries(tokens, top_k, cols, 8, rows);
  if (st != UW_OK) return st;
  if (ldx < cols || ldx % 8) return fail(UW_ERR_SHAPE, "row stride %lld of x must be >= cols and a multiple of 8", (long long)ldx);
  if (!aligned(x_dev, 16) || !aligned(xs_dev, 16) || !aligned(slot_dev, 4))
    return fail(UW_ERR_INVALID_ARG, "x and xs must be 16-byte aligned");
  const size_t out = size_t(rows) * cols * 2;
  if (overlap(x_dev, span(tokens, cols, ldx, 2), xs_dev, out) || overlap(slot_dev, size_t(tokens) * top_k * 4, xs_dev, out))
    return fail(UW_ERR_INVALID_ARG, "xs overlaps an input");
  UW_HIP(uw::launch_dispatch_rows(x_dev, ldx, slot_dev, tokens, top_k, cols, xs_dev, rows,
                                  static_cast<hipStream_t>(stream)));
  return UW_OK;
}

uw_status uw_combine_rows(const float* ys_dev, int64_t rows, const int32_t* slot_dev, const float* weights_dev,
                          int64_t tokens, int32_t top_k, int64_t cols, const float* base_dev, void* y_dev,
                          int32_t y_type, void* stream) {
  if (!ys_dev || !slot_dev || !weights_dev || !y_dev) return fail(UW_ERR_INVALID_ARG, "null argument");
  uw_status st = check_entries(tokens, top_k, cols, 8, rows);
  if (st != UW_OK) return st;
  if (y_type != UW_F32 && y_type != UW_BF16) return fail(UW_ERR_INVALID_ARG, "unknown output type %d", y_type);
  if (!aligned(ys_dev, 16) || !aligned(y_dev, 16) || (base_dev && !aligned(base_dev, 16)) || !aligned(slot_dev, 4) ||
      !aligned(weights_dev, 4))
    return fail(UW_ERR_INVALID_ARG, "ys, base and y must be 16-byte aligned");
  const size_t out = size_t(tokens) * cols * (y_type == UW_F32 ? 4 : 2), in = size_t(tokens) * top_k * 4;
  const bool in_place = base_dev == y_dev && y_type == UW_F32;
  if (overlap(ys_dev, size_t(rows) * cols * 4, y_dev, out) || overlap(slot_dev, in, y_dev, out) ||
      overlap(weights_dev, in, y_dev, out) ||
      (base_dev && !in_place && overlap(base_dev, size_t(tokens) * cols * 4, y_dev, out)))
    return fail(UW_ERR_INVALID_ARG, "y overlaps an input (a float32 y may be base itself)");
  UW_HIP(uw::launch_combine_rows(ys_dev, slot_dev, weights_dev, tokens, top_k, cols, rows, base_dev, y_dev,
                                 y_type == UW_BF16, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

uw_status uw_lora_create(int64_t rows, int64_t cols, int32_t slots, int32_t max_rank, uw_lora* out) {
  if (!out) return fail(UW_ERR_INVALID_ARG, "null output");
  if (rows < 16 || cols < 64 || rows % 16 || cols % 64 || rows > (int64_t(1) << 23) || cols > (int64_t(1) << 23))
    return fail(UW_ERR_SHAPE, "rows must be a multiple of 16 and cols a multiple of 64");
  uw_status st = check_slots(slots);
  if (st != UW_OK) return st;
  if (max_rank < 1 || max_rank > UW_LORA_MAX_RANK)
    return fail(UW_ERR_INVALID_ARG, "max_rank must be 1..%d", UW_LORA_MAX_RANK);
  int ndev = 0, dev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess || ndev < 1) return fail(UW_ERR_NO_DEVICE, "no HIP device");
  UW_HIP(hipGetDevice(&dev));
  uw_adapters* h = new (std::nothrow) uw_adapters;
  if (!h) return fail(UW_ERR_OOM, "host allocation failed");
  h->rows = rows;
  h->cols = cols;
  h->slots = slots;
  h->max_rank = max_rank;
  h->rank16 = (max_rank + 15) / 16 * 16;
  h->device = dev;
  h->rows64 = (rows + 63) / 64 * 64;
  const size_t each = size_t(slots) * h->rank16 * 2, na = align256(each * cols), nb = align256(each * h->rows64);
  const size_t nt = align256(size_t(slots) * sizeof(uw::LoraSlot));
  if (hipMalloc(&h->mem, na + nb + nt) != hipSuccess) {
    delete h;
    return fail(UW_ERR_OOM, "device allocation of %zu bytes failed", na + nb + nt);
  }
  h->a = static_cast<uint16_t*>(h->mem);
  h->b = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(h->mem) + na);
  h->table = reinterpret_cast<uw::LoraSlot*>(static_cast<uint8_t*>(h->mem) + na + nb);
  // empty slots (rank 0), finished on return: later calls may use any stream
  if (hipMemset(h->table, 0, nt) != hipSuccess || hipDeviceSynchronize() != hipSuccess) {
    (void)hipFree(h->mem);
    delete h;
    return fail(UW_ERR_HIP, "clearing the adapter table failed");
  }
  *out = h;
  return UW_OK;
}

uw_status uw_lora_load(uw_lora h, int32_t slot, const uint16_t* a_dev, const uint16_t* b_dev, int32_t rank, float scale,
                       void* stream) {
  if (!h) return fail(UW_ERR_INVALID_ARG, "null handle");
  if (slot < 0 || slot >= h->slots) return fail(UW_ERR_INVALID_ARG, "slot %d outside 0..%d", slot, h->slots - 1);
  if (rank < 0 || rank > h->max_rank) return fail(UW_ERR_INVALID_ARG, "rank %d outside 0..%d", rank, h->max_rank);
  if (rank > 0 && (!a_dev || !b_dev)) return fail(UW_ERR_INVALID_ARG, "null adapter matrix");
  if (rank > 0 && (!aligned(a_dev, 2) || !aligned(b_dev, 2))) return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
  int dev = 0;
  UW_HIP(hipGetDevice(&dev));
  if (dev != h->device) return fail(UW_ERR_INVALID_ARG, "the adapters are on device %d, current is %d", h->device, dev);
  const int64_t r16 = h->rank16;
  UW_HIP(uw::launch_lora_load(a_dev, b_dev, h->rows, h->cols, rank, scale, h->a + slot * r16 * h->cols,
                              h->b + slot * r16 * h->rows64, h->table + slot, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

void uw_lora_free(uw_lora h) {
  if (!h) return;
  int dev = 0;  // the work that may still read the slots runs on the adapters' device
  const bool other = hipGetDevice(&dev) == hipSuccess && dev != h->device && hipSetDevice(h->device) == hipSuccess;
  (void)hipDeviceSynchronize();
  (void)hipFree(h->mem);
  if (other) (void)hipSetDevice(dev);
  delete h;
}

size_t uw_lora_plan_bytes(int64_t tokens, int32_t slots) {
  if (tokens < 1 || tokens > kMaxLoraTokens || slots < 1 || slots > uw::kGroupMax) return 0;
  return plan_parts(tokens, slots).total;
}

uw_status uw_lora_plan(const int32_t* slot_dev, int64_t tokens, int32_t slots, void* plan_dev, size_t plan_bytes,
                       void* stream) {
  if (!slot_dev) return fail(UW_ERR_INVALID_ARG, "null argument");
  uw_status st = check_tokens(tokens, kMaxLoraTokens);
  if (st != UW_OK || (st = check_slots(slots)) != UW_OK) return st;
  if ((st = check_plan(plan_dev, plan_bytes, tokens, slots)) != UW_OK) return st;
  if (!aligned(slot_dev, 4)) return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
  const PlanParts p = plan_parts(tokens, slots);
  if (overlap(slot_dev, size_t(tokens) * 4, plan_dev, p.total))
    return fail(UW_ERR_INVALID_ARG, "the plan overlaps the slots");
  uint8_t* m = static_cast<uint8_t*>(plan_dev);
  uw::GroupArgs a{slot_dev,
                  tokens,
                  slots,
                  nullptr,
                  reinterpret_cast<int32_t*>(m + p.order),
                  nullptr,
                  reinterpret_cast<int32_t*>(m + p.work),
                  reinterpret_cast<uw::PlanHeader*>(m),
                  reinterpret_cast<uw::PlanTile*>(m + p.tiles)};
  UW_HIP(uw::launch_group_rows(a, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

size_t uw_lora_workspace_bytes(const uw_lora* adapters, int32_t n, int64_t tokens) {
  if (!adapters || n < 1 || n > uw::kLoraMaxProj || tokens < 1 || tokens > kMaxLoraTokens) return 0;
  size_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (!adapters[i]) return 0;
    const int k = uw::lora_ksplit(tokens, adapters[i]->slots, adapters[i]->cols, n);
    total += align256(size_t(k) * size_t(tokens) * adapters[i]->rank16 * 4);
  }
  return total;
}

uw_status uw_lora_apply(const uw_lora* adapters, int32_t n, const void* plan_dev, size_t plan_bytes,
                        const uint16_t* x_dev, int64_t ldx, const float* const* bases_dev, const int64_t* ldbase,
                        float* const* ys_dev, const int64_t* ldy, int64_t tokens, void* work_dev, size_t work_bytes,
                        void* stream) {
  if (!adapters || !x_dev || !ys_dev || !ldy || !work_dev || (bases_dev && !ldbase))
    return fail(UW_ERR_INVALID_ARG, "null argument");
  if (n < 1 || n > uw::kLoraMaxProj) return fail(UW_ERR_INVALID_ARG, "n must be 1..%d projections", uw::kLoraMaxProj);
  uw_status st = check_tokens(tokens, kMaxLoraTokens);
  if (st != UW_OK) return st;
  for (int i = 0; i < n; ++i) {
    if (!adapters[i] || !ys_dev[i]) return fail(UW_ERR_INVALID_ARG, "null adapters or output %d", i);
    if (adapters[i]->cols != adapters[0]->cols || adapters[i]->slots != adapters[0]->slots)
      return fail(UW_ERR_SHAPE, "projection %d has other cols or slots than projection 0", i);
    if (adapters[i]->device != adapters[0]->device)
      return fail(UW_ERR_INVALID_ARG, "projection %d is on another device", i);
  }
  const int64_t cols = adapters[0]->cols;
  const int32_t slots = adapters[0]->slots;
  if ((st = check_plan(plan_dev, plan_bytes, tokens, slots)) != UW_OK) return st;
  if (ldx < cols || ldx % 8) return fail(UW_ERR_SHAPE, "row stride %lld of x must be >= cols and a multiple of 8", (long long)ldx);
  if (!aligned(x_dev, 16)) return fail(UW_ERR_INVALID_ARG, "x must be 16-byte aligned");
  if (!aligned(work_dev, 256)) return fail(UW_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
  const size_t need = uw_lora_workspace_bytes(adapters, n, tokens);
  if (work_bytes < need)
    return fail(UW_ERR_INVALID_ARG, "workspace of %zu bytes, %lld tokens need %zu", work_bytes, (long long)tokens, need);
  const PlanParts parts = plan_parts(tokens, slots);
  // the products with A go to the workspace while other workgroups read x and the plan
  if (overlap(work_dev, need, x_dev, span(tokens, cols, ldx, 2)) || overlap(work_dev, need, plan_dev, parts.total))
    return fail(UW_ERR_INVALID_ARG, "the workspace overlaps x or the plan");
  const uint8_t* m = static_cast<const uint8_t*>(plan_dev);
  uw::LoraArgs a{};
  int64_t written = 0;
  a.ksplit = uw::lora_ksplit(tokens, slots, cols, n);
  a.halves = uw::lora_halves(tokens, slots, n);
  uint8_t* cur = static_cast<uint8_t*>(work_dev);
  for (int i = 0; i < n; ++i) {
    const uw_adapters* h = adapters[i];
    const float* base = bases_dev ? bases_dev[i] : nullptr;
    const int64_t lb = base ? ldbase[i] : 0;
    if (ldy[i] < h->rows || ldy[i] % 4 || (base && (lb < h->rows || lb % 4)))
      return fail(UW_ERR_SHAPE, "row strides of projection %d must be >= rows and multiples of 4", i);
    if (!aligned(ys_dev[i], 16) || (base && !aligned(base, 16)))
      return fail(UW_ERR_INVALID_ARG, "bases and outputs must be 16-byte aligned");
    if (base && overlap(work_dev, need, base, span(tokens, h->rows, lb, 4)))
      return fail(UW_ERR_INVALID_ARG, "the workspace overlaps base %d", i);
    const size_t out = span(tokens, h->rows, ldy[i], 4);
    const bool in_place = base == ys_dev[i] && lb == ldy[i];
    bool bad = overlap(x_dev, span(tokens, cols, ldx, 2), ys_dev[i], out) ||
               overlap(plan_dev, parts.total, ys_dev[i], out) || overlap(work_dev, need, ys_dev[i], out);
    for (int j = 0; j < n; ++j) {
      if (j < i) bad = bad || overlap_rows(ys_dev[j], adapters[j]->rows, ldy[j], ys_dev[i], h->rows, ldy[i], tokens);
      const float* other = bases_dev ? bases_dev[j] : nullptr;
      if (other && !(j == i && in_place))
        bad = bad || overlap_rows(other, adapters[j]->rows, ldbase[j], ys_dev[i], h->rows, ldy[i], tokens);
    }
    if (bad) return fail(UW_ERR_INVALID_ARG, "output %d overlaps an input or another output (it may be its own base)", i);
    uw::LoraProj& p = a.proj[i];
    p.a = h->a;
    p.b = h->b;
    p.table = h->table;
    p.base = base;
    p.y = ys_dev[i];
    p.ldbase = lb;
    p.ldy = ldy[i];
    p.rows = (int32_t)h->rows;
    p.rank16 = h->rank16;
    written += tokens * h->rows * 4;
    p.part = reinterpret_cast<float*>(cur);
    cur += align256(size_t(a.ksplit) * size_t(tokens) * h->rank16 * 4);
  }
  int dev = 0;
  UW_HIP(hipGetDevice(&dev));
  if (dev != adapters[0]->device)
    return fail(UW_ERR_INVALID_ARG, "the adapters are on device %d, current is %d", adapters[0]->device, dev);
  a.header = reinterpret_cast<const uw::PlanHeader*>(m);
  a.tiles = reinterpret_cast<const uw::PlanTile*>(m + parts.tiles);
  a.order = reinterpret_cast<const int32_t*>(m + parts.order);
  a.x = x_dev;
  a.ldx = ldx;
  a.tokens = (int32_t)tokens;
  a.slots = slots;
  a.cols = (int32_t)cols;
  a.nproj = n;
  a.stream = written >= (int64_t(128) << 20);  // half of the 256 MB Infinity Cache
  a.tiles_max = (int32_t)uw::lora_tiles_max(tokens, slots);
  UW_HIP(uw::launch_lora_apply(a, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

}  // extern "C"
