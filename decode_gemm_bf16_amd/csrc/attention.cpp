// C ABI (include/uw.h) of the paged cache of keys and values and of attention over
// it: every argument is checked on the host before any launch.
#include "attention.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <limits>

#include "../../include/uw.h"
#include "runtime_internal.h"

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

constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxSeqs = 65535;
constexpr int64_t kMaxLayers = 4096;
constexpr int64_t kMaxPlaces = (int64_t(1) << 31) - 1;

// A buffer of a call: its first byte and its size.
struct Span {
  const void* p;
  size_t n;
};

bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

size_t rows_bytes(int64_t rows, int64_t cols, int64_t ld, size_t size) {
  return rows < 1 ? 0 : (size_t(rows - 1) * ld + cols) * size;
}

// The first `outs` buffers are written: none may meet another of the call.
uw_status check_apart(const Span* s, int outs, int all) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < all; ++j)
      if (meet(s[i], s[j])) return fail(UW_ERR_INVALID_ARG, "an output overlaps an input or another output");
  return UW_OK;
}

uw_status check_cache_sizes(const uw_cache_config* c) {
  if (!c) return fail(UW_ERR_INVALID_ARG, "null argument");
  if (c->kv_heads < 1 || c->kv_heads > 128) return fail(UW_ERR_SHAPE, "kv_heads = %d must be 1..128", c->kv_heads);
  if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 256)
    return fail(UW_ERR_SHAPE, "dim = %d must be 64, 96, 128 or 256", c->dim);
  if (c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256)
    return fail(UW_ERR_SHAPE, "page = %d must be 32, 64, 128 or 256", c->page);
  if (c->pages < 1 || c->pages > kMaxPlaces / c->page)
    return fail(UW_ERR_INVALID_ARG, "pages = %lld out of range", (long long)c->pages);
  return UW_OK;
}

uw_status check_cache(const uw_cache_config* c, const void* k, const void* v) {
  if (!c || !k || !v) return fail(UW_ERR_INVALID_ARG, "null argument");
  const uw_status st = check_cache_sizes(c);
  if (st != UW_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(UW_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
  return UW_OK;
}

uw_status check_heads(const uw_cache_config* c) {
  if (c->heads < c->kv_heads || c->heads > 256 || c->heads % c->kv_heads || c->heads / c->kv_heads > 64)
    return fail(UW_ERR_SHAPE, "heads = %d must be a multiple of the %d kv_heads, at most 64 times and 256", c->heads,
                c->kv_heads);
  return UW_OK;
}

uw_status check_tokens(int64_t tokens) {
  if (tokens < 1 || tokens > kMaxTokens)
    return fail(UW_ERR_INVALID_ARG, "tokens = %lld must be 1..%lld", (long long)tokens, (long long)kMaxTokens);
  return UW_OK;
}

uw_status check_layers(int64_t layers) {
  if (layers < 1 || layers > kMaxLayers)
    return fail(UW_ERR_INVALID_ARG, "layers = %lld must be 1..%lld", (long long)layers, (long long)kMaxLayers);
  return UW_OK;
}

uw_status check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld % 8)
    return fail(UW_ERR_SHAPE, "row stride %lld of %s must be at least %lld and a multiple of 8", (long long)ld, name,
                (long long)cols);
  return UW_OK;
}

int log2_of(int32_t v) { return v == 32 ? 5 : v == 64 ? 6 : v == 128 ? 7 : 8; }

size_t cache_bytes(const uw_cache_config* c, int64_t layers = 1) {
  return size_t(layers) * c->pages * c->kv_heads * c->page * c->dim * 2;
}

uw_status check_sequences(int64_t seqs, int64_t ldt, int64_t max_pages) {
  if (seqs < 1 || seqs > kMaxSeqs) return fail(UW_ERR_INVALID_ARG, "seqs must be 1..%lld", (long long)kMaxSeqs);
  if (max_pages < 1 || max_pages > (int64_t(1) << 24) || ldt < max_pages)
    return fail(UW_ERR_SHAPE, "max_pages = %lld must be 1..2^24 and at most the tables' row stride %lld",
                (long long)max_pages, (long long)ldt);
  return UW_OK;
}

uw_status check_attend_sizes(int64_t tokens, int64_t max_tokens, int64_t max_length) {
  if (max_tokens < 1 || max_tokens > tokens || max_length < 1 || max_length > (int64_t(1) << 30))
    return fail(UW_ERR_INVALID_ARG, "max_tokens must be 1..tokens and max_length 1..2^30");
  return UW_OK;
}

}  // namespace

namespace uw {

uw_status attention_sizes_check(const uw_cache_config* config, int64_t tokens, int64_t seqs, int64_t max_tokens,
                                int64_t max_length) {
  uw_status st = check_cache_sizes(config);
  if (st != UW_OK || (st = check_heads(config)) != UW_OK || (st = check_tokens(tokens)) != UW_OK ||
      (st = check_sequences(seqs, 1, 1)) != UW_OK)
    return st;
  return check_attend_sizes(tokens, max_tokens, max_length);
}

uw_status cache_write_prepare(const uw_cache_config* config, const uw_rotary* rotary, const void* q_dev, int64_t ldq,
                              const void* k_dev, int64_t ldk, const void* v_dev, int64_t ldv, int32_t type,
                              const int32_t* positions_dev, const float* freqs_dev, const int32_t* axis_dev,
                              const int32_t* slots_dev, int64_t tokens, uint16_t* q_out_dev, int64_t ldq_out,
                              uint16_t* k_cache_dev, uint16_t* v_cache_dev, CacheWriteArgs* out) {
  uw_status st = check_cache(config, k_cache_dev, v_cache_dev);
  if (st != UW_OK) return st;
  const uw_cache_config& c = *config;
  if (!rotary || !k_dev || !v_dev || !slots_dev || (q_dev && !q_out_dev)) return fail(UW_ERR_INVALID_ARG, "null argument");
  if ((q_dev && (st = check_heads(config)) != UW_OK) || (st = check_tokens(tokens)) != UW_OK) return st;
  if (type != UW_F32 && type != UW_BF16) return fail(UW_ERR_INVALID_ARG, "unknown type %d", type);
  if (rotary->axes < 1 || rotary->axes > kRotaryMaxAxes)
    return fail(UW_ERR_INVALID_ARG, "axes = %d must be 1..%d", rotary->axes, kRotaryMaxAxes);
  if (rotary->pairs < 0 || rotary->pairs > c.dim / 2)
    return fail(UW_ERR_SHAPE, "pairs = %d must be 0..%d", rotary->pairs, c.dim / 2);
  if (rotary->pairs > 0 && (!positions_dev || !freqs_dev)) return fail(UW_ERR_INVALID_ARG, "null positions or frequencies");
  const int64_t qc = q_dev ? int64_t(c.heads) * c.dim : 0, kc = int64_t(c.kv_heads) * c.dim;
  if ((q_dev && ((st = check_ld(ldq, qc, "q")) != UW_OK || (st = check_ld(ldq_out, qc, "q_out")) != UW_OK)) ||
      (st = check_ld(ldk, kc, "k")) != UW_OK || (st = check_ld(ldv, kc, "v")) != UW_OK)
    return st;
  if (!aligned(q_dev, 16) || !aligned(k_dev, 16) || !aligned(v_dev, 16) || (q_dev && !aligned(q_out_dev, 16)))
    return fail(UW_ERR_INVALID_ARG, "q, k, v and q_out must be 16-byte aligned");
  if (!aligned(positions_dev, 4) || !aligned(freqs_dev, 4) || !aligned(axis_dev, 4) || !aligned(slots_dev, 4))
    return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
  const size_t size = type == UW_F32 ? 4 : 2, np = size_t(rotary->pairs) * 4;
  const bool turn = rotary->pairs > 0;
  const Span spans[] = {{q_dev ? q_out_dev : nullptr, rows_bytes(tokens, qc, ldq_out, 2)},
                        {k_cache_dev, cache_bytes(config)},
                        {v_cache_dev, cache_bytes(config)},
                        {q_dev, rows_bytes(tokens, qc, ldq, size)},
                        {k_dev, rows_bytes(tokens, kc, ldk, size)},
                        {v_dev, rows_bytes(tokens, kc, ldv, size)},
                        {turn ? positions_dev : nullptr, size_t(tokens) * rotary->axes * 4},
                        {turn ? freqs_dev : nullptr, np},
                        {turn ? axis_dev : nullptr, np},
                        {slots_dev, size_t(tokens) * 4}};
  if ((st = check_apart(spans, 3, 10)) != UW_OK) return st;
  CacheWriteArgs& a = *out;
  a.q = q_dev;
  a.k = k_dev;
  a.v = v_dev;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldqo = ldq_out;
  a.positions = positions_dev;
  a.freqs = freqs_dev;
  a.axis = axis_dev;
  a.slots = slots_dev;
  a.qo = q_out_dev;
  a.kc = k_cache_dev;
  a.vc = v_cache_dev;
  a.tokens = tokens;
  a.heads = q_dev ? c.heads : 0;
  a.kv_heads = c.kv_heads;
  a.dim = c.dim;
  a.page_log2 = log2_of(c.page);
  a.pages = (int32_t)c.pages;
  a.axes = rotary->axes;
  a.pairs = rotary->pairs;
  a.adjacent = rotary->adjacent != 0;
  a.bf16 = type == UW_BF16;
  return UW_OK;
}

uw_status attend_prepare(const uw_cache_config* config, const uw_attend_config* options, const uint16_t* q_dev,
                         int64_t ldq, const uint16_t* k_cache_dev, const uint16_t* v_cache_dev, const int32_t* offsets_dev,
                         const int32_t* lengths_dev, const int32_t* tables_dev, int64_t ldt, int64_t max_pages,
                         const float* slopes_dev, const int32_t* prefix_dev, const int32_t* first_dev,
                         const uint64_t* mask_dev, int32_t mask_words, int64_t tokens, int64_t seqs, int64_t max_tokens,
                         int64_t max_length, void* y_dev, int64_t ldy, int32_t y_type, float* lse_dev, void* work_dev,
                         size_t work_bytes, AttendArgs* out, AttendPlan* plan_out) {
  uw_status st = check_cache(config, k_cache_dev, v_cache_dev);
  if (st != UW_OK) return st;
  const uw_cache_config& c = *config;
  if (!options || !q_dev || !offsets_dev || !lengths_dev || !tables_dev || !y_dev)
    return fail(UW_ERR_INVALID_ARG, "null argument");
  if ((st = check_heads(config)) != UW_OK || (st = check_tokens(tokens)) != UW_OK ||
      (st = check_sequences(seqs, ldt, max_pages)) != UW_OK ||
      (st = check_attend_sizes(tokens, max_tokens, max_length)) != UW_OK)
    return st;
  if (y_type != UW_F32 && y_type != UW_BF16) return fail(UW_ERR_INVALID_ARG, "unknown output type %d", y_type);
  if (!std::isfinite(options->scale) || options->scale <= 0.f)
    return fail(UW_ERR_INVALID_ARG, "scale must be positive and finite");
  if (!std::isfinite(options->cap) || options->cap < 0.f) return fail(UW_ERR_INVALID_ARG, "cap must be 0 or positive and finite");
  if (options->window < 0) return fail(UW_ERR_INVALID_ARG, "window must be 0 or positive");
  if (mask_dev && (mask_words < 1 || mask_words > 1024)) return fail(UW_ERR_SHAPE, "mask_words = %d must be 1..1024", mask_words);
  if (mask_dev && prefix_dev) return fail(UW_ERR_UNSUPPORTED, "a prefix and a mask of drafted tokens exclude each other");
  const int64_t cols = int64_t(c.heads) * c.dim;
  if ((st = check_ld(ldq, cols, "q")) != UW_OK || (st = check_ld(ldy, cols, "y")) != UW_OK) return st;
  if (!aligned(q_dev, 16) || !aligned(y_dev, 16)) return fail(UW_ERR_INVALID_ARG, "q and y must be 16-byte aligned");
  if (!aligned(offsets_dev, 4) || !aligned(lengths_dev, 4) || !aligned(tables_dev, 4) || !aligned(slopes_dev, 4) ||
      !aligned(prefix_dev, 4) || !aligned(first_dev, 4) || !aligned(mask_dev, 8) || !aligned(lse_dev, 4))
    return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
  AttendPlan& plan = *plan_out;
  plan = attend_plan(tokens, seqs, c.heads, c.kv_heads, c.dim, max_tokens, max_length, prefix_dev ? 0 : options->window);
  if (plan.bytes && (!work_dev || work_bytes < plan.bytes))
    return fail(UW_ERR_INVALID_ARG, "workspace of %zu bytes, the call needs %zu", work_dev ? work_bytes : size_t(0), plan.bytes);
  if (plan.bytes && !aligned(work_dev, 16)) return fail(UW_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
  const Span spans[] = {{y_dev, rows_bytes(tokens, cols, ldy, y_type == UW_F32 ? 4 : 2)},
                        {lse_dev, size_t(tokens) * c.heads * 4},
                        {work_dev, plan.bytes},
                        {q_dev, rows_bytes(tokens, cols, ldq, 2)},
                        {k_cache_dev, cache_bytes(config)},
                        {v_cache_dev, cache_bytes(config)},
                        {offsets_dev, size_t(seqs + 1) * 4},
                        {lengths_dev, size_t(seqs) * 4},
                        {tables_dev, rows_bytes(seqs, max_pages, ldt, 4)},
                        {slopes_dev, size_t(c.heads) * 4},
                        {prefix_dev, size_t(seqs) * 4},
                        {first_dev, size_t(tokens) * 4},
                        {mask_dev, size_t(tokens) * size_t(mask_dev ? mask_words : 0) * 8}};
  if ((st = check_apart(spans, 3, 13)) != UW_OK) return st;
  AttendArgs& a = *out;
  a.q = q_dev;
  a.kc = k_cache_dev;
  a.vc = v_cache_dev;
  a.offsets = offsets_dev;
  a.lengths = lengths_dev;
  a.tables = tables_dev;
  a.slopes = slopes_dev;
  a.prefix = prefix_dev;
  a.first = first_dev;
  a.mask = mask_dev;
  a.y = y_dev;
  a.lse = lse_dev;
  a.part = static_cast<float*>(work_dev);
  a.ldq = ldq;
  a.ldy = ldy;
  a.ldt = ldt;
  a.tokens = (int32_t)tokens;
  a.seqs = (int32_t)seqs;
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.group = c.heads / c.kv_heads;
  a.dim = c.dim;
  a.page_log2 = log2_of(c.page);
  a.pages = (int32_t)c.pages;
  a.max_pages = (int32_t)max_pages;
  a.words = mask_dev ? mask_words : 0;
  a.window = options->window < (1 << 30) ? options->window : 0;  // (no two places are further apart)
  a.scale = options->scale;
  a.cap = options->cap;
  // (kept finite, so that a product of zero stays zero and a cap less itself is zero)
  const double log2e = 1.4426950408889634, most = std::numeric_limits<float>::max();
  a.cap_in = a.cap > 0.f ? float(std::min(double(a.scale) / a.cap * 2 * log2e, most)) : 0.f;
  a.cap_out = float(std::min(a.cap * log2e, most / 2));
  a.y_bf16 = y_type == UW_BF16;
  return UW_OK;
}

}  // namespace uw

extern "C" {

uw_status uw_cache_write(const uw_cache_config* config, const uw_rotary* rotary, const void* q_dev, int64_t ldq,
                         const void* k_dev, int64_t ldk, const void* v_dev, int64_t ldv, int32_t type,
                         const int32_t* positions_dev, const float* freqs_dev, const int32_t* axis_dev,
                         const int32_t* slots_dev, int64_t tokens, uint16_t* q_out_dev, int64_t ldq_out,
                         uint16_t* k_cache_dev, uint16_t* v_cache_dev, void* stream) {
  uw::CacheWriteArgs a;
  const uw_status st = uw::cache_write_prepare(config, rotary, q_dev, ldq, k_dev, ldk, v_dev, ldv, type, positions_dev,
                                               freqs_dev, axis_dev, slots_dev, tokens, q_out_dev, ldq_out, k_cache_dev,
                                               v_cache_dev, &a);
  if (st != UW_OK) return st;
  UW_HIP(uw::launch_cache_write(a, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

size_t uw_attend_workspace_bytes(int64_t tokens, int64_t seqs, int32_t heads, int32_t kv_heads, int32_t dim,
                                 int64_t max_tokens, int64_t max_length) {
  const uw_cache_config c = {heads, kv_heads, dim, 32, 1};
  if (uw::attention_sizes_check(&c, tokens, seqs, max_tokens, max_length) != UW_OK) return 0;
  return uw::attend_plan(tokens, seqs, heads, kv_heads, dim, max_tokens, max_length).bytes;
}

uw_status uw_attend(const uw_cache_config* config, const uw_attend_config* options, const uint16_t* q_dev, int64_t ldq,
                    const uint16_t* k_cache_dev, const uint16_t* v_cache_dev, const int32_t* offsets_dev,
                    const int32_t* lengths_dev, const int32_t* tables_dev, int64_t ldt, int64_t max_pages,
                    const float* slopes_dev, const int32_t* prefix_dev, const int32_t* first_dev,
                    const uint64_t* mask_dev, int32_t mask_words, int64_t tokens, int64_t seqs, int64_t max_tokens,
                    int64_t max_length, void* y_dev, int64_t ldy, int32_t y_type, float* lse_dev, void* work_dev,
                    size_t work_bytes, void* stream) {
  uw::AttendArgs a;
  uw::AttendPlan plan;
  const uw_status st = uw::attend_prepare(
      config, options, q_dev, ldq, k_cache_dev, v_cache_dev, offsets_dev, lengths_dev, tables_dev, ldt, max_pages,
      slopes_dev, prefix_dev, first_dev, mask_dev, mask_words, tokens, seqs, max_tokens, max_length, y_dev, ldy, y_type,
      lse_dev, work_dev, work_bytes, &a, &plan);
  if (st != UW_OK) return st;
  UW_HIP(uw::launch_attend(a, plan, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

uw_status uw_cache_copy_pages(const uw_cache_config* config, int64_t layers, uint16_t* k_cache_dev,
                              uint16_t* v_cache_dev, const int32_t* src_dev, const int32_t* dst_dev, int64_t n,
                              void* stream) {
  uw_status st = check_cache(config, k_cache_dev, v_cache_dev);
  if (st != UW_OK || (st = check_layers(layers)) != UW_OK) return st;
  if (!src_dev || !dst_dev) return fail(UW_ERR_INVALID_ARG, "null argument");
  if (n < 1 || n > config->pages) return fail(UW_ERR_INVALID_ARG, "n = %lld must be 1..pages", (long long)n);
  if (!aligned(src_dev, 4) || !aligned(dst_dev, 4)) return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
  const size_t bytes = cache_bytes(config, layers);
  const Span spans[] = {{k_cache_dev, bytes}, {v_cache_dev, bytes}, {src_dev, size_t(n) * 4}, {dst_dev, size_t(n) * 4}};
  if ((st = check_apart(spans, 2, 4)) != UW_OK) return st;
  UW_HIP(uw::launch_cache_copy(reinterpret_cast<uint8_t*>(k_cache_dev), reinterpret_cast<uint8_t*>(v_cache_dev), layers,
                               config->pages, int64_t(config->kv_heads) * config->page * config->dim * 2, src_dev,
                               dst_dev, n, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

uw_status uw_cache_keep(const uw_cache_config* config, int64_t layers, uint16_t* k_cache_dev, uint16_t* v_cache_dev,
                        const int32_t* tables_dev, int64_t ldt, int64_t max_pages, const int32_t* starts_dev,
                        const int32_t* kept_dev, int32_t most, int64_t seqs, int32_t* lengths_dev, void* stream) {
  uw_status st = check_cache(config, k_cache_dev, v_cache_dev);
  if (st != UW_OK || (st = check_layers(layers)) != UW_OK || (st = check_sequences(seqs, ldt, max_pages)) != UW_OK)
    return st;
  if (!tables_dev || !starts_dev || !kept_dev || !lengths_dev) return fail(UW_ERR_INVALID_ARG, "null argument");
  if (most < 1 || most > uw::kKeepMost) return fail(UW_ERR_SHAPE, "most = %d must be 1..%d", most, uw::kKeepMost);
  if (!aligned(tables_dev, 4) || !aligned(starts_dev, 4) || !aligned(kept_dev, 4) || !aligned(lengths_dev, 4))
    return fail(UW_ERR_INVALID_ARG, "misaligned pointer");
  const size_t bytes = cache_bytes(config, layers), ns = size_t(seqs) * 4;
  const Span spans[] = {{k_cache_dev, bytes},
                        {v_cache_dev, bytes},
                        {lengths_dev, ns},
                        {tables_dev, rows_bytes(seqs, max_pages, ldt, 4)},
                        {starts_dev, ns},
                        {kept_dev, ns * most}};
  if ((st = check_apart(spans, 3, 6)) != UW_OK) return st;
  uw::CacheKeepArgs a;
  a.kc = k_cache_dev;
  a.vc = v_cache_dev;
  a.tables = tables_dev;
  a.starts = starts_dev;
  a.kept = kept_dev;
  a.lengths = lengths_dev;
  a.ldt = ldt;
  a.layers = (int32_t)layers;
  a.seqs = (int32_t)seqs;
  a.most = most;
  a.max_pages = (int32_t)max_pages;
  a.kv_heads = config->kv_heads;
  a.dim = config->dim;
  a.page_log2 = log2_of(config->page);
  a.pages = (int32_t)config->pages;
  UW_HIP(uw::launch_cache_keep(a, static_cast<hipStream_t>(stream)));
  return UW_OK;
}

}  // extern "C"
