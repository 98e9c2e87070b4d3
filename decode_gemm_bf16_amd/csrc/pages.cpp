// The pages of a cache, counted on the host (include/uw.h): which are free, how many
// tables hold each of the others, which have to be copied or moved.  The rows
// themselves are copied by uw_cache_copy_pages.
#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <functional>
#include <new>
#include <vector>

#include "../../include/uw.h"
#include "runtime_internal.h"

struct uw_page_counts {
  std::vector<int32_t> count;  // tables that hold a page; 0: free
  // Pages from `fresh` on have not been taken yet; the free ones before it are in `freed`, a
  // heap with the lowest in front and room for every page: freeing one cannot fail.
  int64_t fresh = 0;
  std::vector<int32_t> freed;
  int64_t used = 0;
};

namespace {

uw_status fail(uw_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return uw::set_error(st, buf);
}

bool taken(const uw_page_counts* p, int32_t page) {
  return page >= 0 && page < (int64_t)p->count.size() && p->count[page] > 0;
}

int32_t take_one(uw_page_counts* p) {
  int32_t page;
  if (!p->freed.empty()) {
    page = p->freed.front();
    std::pop_heap(p->freed.begin(), p->freed.end(), std::greater<int32_t>());
    p->freed.pop_back();
  } else {
    page = (int32_t)p->fresh++;
  }
  p->count[page] = 1;
  ++p->used;
  return page;
}

void drop_one(uw_page_counts* p, int32_t page) {
  if (--p->count[page] > 0) return;
  p->freed.push_back(page);
  std::push_heap(p->freed.begin(), p->freed.end(), std::greater<int32_t>());
  --p->used;
}

uw_status check_list(uw_pages p, const int32_t* pages, int64_t n) {
  if (!p || n < 0 || (n > 0 && !pages)) return fail(UW_ERR_INVALID_ARG, "null argument or negative number");
  for (int64_t i = 0; i < n; ++i)
    if (!taken(p, pages[i])) return fail(UW_ERR_INVALID_ARG, "page %d is not taken", pages[i]);
  return UW_OK;
}

template <typename F>
uw_status guarded(F f) {  // no exception leaves a C entry
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(UW_ERR_OOM, "host allocation failed");
  }
}

}  // namespace

extern "C" {

uw_status uw_pages_create(int64_t pages, uw_pages* out) {
  if (!out) return fail(UW_ERR_INVALID_ARG, "null output");
  if (pages < 1 || pages > (int64_t(1) << 26)) return fail(UW_ERR_INVALID_ARG, "pages must be 1..2^26");
  return guarded([&] {
    uw_page_counts* p = new uw_page_counts;
    try {
      p->count.assign(size_t(pages), 0);
      p->freed.reserve(size_t(pages));
    } catch (...) {
      delete p;
      throw;
    }
    *out = p;
    return UW_OK;
  });
}

void uw_pages_free(uw_pages p) { delete p; }

int64_t uw_pages_left(uw_pages p) { return p ? (int64_t)p->count.size() - p->used : 0; }

int32_t uw_pages_holders(uw_pages p, int32_t page) { return p && taken(p, page) ? p->count[page] : 0; }

uw_status uw_pages_take(uw_pages p, int64_t n, int32_t* pages) {
  if (!p || n < 0 || (n > 0 && !pages)) return fail(UW_ERR_INVALID_ARG, "null argument or negative number");
  if (n > uw_pages_left(p))
    return fail(UW_ERR_OOM, "%lld pages asked for, %lld left", (long long)n, (long long)uw_pages_left(p));
  for (int64_t i = 0; i < n; ++i) pages[i] = take_one(p);
  return UW_OK;
}

uw_status uw_pages_share(uw_pages p, const int32_t* pages, int64_t n) {
  const uw_status st = check_list(p, pages, n);
  if (st != UW_OK) return st;
  for (int64_t i = 0; i < n; ++i)
    if (p->count[pages[i]] > (1 << 30)) return fail(UW_ERR_INVALID_ARG, "page %d has too many holders", pages[i]);
  for (int64_t i = 0; i < n; ++i) ++p->count[pages[i]];
  return UW_OK;
}

uw_status uw_pages_drop(uw_pages p, const int32_t* pages, int64_t n) {
  uw_status st = check_list(p, pages, n);
  if (st != UW_OK) return st;
  return guarded([&] {
    // a list may name a page as often as it has holders
    std::vector<int32_t> sorted(pages, pages + n);
    std::sort(sorted.begin(), sorted.end());
    for (int64_t i = 0, run = 0; i < n; ++i) {
      run = i > 0 && sorted[i] == sorted[i - 1] ? run + 1 : 1;
      if (run > p->count[sorted[i]]) return fail(UW_ERR_INVALID_ARG, "page %d is dropped more often than held", sorted[i]);
    }
    for (int64_t i = 0; i < n; ++i) drop_one(p, pages[i]);
    return UW_OK;
  });
}

uw_status uw_pages_own(uw_pages p, int32_t page, int32_t* own) {
  if (!own) return fail(UW_ERR_INVALID_ARG, "null output");
  const uw_status st = check_list(p, &page, 1);
  if (st != UW_OK) return st;
  if (p->count[page] == 1) {
    *own = page;
    return UW_OK;
  }
  if (uw_pages_left(p) < 1) return fail(UW_ERR_OOM, "no page is left");
  return guarded([&] {
    *own = take_one(p);
    drop_one(p, page);
    return UW_OK;
  });
}

uw_status uw_pages_compact(uw_pages p, int32_t* src, int32_t* dst, int64_t* n) {
  if (!p || !src || !dst || !n) return fail(UW_ERR_INVALID_ARG, "null argument");
  return guarded([&] {
    const int64_t used = p->used, all = (int64_t)p->count.size();
    int64_t moves = 0, to = 0;
    for (int64_t from = used; from < all; ++from) {
      if (p->count[from] == 0) continue;
      while (p->count[to] > 0) ++to;
      p->count[to] = p->count[from];
      p->count[from] = 0;
      src[moves] = (int32_t)from;
      dst[moves++] = (int32_t)to;
    }
    p->fresh = used;
    p->freed.clear();
    *n = moves;
    return UW_OK;
  });
}

}  // extern "C"
