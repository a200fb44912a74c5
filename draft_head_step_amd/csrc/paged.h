// Index arithmetic of the paged cache, shared by its kernels and (compiled for
// the host) by the CPU tests.  Every address that a kernel forms from page
// tables, slots or lengths in device memory goes through these functions, so
// what they refuse is never touched.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define DSPARK_HD __host__ __device__ __forceinline__
#else
#define DSPARK_HD inline
#endif

namespace dspark {

constexpr int kMinPage = 16;
constexpr int kMaxPage = 1024;
constexpr int64_t kMaxLen = 0x7fffffff;   // of a request, kept as int32

// log2 of a page size, -1 if it is not a power of two in [16, 1024].
DSPARK_HD int page_shift(int page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

// Pages that hold `len` tokens (len >= 0).
DSPARK_HD int64_t pages_of(int64_t len, int shift) {
  return (len + ((int64_t)1 << shift) - 1) >> shift;
}

DSPARK_HD bool page_ok(int32_t page, int num_pages) {
  return (uint32_t)page < (uint32_t)num_pages;
}

DSPARK_HD bool slot_ok(int64_t slot, int shift, int num_pages) {
  return slot >= 0 && slot < ((int64_t)num_pages << shift);
}

// What dspark_page_map does for one request: the pages that it has and wants,
// and whether its lengths fit, into the table and into an int32 (otherwise it
// asks for nothing).
struct PageNeed {
  int64_t has, want;
  bool fits;
};
DSPARK_HD PageNeed page_need(int32_t cur, int32_t first, int32_t end, int shift, int max_pages) {
  PageNeed p;
  const int64_t n = (int64_t)end - first;
  p.fits = cur >= 0 && n >= 0 && first >= 0;
  p.has = p.fits ? pages_of(cur, shift) : 0;
  p.want = p.fits ? pages_of((int64_t)cur + n, shift) : 0;
  p.fits = p.fits && p.want <= max_pages && cur + n <= kMaxLen;
  return p;
}

// What dspark_page_trim does for one request.
DSPARK_HD PageNeed page_give(int32_t cur, int32_t keep, int shift, int max_pages) {
  PageNeed p;
  const int32_t k = keep < 0 ? 0 : keep > cur ? cur : keep;
  p.fits = cur >= 0 && pages_of(cur, shift) <= max_pages;
  p.has = p.fits ? pages_of(cur, shift) : 0;
  p.want = p.fits ? pages_of(k, shift) : 0;
  return p;
}

// A pool's head and count, brought into their ranges.
DSPARK_HD int ring_head(int32_t head, int num_pages) {
  const int h = head % num_pages;
  return h < 0 ? h + num_pages : h;
}
DSPARK_HD int ring_count(int32_t count, int num_pages) {
  return count < 0 ? 0 : count > num_pages ? num_pages : count;
}
// Ring place `i` entries behind `head` (0 <= i <= 2 * num_pages).
DSPARK_HD int ring_at(int head, int64_t i, int num_pages) {
  return (int)((head + i) % num_pages);
}

// Element offsets in the two caches; c = elements in 16 bytes.
DSPARK_HD int64_t k_offset(int64_t page, int h, int d, int o, int Hk, int D, int shift, int c) {
  return ((((page * Hk + h) * (D / c) + d / c) << shift) + o) * c + d % c;
}
DSPARK_HD int64_t v_offset(int64_t page, int h, int d, int o, int Hk, int D, int shift) {
  return (((page * Hk + h) * D + d) << shift) + o;
}

// Whether an accepted path can be moved: path[0] = 0, then strictly increasing, so that
// path[i] >= i.  That is asked for too: entries are judged apart, and one behind a bad
// entry must not lead to a position before the segment.
DSPARK_HD bool path_step_ok(const int32_t* path, int i) {
  return i == 0 ? path[0] == 0 : path[i] > path[i - 1] && path[i] >= i;
}

// A parent link of node i.
DSPARK_HD bool parent_ok(int32_t parent, int i) { return parent >= -1 && parent < i; }

}  // namespace dspark
