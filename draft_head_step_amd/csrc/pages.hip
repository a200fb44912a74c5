// Page bookkeeping of the paged cache for CDNA4 (gfx950): pages and slots for
// the new elements of a batch, and pages back to the pool.
//
//   page_map:  need_r = ceil((cur_r + n_r) / P) - ceil(cur_r / P) from a ring of
//              free pages, S = exclusive scan(need); request r is served if
//              S_r + need_r <= count.
//   page_trim: give_r = ceil(cur_r / P) - ceil(keep_r / P) to the ring's end.
//
// One launch each, and no workgroup waits for another: every workgroup scans
// all R needs by itself (8 bytes a request, from L2 after the first), then
// takes its share of the page entries and of the slots.  A slot on a page that
// this very call hands out is computed from the ring, not read back from the
// table.  The free pages are a ring and not a stack, so that the entries that
// a call reads (from the head) and those that it writes (behind the end) are
// never the same, and the pool's state after the call goes to another address
// than the state before it: the kernel needs no ticket, no second launch and
// no cleared counters, and can be run again with the same result.
//
// Bound by the chain of dependent reads (lengths, scan, search, ring or table), not
// by bytes: 256 requests of a step take 7.0 us to map and 3.3 to trim, 64 prompts
// of 0.5 million elements (4.4 MB, of which the slots are 4.2) 10.3 and 6.8.
#include "dspark_internal.h"
#include "paged.h"

namespace dspark {
namespace {

constexpr int kT = 256;
constexpr int kW = kT / 64;
constexpr int kSlotsPerThread = 4;

// Exclusive prefix of v over the workgroup, and the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sh, int64_t* total) {
  const int lane = threadIdx.x & 63;
  const int w = threadIdx.x >> 6;
  int64_t inc = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up(inc, off);
    inc += lane >= off ? o : 0;
  }
  __syncthreads();
  if (lane == 63) sh[w] = inc;
  __syncthreads();
  int64_t pre = 0, all = 0;
#pragma unroll
  for (int j = 0; j < kW; ++j) {
    pre += j < w ? sh[j] : 0;
    all += sh[j];
  }
  *total = all;
  return pre + inc - v;
}

// Last r in [0, n) with a[r] <= x (a[0] <= x, a not decreasing).
__device__ __forceinline__ int last_le(const int32_t* a, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// LDS: before[R] = pages that requests 0 .. r-1 take (served ones only, so it
// ends at the number taken), bit r of ok[] = served.
__global__ __launch_bounds__(kT) void page_map_kernel(
    const int32_t* __restrict__ cur, const int32_t* __restrict__ cu, int R, int max_tokens,
    int shift, int max_pages, int num_pages, int32_t* __restrict__ table,
    const int32_t* __restrict__ ring, const dspark_page_pool* __restrict__ pool,
    dspark_page_pool* __restrict__ pool_out, int64_t* __restrict__ slots,
    int32_t* __restrict__ new_len) {
  extern __shared__ int32_t lds[];
  int32_t* before = lds;              // [R]
  int32_t* start = lds + R;           // [R]
  uint32_t* ok = reinterpret_cast<uint32_t*>(lds + 2 * R);   // [ceil(R / 32)]
  __shared__ int64_t sh[kW];
  const int t = threadIdx.x;
  const int head = ring_head(pool->head, num_pages);
  const int count = ring_count(pool->count, num_pages);
  for (int i = t; i < (R + 31) / 32; i += kT) ok[i] = 0;
  // each thread's own run of requests
  const int per = (R + kT - 1) / kT;
  const int r0 = min(t * per, R), r1 = min(r0 + per, R);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    const PageNeed p = page_need(cur[r], cu[r], cu[r + 1], shift, max_pages);
    mine += p.fits ? p.want - p.has : 0;
  }
  int64_t total;
  int64_t s = block_scan(mine, sh, &total);   // its barriers cover the clears above
  // A request with a need is served if S + need <= count.  S only grows, so
  // once one is turned down every later one with a need is too, and the pages
  // taken are a prefix: min(S, first S that failed).
  int refused = 0;
  int64_t taken = 0;
  for (int r = r0; r < r1; ++r) {
    const PageNeed p = page_need(cur[r], cu[r], cu[r + 1], shift, max_pages);
    const int64_t need = p.fits ? p.want - p.has : 0;
    const bool served = p.fits && (need == 0 || s + need <= count);
    before[r] = (int32_t)(s < count ? s : count);
    start[r] = cu[r];
    if (served) atomicOr(&ok[r >> 5], 1u << (r & 31));
    if (served && need > 0) taken = s + need;
    refused += served ? 0 : 1;
    s += need;
    if (blockIdx.x == 0) new_len[r] = served ? (int32_t)(cur[r] + (cu[r + 1] - cu[r])) : cur[r];
  }
  // the most that any served request took up to its end
  {
    const int lane = t & 63, w = t >> 6;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const int64_t o = __shfl_xor(taken, off);
      taken = o > taken ? o : taken;
      refused += __shfl_xor(refused, off);
    }
    __syncthreads();
    if (lane == 0) sh[w] = (taken << 20) | refused;   // refused <= 16384 < 2^20
    __syncthreads();
    taken = 0;
    refused = 0;
#pragma unroll
    for (int j = 0; j < kW; ++j) {
      const int64_t a = sh[j] >> 20;
      taken = a > taken ? a : taken;
      refused += (int)(sh[j] & ((1 << 20) - 1));
    }
  }
  if (blockIdx.x == 0 && t == 0) {
    dspark_page_pool o;
    o.head = ring_at(head, taken, num_pages);
    o.count = count - (int)taken;
    o.refused = refused;
    o.reserved = 0;
    *pool_out = o;
  }
  const int64_t step = (int64_t)gridDim.x * kT;
  const int64_t first = (int64_t)blockIdx.x * kT + t;
  // Page entries: entry i of the ring goes to the last request whose run starts
  // at or before it (those without a need share their start with the next one).
  for (int64_t i = first; i < taken; i += step) {
    const int r = last_le(before, R, (int32_t)i);
    const int64_t at = pages_of(cur[r], shift) + (i - before[r]);
    table[(size_t)r * max_pages + at] = ring[ring_at(head, i, num_pages)];
  }
  // Slots: kSlotsPerThread elements in a row for each thread.
  const int32_t all = cu[R];
  const int64_t N = all < max_tokens ? all : max_tokens;
  for (int64_t e0 = first * kSlotsPerThread; e0 < N; e0 += step * kSlotsPerThread) {
    int r = last_le(start, R, (int32_t)e0);
    int64_t end = r + 1 < R ? start[r + 1] : all;
#pragma unroll
    for (int u = 0; u < kSlotsPerThread; ++u) {
      const int64_t e = e0 + u;
      if (e >= N) break;
      while (e >= end) {   // also over empty segments
        ++r;
        end = r + 1 < R ? start[r + 1] : all;
      }
      int64_t slot = -1;
      if (e >= start[r] && ((ok[r >> 5] >> (r & 31)) & 1u)) {
        const int32_t c = cur[r];
        const int64_t pos = c + (e - start[r]);
        const int64_t at = pos >> shift;
        const int64_t has = pages_of(c, shift);
        const int32_t page = at < has ? table[(size_t)r * max_pages + at]
                                      : ring[ring_at(head, before[r] + (at - has), num_pages)];
        if (page_ok(page, num_pages))
          slot = ((int64_t)page << shift) + (pos & ((1 << shift) - 1));
      }
      slots[e] = slot;
    }
  }
}

__global__ __launch_bounds__(kT) void page_trim_kernel(
    const int32_t* __restrict__ cur, const int32_t* __restrict__ keep, int R, int shift,
    int max_pages, int num_pages, const int32_t* __restrict__ table, int32_t* __restrict__ ring,
    const dspark_page_pool* __restrict__ pool, dspark_page_pool* __restrict__ pool_out) {
  extern __shared__ int32_t lds[];
  int32_t* before = lds;   // [R]
  __shared__ int64_t sh[kW];
  const int t = threadIdx.x;
  const int head = ring_head(pool->head, num_pages);
  const int count = ring_count(pool->count, num_pages);
  const int per = (R + kT - 1) / kT;
  const int r0 = min(t * per, R), r1 = min(r0 + per, R);
  int64_t mine = 0;
  int refused = 0;
  for (int r = r0; r < r1; ++r) {
    const PageNeed p = page_give(cur[r], keep[r], shift, max_pages);
    mine += p.has - p.want;
    refused += p.fits ? 0 : 1;
  }
  int64_t total;
  int64_t s = block_scan(mine, sh, &total);
  const bool over = count + total > num_pages;
  for (int r = r0; r < r1; ++r) {
    const PageNeed p = page_give(cur[r], keep[r], shift, max_pages);
    before[r] = (int32_t)(s < num_pages ? s : num_pages);
    s += p.has - p.want;
  }
  int64_t down;
  block_scan(refused, sh, &down);   // its barriers also publish before[]
  if (blockIdx.x == 0 && t == 0) {
    dspark_page_pool o;
    o.head = head;
    o.count = over ? count : (int)(count + total);
    o.refused = over ? R : (int)down;
    o.reserved = 0;
    *pool_out = o;
  }
  if (over) return;
  const int64_t step = (int64_t)gridDim.x * kT;
  for (int64_t i = (int64_t)blockIdx.x * kT + t; i < total; i += step) {
    const int r = last_le(before, R, (int32_t)i);
    const PageNeed p = page_give(cur[r], keep[r], shift, max_pages);
    ring[ring_at(head, count + i, num_pages)] =
        table[(size_t)r * max_pages + p.want + (i - before[r])];
  }
}

// Workgroups for `items` of work per call: one scan of R lengths costs each of
// them a few microseconds, so a small call runs on few.
int grid_for(int64_t items, int per_group) {
  const int64_t g = (items + per_group - 1) / per_group;
  return (int)(g < 1 ? 1 : g > 256 ? 256 : g);
}

}  // namespace

dspark_status launch_page_map(const int32_t* cur_len, const int32_t* cu, int R, int max_tokens,
                              int shift, int max_pages, int num_pages, int32_t* table,
                              const int32_t* ring, const dspark_page_pool* pool,
                              dspark_page_pool* pool_out, int64_t* slots, int32_t* new_len,
                              hipStream_t stream) {
  const size_t lds = (2 * (size_t)R + (R + 31) / 32) * sizeof(int32_t);
  if (lds > 48 * 1024) {
    const dspark_status st = allow_lds(reinterpret_cast<const void*>(&page_map_kernel),
                                       (2 * DSPARK_MAX_PAGE_REQUESTS +
                                        DSPARK_MAX_PAGE_REQUESTS / 32) * (int)sizeof(int32_t),
                                       "page_map");
    if (st != DSPARK_OK) return st;
  }
  hipLaunchKernelGGL(page_map_kernel, dim3(grid_for(max_tokens, kT * kSlotsPerThread)), dim3(kT),
                     lds, stream, cur_len, cu, R, max_tokens, shift, max_pages, num_pages, table,
                     ring, pool, pool_out, slots, new_len);
  return check_launch("page_map_kernel");
}

dspark_status launch_page_trim(const int32_t* cur_len, const int32_t* keep_len, int R, int shift,
                               int max_pages, int num_pages, const int32_t* table, int32_t* ring,
                               const dspark_page_pool* pool, dspark_page_pool* pool_out,
                               hipStream_t stream) {
  const size_t lds = (size_t)R * sizeof(int32_t);
  if (lds > 48 * 1024) {
    const dspark_status st = allow_lds(reinterpret_cast<const void*>(&page_trim_kernel),
                                       DSPARK_MAX_PAGE_REQUESTS * (int)sizeof(int32_t),
                                       "page_trim");
    if (st != DSPARK_OK) return st;
  }
  const int64_t most = (int64_t)R * max_pages;   // pages that could come back
  hipLaunchKernelGGL(page_trim_kernel, dim3(grid_for(most < num_pages ? most : num_pages, 4 * kT)),
                     dim3(kT), lds, stream, cur_len, keep_len, R, shift, max_pages, num_pages,
                     table, ring, pool, pool_out);
  return check_launch("page_trim_kernel");
}

}  // namespace dspark
