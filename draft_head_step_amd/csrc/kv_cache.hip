// Writes to the paged key/value cache for CDNA4 (gfx950).
//
//   kv_store:  K and V rows of new elements into their slots.  The keys keep 16
//              bytes (c elements) of a row together, [D / c][P][c]; the values
//              lie transposed, [D][P].  A workgroup takes 32 or 64 elements of
//              one head: rows are read 16 bytes a lane, pass through LDS, and are
//              written with neighbouring lanes on neighbouring elements, which
//              in a run of slots are neighbouring addresses in both caches.
//              The keys' stores are non-temporal (whole lines that nobody reads
//              soon: 38 us, then 30); values share lines with other workgroups
//              and are not.  18.8 thousand elements of 8 heads of 128 take 29 us
//              in bf16 (5.4 TB/s, a copy of 2 GB reaches 4.95) and 26 us in e4m3
//              (4.5 TB/s; 39 with a division for every value).
//   kv_commit: the accepted path's keys and values to the front.  A thread
//              owns 16-byte pieces of the keys and value channels and moves each
//              for i = 1, 2, ... in turn, four positions' loads at a time.
//              path[i] >= i and path increases, so position i, once written, is
//              no later source.  Places in the cache are worked out once per
//              request, in LDS.  Values move one number at a time, and 64 lanes
//              of a load or store touch 64 channels, each a page's width from the
//              next: 64 paths in 32 layers of 8 heads of 128 in e4m3 (20 MB to
//              read and write) take 35 us in pages of 16, 58 in pages of 32 and 140
//              in pages of 128 (bf16: 83, 124 and 162).  In pages of 32 the counters
//              see 52 MB read and 78 written, half of what a copy moves in that
//              time, so the accesses and not the bytes are what it costs.  One
//              layer of 32 paths in bf16 takes 6.9.
#include <type_traits>

#include "dspark_internal.h"
#include "paged.h"

namespace dspark {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kT = 256;
// Rows of one head from which a workgroup takes 64 elements: four workgroups a CU.
// 64 instead of 32: 28.5 us and 29.7 for 151 thousand rows of 128 (pages of 64: 29.3
// and 32.1; heads of 64: 12.8 and 15.4; of 256: 67 and 76, in e4m3 51 and 49), but
// 9.1 and 8.4 for the 7 thousand of a step.
constexpr int64_t kManyRows = 64 * 1024;

__device__ __forceinline__ float widen(uint16_t x, bool bf) {
  return bf ? __builtin_bit_cast(float, (uint32_t)x << 16)
            : (float)__builtin_bit_cast(_Float16, x);
}

// rne_e4m3 of x clamped to the finite range; comparisons leave NaN as it is.
__device__ __forceinline__ uint8_t to_e4m3(float x) {
  x = x > 448.0f ? 448.0f : x;
  x = x < -448.0f ? -448.0f : x;
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false);
}

// e4m3 of x / scale for eight values.  x times 1 / scale a little less and a little
// more (2^-21: the reciprocal, its shift, the product and the quotient are each off
// by 2^-24 at most) encloses the rounded quotient, and rounding to e4m3 is monotone:
// where both ends round alike and stay in range that is the result, a fifth of the
// instructions of a division.  Otherwise the division decides.
struct Scale {
  float s, low, high;
  bool wide;   // the reciprocal is no normal number with room for the products
};
__device__ __forceinline__ Scale make_scale(float s) {
  const float r = 1.0f / s;
  return {s, r * (1.0f - 0x1p-21f), r * (1.0f + 0x1p-21f),
          !(fabsf(r) >= 0x1p-100f && fabsf(r) <= 0x1p100f)};
}
__device__ __forceinline__ void eight_to_e4m3(u32x4 a, int bf, const Scale& sc, uint8_t* out) {
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = widen((uint16_t)(a[j >> 1] >> ((j & 1) * 16)), bf);
  uint32_t lo[2], hi[2];
  float top = 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float* y = x + 4 * w;
    int l = 0, u = 0;
    l = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * sc.low, y[1] * sc.low, l, false);
    l = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * sc.low, y[3] * sc.low, l, true);
    float z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z[j] = y[j] * sc.high;
      top = fmaxf(top, fabsf(z[j]));
    }
    u = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], u, false);
    u = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], u, true);
    lo[w] = l;
    hi[w] = u;
  }
  if (sc.wide || !(top <= 448.0f) || lo[0] != hi[0] || lo[1] != hi[1]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = to_e4m3(x[j] / sc.s);
  } else {
    __builtin_memcpy(out, lo, 8);
  }
}

// Grid: (ceil(max_tokens / kTok), Hk).  F8: 8-bit cache of 16-bit inputs.
template <int D, bool F8, int kTok>
__global__ __launch_bounds__(kT) void kv_store_kernel(
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t k_stride,
    int64_t v_stride, int bf, const int64_t* __restrict__ slots, const int32_t* __restrict__ count,
    int max_tokens, int Hk, int shift, int num_pages, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache) {
  constexpr int kEl = F8 ? 1 : 2;
  constexpr int kC = 16 / kEl;
  constexpr int kRow = D * kEl;        // bytes of a stored row
  // rows padded by 16 bytes: the transposed reads then spread over the banks
  __shared__ __align__(16) uint8_t ks[kTok][kRow + 16];
  __shared__ __align__(16) uint8_t vs[kTok][kRow + 16];
  __shared__ int64_t slot[kTok];
  const int t = threadIdx.x;
  const int h = blockIdx.y;
  const int64_t e0 = (int64_t)blockIdx.x * kTok;
  int64_t n = max_tokens;
  if (count) n = count[0] < n ? count[0] : n;
  n = n - e0 < kTok ? n - e0 : kTok;
  if (n <= 0) return;
  if (t < kTok) slot[t] = t < n ? slots[e0 + t] : -1;
  const Scale sk = make_scale(F8 ? k_scale[h] : 1.0f);
  const Scale sv = make_scale(F8 ? v_scale[h] : 1.0f);
  constexpr int kPieces = D / 8;   // 16-byte pieces of an input row
  // all of a thread's loads before the first conversion
  constexpr int kLoads = (kTok * kPieces + kT - 1) / kT;
  u32x4 la[kLoads], lb[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = min(t + u * kT, (int)n * kPieces - 1);
    const int e = i / kPieces, p = i - e * kPieces;
    la[u] = *reinterpret_cast<const u32x4*>(k + (e0 + e) * k_stride + h * D + p * 8);
    lb[u] = *reinterpret_cast<const u32x4*>(v + (e0 + e) * v_stride + h * D + p * 8);
  }
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = t + u * kT;
    if (i >= (int)n * kPieces) break;
    const int e = i / kPieces, p = i - e * kPieces;
    const u32x4 a = la[u], b = lb[u];
    if (F8) {
      uint8_t oa[8], ob[8];
      eight_to_e4m3(a, bf, sk, oa);
      eight_to_e4m3(b, bf, sv, ob);
      __builtin_memcpy(&ks[e][p * 8], oa, 8);
      __builtin_memcpy(&vs[e][p * 8], ob, 8);
    } else {
      *reinterpret_cast<u32x4*>(&ks[e][p * 16]) = a;
      *reinterpret_cast<u32x4*>(&vs[e][p * 16]) = b;
    }
  }
  __syncthreads();
  const int e = t & (kTok - 1);
  const int64_t s = slot[e];
  if (!slot_ok(s, shift, num_pages)) return;
  const int64_t page = s >> shift;
  const int o = (int)(s & ((1 << shift) - 1));
  for (int p = t / kTok; p < D / kC; p += kT / kTok)
    __builtin_nontemporal_store(
        *reinterpret_cast<const u32x4*>(&ks[e][p * 16]),
        reinterpret_cast<u32x4*>(k_cache + k_offset(page, h, p * kC, o, Hk, D, shift, kC) * kEl));
  for (int d = t / kTok; d < D; d += kT / kTok) {
    uint8_t* to = v_cache + v_offset(page, h, d, o, Hk, D, shift) * kEl;
    if (F8) *to = vs[e][d];
    else *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(&vs[e][d * 2]);
  }
}

constexpr int kMoves = 64;   // positions whose places are in LDS at once
constexpr int kAhead = 4;    // of them, loaded before the first is stored

// Grid: (R, layers).  One workgroup moves all heads of one request and layer.
template <int EL>
__global__ __launch_bounds__(kT) void kv_commit_kernel(
    uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, int64_t k_layer, int64_t v_layer,
    const int32_t* __restrict__ table, const int32_t* __restrict__ ctx_len,
    const int32_t* __restrict__ mapped_len, const int32_t* __restrict__ path,
    const int32_t* __restrict__ accepted, int max_nodes, int Hk, int D, int shift, int max_pages,
    int num_pages, int32_t* __restrict__ new_len) {
  constexpr int kC = 16 / EL;
  typedef std::conditional_t<EL == 1, uint8_t, uint16_t> V;
  __shared__ int bad, moves;
  // element offsets of head 0, channel 0 of both ends in the two caches
  __shared__ int64_t k_from[kMoves], k_to[kMoves], v_from[kMoves], v_to[kMoves];
  const int t = threadIdx.x;
  const int r = blockIdx.x;
  const int32_t* row = path + (size_t)r * max_nodes;
  const int32_t* pages = table + (size_t)r * max_pages;
  const int64_t ctx = ctx_len[r];
  const int acc = accepted[r];
  // what lies behind the mapped length is not the request's, whatever its row names there
  const int64_t room = min(min((int64_t)max_pages << shift, kMaxLen),
                           mapped_len ? (int64_t)mapped_len[r] : kMaxLen);
  if (t == 0) bad = moves = 0;
  __syncthreads();
  const bool range = ctx >= 0 && acc >= -1 && acc < max_nodes && ctx + 1 + acc <= room;
  if (!range) {
    if (t == 0) bad = 1;
  } else {
    for (int i = t; i <= acc; i += kT) {
      bool fine = path_step_ok(row, i) && ctx + row[i] < room;
      if (fine && i > 0)
        fine = page_ok(pages[(ctx + row[i]) >> shift], num_pages) &&
               page_ok(pages[(ctx + i) >> shift], num_pages);
      if (!fine) atomicOr(&bad, 1);
      if (row[i] != i) atomicOr(&moves, 1);
    }
  }
  __syncthreads();
  const bool skip = bad != 0;
  if (blockIdx.y == 0 && t == 0)
    new_len[r] = !skip ? (int32_t)(ctx + 1 + acc) : mapped_len ? (int32_t)ctx : -1;
  if (skip || !moves) return;   // a chain's path is where it belongs
  uint8_t* kc = k_cache + (int64_t)blockIdx.y * k_layer * EL;
  V* vc = reinterpret_cast<V*>(v_cache + (int64_t)blockIdx.y * v_layer * EL);
  const int m = (1 << shift) - 1;
  const int k_pieces = Hk * (D / kC);
  for (int i0 = 1; i0 <= acc; i0 += kMoves) {
    const int n = min(kMoves, acc - i0 + 1);
    __syncthreads();
    if (t < n) {
      const int64_t from = ctx + row[i0 + t], to = ctx + i0 + t;
      const int64_t fp = pages[from >> shift], tp = pages[to >> shift];
      k_from[t] = k_offset(fp, 0, 0, (int)(from & m), Hk, D, shift, kC);
      k_to[t] = k_offset(tp, 0, 0, (int)(to & m), Hk, D, shift, kC);
      v_from[t] = v_offset(fp, 0, 0, (int)(from & m), Hk, D, shift);
      v_to[t] = v_offset(tp, 0, 0, (int)(to & m), Hk, D, shift);
    }
    __syncthreads();
    // pieces of one head follow each other at a page's distance, and so do the heads
    for (int w = t; w < k_pieces; w += kT) {
      const int64_t at = ((int64_t)w << shift) * kC;
      for (int i = 0; i < n; i += kAhead) {
        u32x4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          x[u] = *reinterpret_cast<const u32x4*>(kc + (k_from[min(i + u, n - 1)] + at) * EL);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (i + u < n) *reinterpret_cast<u32x4*>(kc + (k_to[i + u] + at) * EL) = x[u];
      }
    }
    for (int w = t; w < Hk * D; w += 2 * kT) {
      const int64_t a0 = (int64_t)w << shift;
      const bool two = w + kT < Hk * D;
      const int64_t a1 = two ? (int64_t)(w + kT) << shift : a0;
      for (int i = 0; i < n; i += kAhead) {
        V x[kAhead], y[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int64_t f = v_from[min(i + u, n - 1)];
          x[u] = vc[f + a0];
          y[u] = vc[f + a1];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (i + u < n) {
            vc[v_to[i + u] + a0] = x[u];
            if (two) vc[v_to[i + u] + a1] = y[u];
          }
        }
      }
    }
  }
}

struct StoreArgs {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, v_stride;
  int bf;
  const int64_t* slots;
  const int32_t* count;
  int n, Hk, shift, num_pages;
  const float* k_scale;
  const float* v_scale;
  uint8_t* k_cache;
  uint8_t* v_cache;
};

template <int D, int kTok>
void store_tiles(bool f8, const StoreArgs& a, hipStream_t stream) {
  auto kernel = f8 ? &kv_store_kernel<D, true, kTok> : &kv_store_kernel<D, false, kTok>;
  const dim3 grid((unsigned)(((int64_t)a.n + kTok - 1) / kTok), (unsigned)a.Hk);
  hipLaunchKernelGGL(kernel, grid, dim3(kT), 0, stream, a.k, a.v, a.k_stride, a.v_stride, a.bf,
                     a.slots, a.count, a.n, a.Hk, a.shift, a.num_pages, a.k_scale, a.v_scale,
                     a.k_cache, a.v_cache);
}
template <int D>
void store_d(bool f8, const StoreArgs& a, hipStream_t stream) {
  if ((int64_t)a.n * a.Hk >= kManyRows) store_tiles<D, 64>(f8, a, stream);
  else store_tiles<D, 32>(f8, a, stream);
}

}  // namespace

dspark_status launch_kv_store(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                              int dtype, const int64_t* slots, const int32_t* count,
                              int max_tokens, int Hk, int D, int shift, int num_pages,
                              int cache_dtype, const float* k_scale, const float* v_scale,
                              void* k_cache, void* v_cache, hipStream_t stream) {
  const bool f8 = cache_dtype == DSPARK_E4M3;
  const StoreArgs a = {static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride,
                       v_stride, dtype == DSPARK_BF16, slots, count, max_tokens, Hk, shift,
                       num_pages, k_scale, v_scale, static_cast<uint8_t*>(k_cache),
                       static_cast<uint8_t*>(v_cache)};
  switch (D) {
    case 64: store_d<64>(f8, a, stream); break;
    case 96: store_d<96>(f8, a, stream); break;
    case 128: store_d<128>(f8, a, stream); break;
    case 192: store_d<192>(f8, a, stream); break;
    default: store_d<256>(f8, a, stream); break;
  }
  return check_launch("kv_store_kernel");
}

dspark_status launch_kv_commit(void* k_cache, void* v_cache, int64_t k_layer_stride,
                               int64_t v_layer_stride, int layers, int bytes_per_element,
                               const int32_t* block_table, const int32_t* ctx_len,
                               const int32_t* mapped_len, const int32_t* path,
                               const int32_t* accepted, int R, int max_nodes, int Hk, int D,
                               int shift, int max_pages, int num_pages, int32_t* new_len,
                               hipStream_t stream) {
  const dim3 grid((unsigned)R, (unsigned)layers);
  auto kernel = bytes_per_element == 1 ? &kv_commit_kernel<1> : &kv_commit_kernel<2>;
  hipLaunchKernelGGL(kernel, grid, dim3(kT), 0, stream, static_cast<uint8_t*>(k_cache),
                     static_cast<uint8_t*>(v_cache), k_layer_stride, v_layer_stride, block_table,
                     ctx_len, mapped_len, path, accepted, max_nodes, Hk, D, shift, max_pages,
                     num_pages, new_len);
  return check_launch("kv_commit_kernel");
}

}  // namespace dspark
