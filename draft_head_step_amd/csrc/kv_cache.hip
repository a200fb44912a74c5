// Writes to the paged key/value cache for CDNA4 (gfx950).
//
//   kv_store:  K and V rows of new elements into their slots.  The keys keep 16
//              bytes (c elements) of a row together, [D / c][P][c]; the values
//              lie transposed, [D][P].  A workgroup takes 16 elements of one
//              head: rows are read 16 bytes a lane, pass through LDS, and are
//              written with neighbouring lanes on neighbouring elements, which
//              in a run of slots are neighbouring addresses in both caches.
//   kv_commit: the accepted path's keys and values to the front.  A thread
//              owns one 16-byte piece of the keys or one value channel and moves
//              it for i = 1, 2, ... in turn.  path[i] >= i and path increases,
//              so position i, once written, is no later source.
#include "dspark_internal.h"
#include "paged.h"

namespace dspark {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kT = 256;
constexpr int kTok = 16;   // elements per workgroup

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

// Grid: (ceil(max_tokens / kTok), Hk).  F8: 8-bit cache of 16-bit inputs.
template <int D, bool F8>
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
  const float sk = F8 ? k_scale[h] : 1.0f;
  const float sv = F8 ? v_scale[h] : 1.0f;
  constexpr int kPieces = D / 8;   // 16-byte pieces of an input row
  for (int i = t; i < (int)n * kPieces; i += kT) {
    const int e = i / kPieces, p = i - e * kPieces;
    const u32x4 a = *reinterpret_cast<const u32x4*>(k + (e0 + e) * k_stride + h * D + p * 8);
    const u32x4 b = *reinterpret_cast<const u32x4*>(v + (e0 + e) * v_stride + h * D + p * 8);
    if (F8) {
      uint8_t oa[8], ob[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        oa[j] = to_e4m3(widen((uint16_t)(a[j >> 1] >> ((j & 1) * 16)), bf) / sk);
        ob[j] = to_e4m3(widen((uint16_t)(b[j >> 1] >> ((j & 1) * 16)), bf) / sv);
      }
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
    *reinterpret_cast<u32x4*>(k_cache + k_offset(page, h, p * kC, o, Hk, D, shift, kC) * kEl) =
        *reinterpret_cast<const u32x4*>(&ks[e][p * 16]);
  for (int d = t / kTok; d < D; d += kT / kTok) {
    uint8_t* to = v_cache + v_offset(page, h, d, o, Hk, D, shift) * kEl;
    if (F8) *to = vs[e][d];
    else *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(&vs[e][d * 2]);
  }
}

// Grid: (R, layers).  One workgroup moves all heads of one request and layer.
template <int EL>
__global__ __launch_bounds__(kT) void kv_commit_kernel(
    uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, int64_t k_layer, int64_t v_layer,
    const int32_t* __restrict__ table, const int32_t* __restrict__ ctx_len,
    const int32_t* __restrict__ path, const int32_t* __restrict__ accepted, int max_nodes, int Hk,
    int D, int shift, int max_pages, int num_pages, int32_t* __restrict__ new_len) {
  constexpr int kC = 16 / EL;
  __shared__ int bad;
  const int t = threadIdx.x;
  const int r = blockIdx.x;
  const int32_t* row = path + (size_t)r * max_nodes;
  const int32_t* pages = table + (size_t)r * max_pages;
  const int64_t ctx = ctx_len[r];
  const int acc = accepted[r];
  const int64_t room = (int64_t)max_pages << shift;
  if (t == 0) bad = 0;
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
    }
  }
  __syncthreads();
  const bool skip = bad != 0;
  if (blockIdx.y == 0 && t == 0) new_len[r] = skip ? -1 : (int32_t)(ctx + 1 + acc);
  if (skip) return;
  uint8_t* kc = k_cache + (int64_t)blockIdx.y * k_layer * EL;
  uint8_t* vc = v_cache + (int64_t)blockIdx.y * v_layer * EL;
  const int pieces = Hk * (D / kC);
  const int m = (1 << shift) - 1;
  for (int w = t; w < pieces + Hk * D; w += kT) {
    const bool key = w < pieces;
    const int h = key ? w / (D / kC) : (w - pieces) / D;
    const int d = key ? (w - h * (D / kC)) * kC : (w - pieces) - h * D;
    for (int i = 1; i <= acc; ++i) {
      const int64_t from = ctx + row[i], to = ctx + i;
      if (from == to) continue;
      const int64_t fp = pages[from >> shift], tp = pages[to >> shift];
      const int fo = (int)(from & m), to_ = (int)(to & m);
      if (key) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(kc + k_offset(fp, h, d, fo, Hk, D, shift, kC) * EL);
        *reinterpret_cast<u32x4*>(kc + k_offset(tp, h, d, to_, Hk, D, shift, kC) * EL) = x;
      } else if (EL == 1) {
        vc[v_offset(tp, h, d, to_, Hk, D, shift)] = vc[v_offset(fp, h, d, fo, Hk, D, shift)];
      } else {
        uint16_t* vw = reinterpret_cast<uint16_t*>(vc);
        vw[v_offset(tp, h, d, to_, Hk, D, shift)] = vw[v_offset(fp, h, d, fo, Hk, D, shift)];
      }
    }
  }
}

template <int D>
void store_d(bool f8, dim3 grid, hipStream_t stream, const uint16_t* k, const uint16_t* v,
             int64_t ks, int64_t vs, int bf, const int64_t* slots, const int32_t* count, int n,
             int Hk, int shift, int num_pages, const float* k_scale, const float* v_scale,
             uint8_t* kc, uint8_t* vc) {
  if (f8)
    hipLaunchKernelGGL((kv_store_kernel<D, true>), grid, dim3(kT), 0, stream, k, v, ks, vs, bf,
                       slots, count, n, Hk, shift, num_pages, k_scale, v_scale, kc, vc);
  else
    hipLaunchKernelGGL((kv_store_kernel<D, false>), grid, dim3(kT), 0, stream, k, v, ks, vs, bf,
                       slots, count, n, Hk, shift, num_pages, k_scale, v_scale, kc, vc);
}

}  // namespace

dspark_status launch_kv_store(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                              int dtype, const int64_t* slots, const int32_t* count,
                              int max_tokens, int Hk, int D, int shift, int num_pages,
                              int cache_dtype, const float* k_scale, const float* v_scale,
                              void* k_cache, void* v_cache, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)max_tokens + kTok - 1) / kTok), (unsigned)Hk);
  const bool f8 = cache_dtype == DSPARK_E4M3;
  auto go = [&](auto store) {
    store(f8, grid, stream, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
          k_stride, v_stride, dtype == DSPARK_BF16, slots, count, max_tokens, Hk, shift, num_pages,
          k_scale, v_scale, static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache));
  };
  switch (D) {
    case 64: go(&store_d<64>); break;
    case 96: go(&store_d<96>); break;
    case 128: go(&store_d<128>); break;
    case 192: go(&store_d<192>); break;
    default: go(&store_d<256>); break;
  }
  return check_launch("kv_store_kernel");
}

dspark_status launch_kv_commit(void* k_cache, void* v_cache, int64_t k_layer_stride,
                               int64_t v_layer_stride, int layers, int bytes_per_element,
                               const int32_t* block_table, const int32_t* ctx_len,
                               const int32_t* path, const int32_t* accepted, int R, int max_nodes,
                               int Hk, int D, int shift, int max_pages, int num_pages,
                               int32_t* new_len, hipStream_t stream) {
  const dim3 grid((unsigned)R, (unsigned)layers);
  auto kernel = bytes_per_element == 1 ? &kv_commit_kernel<1> : &kv_commit_kernel<2>;
  hipLaunchKernelGGL(kernel, grid, dim3(kT), 0, stream, static_cast<uint8_t*>(k_cache),
                     static_cast<uint8_t*>(v_cache), k_layer_stride, v_layer_stride, block_table,
                     ctx_len, path, accepted, max_nodes, Hk, D, shift, max_pages, num_pages,
                     new_len);
  return check_launch("kv_commit_kernel");
}

}  // namespace dspark
