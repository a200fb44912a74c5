// Attention of drafted elements over a paged cache for CDNA4 (gfx950).
//
// out = sum_t p_t v_t / sum_t p_t with p_t = 2^(x_t - m), x_t = scale log2(e)
// q . k_t, m the running maximum: one pass over the cache with the sums
// rescaled when m grows.
//
// One wave per (element, query head): a lane scores one position of a tile of
// 64, the wave updates (m, l), then each lane accumulates D / 64 channels.
#include <math.h>

#include "dspark_internal.h"
#include "paged.h"

namespace dspark {
namespace {

constexpr int kT = 64;
constexpr int kMaxD = 256;

__device__ __forceinline__ float load_el(const void* p, int64_t i, int type) {
  if (type == DSPARK_BF16)
    return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  if (type == DSPARK_FP16) return (float)static_cast<const _Float16*>(p)[i];
  return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(p)[i], 0);
}
__device__ __forceinline__ void store_el(void* p, int64_t i, int type, float x) {
  if (type == DSPARK_BF16) static_cast<__bf16*>(p)[i] = (__bf16)x;
  else static_cast<_Float16*>(p)[i] = (_Float16)x;
}

__global__ __launch_bounds__(kT) void tree_attention_simple_kernel(TreeAttnArgs a) {
  __shared__ float q[kMaxD];
  __shared__ float p[kT];
  __shared__ int32_t pg[kT];
  const int lane = threadIdx.x;
  const int e = blockIdx.x / a.Hq;
  const int y = blockIdx.x - e * a.Hq;
  if (e >= a.cu[a.R]) return;
  // request of e: last r with cu[r] <= e
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= e) lo = mid; else hi = mid;
  }
  const int r = lo;
  const int i = e - a.cu[r];
  const int n = a.cu[r + 1] - a.cu[r];
  if (i < 0 || i >= n) return;
  const int h = y / (a.Hq / a.Hk);
  const int64_t ctx = a.ctx[r];
  const int64_t total = ctx + n;
  bool bad = ctx < 0 || pages_of(total, a.shift) > a.max_pages;
  const int c = a.cache_dtype == DSPARK_E4M3 ? 16 : 8;
  const float ks = a.k_scale ? a.k_scale[h] : 1.0f;
  const float vs = a.v_scale ? a.v_scale[h] : 1.0f;
  for (int d = lane; d < a.D; d += kT)
    q[d] = load_el(a.q, (int64_t)e * a.q_stride + y * a.D + d, a.dtype);
  __syncthreads();
  float m = -INFINITY, l = 0.0f;
  float acc[kMaxD / kT] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t t0 = 0; t0 < total && !bad; t0 += kT) {
    const int64_t t = t0 + lane;
    bool seen = t < total;
    int32_t page = 0;
    if (seen) {
      page = a.table[(int64_t)r * a.max_pages + (t >> a.shift)];
      if (!page_ok(page, a.num_pages)) {
        bad = true;
        page = 0;
      }
      if (t >= ctx) {
        const int j = (int)(t - ctx);
        seen = a.mask ? (j >> 5) < a.mask_words &&
                            ((a.mask[(int64_t)e * a.mask_words + (j >> 5)] >> (j & 31)) & 1u)
                      : j <= i;
      }
    }
    bad = __any(bad);
    if (bad) break;
    const int o = (int)(t & ((1 << a.shift) - 1));
    float x = -INFINITY;
    if (seen) {
      float s = 0.0f;
      for (int d = 0; d < a.D; ++d)
        s = fmaf(q[d], load_el(a.k_cache, k_offset(page, h, d, o, a.Hk, a.D, a.shift, c), a.cache_dtype), s);
      x = s * (a.scale2 * ks);
    }
    float top = x;
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    const float nm = fmaxf(m, top);
    const float base = nm == -INFINITY ? 0.0f : nm;
    const float keep = __builtin_amdgcn_exp2f(m - base);
    const float w = seen ? __builtin_amdgcn_exp2f(x - base) : 0.0f;
    float sum = w;
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
    l = l * keep + sum;
    m = nm;
    __syncthreads();
    p[lane] = w;
    pg[lane] = seen ? page : -1;
    __syncthreads();
    for (int u = 0; u < kMaxD / kT; ++u) {
      const int d = lane + u * kT;
      if (d >= a.D) break;
      acc[u] *= keep;
      for (int s = 0; s < kT; ++s)
        if (pg[s] >= 0)
          acc[u] = fmaf(p[s], load_el(a.v_cache, v_offset(pg[s], h, d, (int)((t0 + s) & ((1 << a.shift) - 1)), a.Hk, a.D, a.shift), a.cache_dtype), acc[u]);
    }
  }
  for (int u = 0; u < kMaxD / kT; ++u) {
    const int d = lane + u * kT;
    if (d >= a.D) break;
    const float x = bad ? NAN : m == -INFINITY ? 0.0f : acc[u] * vs / l;
    store_el(a.out, (int64_t)e * a.out_stride + y * a.D + d, a.dtype, x);
  }
  if (a.lse && lane == 0)
    a.lse[(int64_t)e * a.Hq + y] =
        bad ? NAN : m == -INFINITY ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t tree_attention_workspace_bytes(int R, int max_tokens, int Hq, int Hk, int D) { return 256; }

dspark_status launch_tree_attention(const TreeAttnArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(tree_attention_simple_kernel, dim3((unsigned)(a.max_tokens * a.Hq)), dim3(kT),
                     0, stream, a);
  return check_launch("tree_attention_simple_kernel");
}

}  // namespace dspark
