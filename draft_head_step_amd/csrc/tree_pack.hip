// Ancestor masks and positions of drafted trees for CDNA4 (gfx950).
//
// mask(i) = mask(parent(i)) | bit i.  One workgroup per request: the parents of
// up to 1024 nodes go to LDS, then each thread walks its node's chain there.  A
// parent's number is smaller than its child's, so a walk meets the bits from
// the highest word down and a row is written word by word with no array of
// words in registers.  Bound by the length of the longest chain (about 64
// cycles of LDS latency a step): 2.3 us for 4 small trees, 3 to 4.6 for 32 trees of
// up to 64 nodes.
#include "dspark_internal.h"
#include "paged.h"

namespace dspark {
namespace {

constexpr int kT = 256;
constexpr int kMaxNodes = DSPARK_MAX_MASK_WORDS * 32;

__global__ __launch_bounds__(kT) void tree_pack_kernel(
    const int32_t* __restrict__ parents, const int32_t* __restrict__ cu,
    const int32_t* __restrict__ pos0, int max_tokens, int words, uint32_t* __restrict__ mask,
    int32_t* __restrict__ flat_pos, int32_t* __restrict__ flat_req) {
  __shared__ int32_t up[kMaxNodes];
  const int r = blockIdx.x;
  const int64_t s = cu[r];
  const int64_t end = min((int64_t)cu[r + 1], (int64_t)max_tokens);
  if (s < 0 || end <= s) return;
  const int64_t n = end - s;
  const int nodes = (int)(n < words * 32 ? n : words * 32);
  for (int i = threadIdx.x; i < nodes; i += kT) up[i] = parents[s + i];
  __syncthreads();
  const int32_t p0 = pos0 ? pos0[r] : 0;
  for (int64_t i = threadIdx.x; i < n; i += kT) {
    uint32_t* row = mask + (size_t)(s + i) * words;
    int w = words - 1;
    int depth = -1;
    bool good = i < nodes;
    if (good) {
      uint32_t bits = 0;
      for (int a = (int)i; a >= 0;) {
        for (; w > (a >> 5); --w) {
          row[w] = bits;
          bits = 0;
        }
        bits |= 1u << (a & 31);
        ++depth;
        const int32_t p = up[a];
        if (!parent_ok(p, a)) {
          good = false;
          break;
        }
        a = p;
      }
      for (; w >= 0; --w) {
        row[w] = bits;
        bits = 0;
      }
    }
    if (!good)
      for (w = 0; w < words; ++w) row[w] = 0;
    if (flat_pos) flat_pos[s + i] = good ? p0 + depth : -1;
    if (flat_req) flat_req[s + i] = r;
  }
}

}  // namespace

dspark_status launch_tree_pack(const int32_t* parents, const int32_t* cu, const int32_t* pos0,
                               int R, int max_tokens, int mask_words, uint32_t* mask,
                               int32_t* flat_pos, int32_t* flat_req, hipStream_t stream) {
  hipLaunchKernelGGL(tree_pack_kernel, dim3(R), dim3(kT), 0, stream, parents, cu, pos0, max_tokens,
                     mask_words, mask, flat_pos, flat_req);
  return check_launch("tree_pack_kernel");
}

}  // namespace dspark
