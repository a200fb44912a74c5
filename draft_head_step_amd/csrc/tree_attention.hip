// Tree attention over a paged cache: launch plan and dispatch by type.  The
// kernels are in tree_attention_kernels.h.
#include "tree_attention_kernels.h"

namespace dspark {

// The element and cache types are compiled in files of their own.
extern template dspark_status run_tree_attention<0, false>(const TreeAttnArgs&, const AttnPlan&, hipStream_t);
extern template dspark_status run_tree_attention<0, true>(const TreeAttnArgs&, const AttnPlan&, hipStream_t);
extern template dspark_status run_tree_attention<1, false>(const TreeAttnArgs&, const AttnPlan&, hipStream_t);
extern template dspark_status run_tree_attention<1, true>(const TreeAttnArgs&, const AttnPlan&, hipStream_t);

namespace {

int compute_units() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) {
    (void)hipGetLastError();
    return 256;
  }
  return n;
}

}  // namespace

// `capacity`: the most positions a request can have (0: not known yet).
AttnPlan plan_tree_attention(int R, int max_tokens, int Hq, int Hk, int D, int64_t capacity) {
  AttnPlan p;
  const int group = Hq / Hk;
  // Rows that a request is likely to bring.  With one 16-row tile a wave more waves
  // fit a CU; with more than two tiles the products weigh as much as the loads.  Any
  // variant runs any number of rows.
  const int64_t rows = (int64_t)((max_tokens + (int64_t)R - 1) / R) * group;
  p.nt = rows <= 8 ? 1 : 2;
  p.ring = rows > (D <= 128 ? 32 : 8);
  const int waves = attn_group(D, p.ring);
  const int per_cu = attn_waves(p.nt, D, p.ring) * 4 / waves;   // four SIMDs
  int64_t groups = (int64_t)compute_units() * per_cu;
  // A tile of up to 512 positions is not cut, and the second launch is left out.  Whole
  // and cut, in us, tables of 512 positions, 32 heads over 8 of 128:
  //   requests x elements   1 x 6  8 x 6  64 x 6  256 x 6  1 x 64  1 x 300  8 x 64  64 x 64
  //   whole                  12.2   14.5    32.3    110.2    32.9     39.9    34.8     72.4
  //   cut                    15.0   20.7    35.0    112.6    29.9     30.2    33.8     74.9
  // (four waves over positions take 512 in four steps each; where all waves are over rows
  // they take 16, and one request of many rows loses: 1 x 64 over 164 positions 20.9 and
  // 24.9 again).  The rule goes by the table's width, all that the host knows: one token
  // over 200 positions takes 11.9 us with a table of 512 positions, 14.9 with a wider one.
  p.whole = capacity > 0 && capacity <= 512;
  if (capacity > 0) {
    // no more workgroups than units of work there can be
    const int64_t tiles = ((int64_t)max_tokens * group + 16 * p.nt - 1) / (16 * p.nt) + R;
    const int64_t units = tiles * Hk * (p.whole ? 1 : (capacity + 31) / 32);
    if (units < groups) groups = units;
  }
  p.groups = (int)(groups < 1 ? 1 : groups);
  const int64_t blocks = ((int64_t)max_tokens * group + 15) / 16;
  p.row_blocks = (int)(blocks < waves * p.nt ? blocks : waves * p.nt);
  // Eight workgroups for each tile that there is at least: its parts are joined by two
  // waves (one request of 64 nodes over 8000 positions: 58 us, then 41; with four parts
  // a tile, 16 chains, 45 and 46).
  const int64_t row_tiles = blocks / (waves * p.nt);
  p.deep = groups >= 8 * Hk * (row_tiles > R ? row_tiles : (int64_t)R);
  const size_t parts = (size_t)groups * 2 * waves * p.nt;
  p.cut_bytes = ((size_t)groups * sizeof(AttnCut) + 255) / 256 * 256;
  p.ml_bytes = parts * 2 * 64 * sizeof(float);
  p.o_bytes = parts * 16 * (size_t)D * sizeof(float);
  return p;
}

size_t tree_attention_workspace_bytes(int R, int max_tokens, int Hq, int Hk, int D) {
  const AttnPlan p = plan_tree_attention(R, max_tokens, Hq, Hk, D, 0);
  return p.cut_bytes + p.ml_bytes + p.o_bytes;
}

dspark_status launch_tree_attention(const TreeAttnArgs& a, hipStream_t stream) {
  const AttnPlan p = plan_tree_attention(a.R, a.max_tokens, a.Hq, a.Hk, a.D,
                                         (int64_t)a.max_pages << a.shift);
  if (a.cache_dtype == DSPARK_E4M3)
    return a.dtype == DSPARK_BF16 ? run_tree_attention<0, true>(a, p, stream)
                                  : run_tree_attention<1, true>(a, p, stream);
  return a.dtype == DSPARK_BF16 ? run_tree_attention<0, false>(a, p, stream)
                                : run_tree_attention<1, false>(a, p, stream);
}

}  // namespace dspark
