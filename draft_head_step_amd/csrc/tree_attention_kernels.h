// Kernels of the attention of drafted elements over a paged cache (gfx950).
//
// With x_t = scale log2(e) k_scale q . k_t and m >= max x_t - kSlack a running
// reference, a row keeps l = sum 2^(x_t - m) and O = sum 2^(x_t - m) v_t: one
// pass over the cache, rescaled when a new maximum leaves m more than kSlack
// behind (so that most steps rescale nothing; the exponent range of fp32 sums and
// of both 16-bit types holds 2^kSlack).
//
// Both products run on the matrix cores transposed, S^T = K Q^T and O^T = V^T P^T:
// a step's positions are the rows of the first result and the contraction of
// the second, and a query row is a matrix column, so a lane holds one row's
// scores, its maximum and its rescale factor.  The caches are stored in operand
// order, so keys and values go from memory to registers to the matrix cores, 16
// bytes a lane, with no LDS on the way.
//
// A step is kTok = 4 c positions, c = 16 / element size.  Key tile kt is the
// positions 16 kt .. 16 kt + 15, so that one load instruction of the wave takes
// whole runs of 256 bytes (with pieces of 64 bytes and non-temporal loads the
// same kernel read 5.6 TB/s instead of 6.9).  Lane group g = lane / 16 then holds
// the scores of positions 16 kt + 4 g + i, and its 16 bytes of a value channel
// are positions c g .. c g + c - 1: the packed probabilities go there by a
// transposition of groups and tiles, two lane swaps a register pair.
//
// Work is split by length, not by request: the row tiles of all requests and
// heads are laid end to end in units of (waves over positions) * kTok positions,
// and each workgroup takes an equal run of units, whatever requests it
// crosses.  A tile cut by a run's end goes to the workspace in parts (fp32), and
// a second launch joins them.  Each workgroup finds its place by scanning the
// lengths itself.  A tile counts for kTileCost positions more than it has: the
// queries, the first loads and the last sums of a tile take about as long as
// reading those (without it the run with the most short requests ended last:
// 64 chains over 37 to 8100 positions took 222 us, then 201).  Where the table has
// room for few positions a tile is one unit, nothing is cut, and the second launch
// is left out.
//
// A workgroup's waves (four or eight) share a tile of 16 NT WR rows: WR waves over
// rows, the others over positions (interleaved steps).  A request's rows are cut
// into tiles with all waves over rows and a last one whose WR goes by what is left,
// so that a chain of a few drafts spreads over positions and a wide tree reads its
// cache once.
//
// Pages of at least a step's positions are the same for a whole wave: their
// addresses are scalars (kPage = 0).  Smaller ones differ between lane groups:
// there the page size is a constant, and so are the distances between a
// lane's loads (kPage = log2 of the page size).
//
// Measured, 32 query heads over 8 of 128 (both launches, idle gaps left out):
//   64 chains of 1 to 6 over 37 to 8100 positions, bf16: 202 us for 1.07 GB, 5.3
//     TB/s.  Bound by the loads in flight; a plain read reaches 6.9.
//   6 trees of 5 to 16 over 30 to 131 thousand positions, e4m3: 202 us for 1.03 GB,
//     5.1 TB/s, with the widening of 8-bit operands beside it.
//   24 trees of 33 to 64 over 1 to 6 thousand positions, 64 heads, fp16: 229 us for
//     126 GFLOP, 545 to 550 TFLOP/s.  A step in the middle of a tile runs at 870 (a large
//     product at 1170), between the matrix cores and the exponentials; the rest is
//     each tile's start and end, and the parts (64 MB out and in, 18 us to join).
//   One token over 200 positions (16 heads over 2 of 64, a table of up to 512
//     positions): 7.2 us, the latency of dependent loads.
//   6 tokens over 8000 positions: 27 us, over 130 thousand 111 us (4.8 TB/s).
//   The same 64 chains in e4m3: 133 us, 4.0 TB/s (some registers spill for a tile's start
//     and end and for masked steps); in bf16 with heads of 192 and 256 295 us and 385,
//     5.5 TB/s.
//   Pieces of 100 to 700 elements behind up to 4000 positions, 6 requests, bf16: 183 us
//     for 101 GFLOP, 550 TFLOP/s; 512 elements behind 16 thousand, 2 requests: 835.
#pragma once

#include <math.h>

#include <type_traits>

#include "dspark_internal.h"
#include "paged.h"

namespace dspark {

// A tile that a workgroup's run ends in: its parts are slot 2 * b + 1 of this
// workgroup b and slots 2 * (b + 1), 2 * (b + 2), ... of the next ones.
struct AttnCut {
  int32_t parts;                   // 0: none
  int32_t start, rows, row0, h;    // the request's first element and rows, the tile's first row
  int32_t pad;
};

struct AttnPlan {
  int groups;       // workgroups
  int nt;           // 16-row tiles per wave
  bool ring;        // waves share keys and values through LDS
  int row_blocks;   // 16-row blocks of a part that may hold rows
  bool whole;       // tiles are not cut
  bool deep;        // a tile is likely to have many parts: two waves share a join
  size_t cut_bytes, ml_bytes, o_bytes;   // workspace: AttnCut[groups], (m, l), O
};
AttnPlan plan_tree_attention(int R, int max_tokens, int Hq, int Hk, int D, int64_t capacity);

template <int DT, bool F8>
dspark_status run_tree_attention(const TreeAttnArgs& a, const AttnPlan& p, hipStream_t stream);

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Waves of a workgroup: eight where they share a ring (a tile of 256 rows reads the
// cache half as often as one of 128), four otherwise and for wide heads.
constexpr int attn_group(int d, bool ring) { return ring && d <= 128 ? 8 : 4; }
constexpr int kJoinWaves = 4;              // of the second launch
constexpr int kJoinThreads = 64 * kJoinWaves;
constexpr float kSlack = 8.0f;
constexpr int kTileCost = 256;

// Operands and conversions of an element type (0 bf16, 1 fp16).
template <int DT> struct El;
template <> struct El<0> {
  static constexpr uint32_t kExp = 0x7f80u, kOne = 0x3f80u;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const bf16x2 p = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, p);
  }
  template <bool HI> static __device__ __forceinline__ uint32_t wide(uint32_t x) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, HI));
  }
};
template <> struct El<1> {
  static constexpr uint32_t kExp = 0x7c00u, kOne = 0x3c00u;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const f16x2 p = {(_Float16)x, (_Float16)y};
    return __builtin_bit_cast(uint32_t, p);
  }
  template <bool HI> static __device__ __forceinline__ uint32_t wide(uint32_t x) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, HI));
  }
};

// Half `s` of 16 e4m3 values as 8 elements; exact, both types hold every e4m3 value.
template <int DT> __device__ __forceinline__ u32x4 widen8(u32x4 x, int s) {
  u32x4 r;
  r[0] = El<DT>::template wide<false>(x[2 * s]);
  r[1] = El<DT>::template wide<true>(x[2 * s]);
  r[2] = El<DT>::template wide<false>(x[2 * s + 1]);
  r[3] = El<DT>::template wide<true>(x[2 * s + 1]);
  return r;
}

// Flags of the two halves of a word, in bits 0 and 16: |half| >= limit (a half's
// sign bit is free for the carry).
__device__ __forceinline__ uint32_t halves_from(uint32_t x, uint32_t limit) {
  return (((x & 0x7fff7fffu) + (0x8000u - limit) * 0x00010001u) >> 15) & 0x00010001u;
}
// Flags of the four bytes, in bits 0, 8, 16 and 24: e4m3 NaN.
__device__ __forceinline__ uint32_t bytes_nan(uint32_t x) {
  return (((x & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u;
}
// Bit i of `bits` as a whole word of ones or zeros.
__device__ __forceinline__ uint32_t spread(uint32_t bits, int i) {
  return (uint32_t)((int32_t)(bits << (31 - i)) >> 31);
}

// Words of the (lane group, tile) matrix to its transpose: x[i] of group g becomes
// x[g] of group i for four tiles; for two, group g gets the halves of tile g / 2
// that groups 2 (g % 2) and 2 (g % 2) + 1 held.
__device__ __forceinline__ void swap32(uint32_t& x, uint32_t& y) {
  const auto s = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  x = s[0];
  y = s[1];
}
__device__ __forceinline__ void swap16(uint32_t& x, uint32_t& y) {
  const auto s = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  x = s[0];
  y = s[1];
}
__device__ __forceinline__ void regroup(uint32_t (&x)[2]) {
  swap32(x[0], x[1]);
  swap16(x[0], x[1]);
}
__device__ __forceinline__ void regroup(uint32_t (&x)[4]) {
  swap32(x[0], x[2]);
  swap32(x[1], x[3]);
  swap16(x[0], x[1]);
  swap16(x[2], x[3]);
}

__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }

// A bit cast of a vector's element reads element 0: elements are copied first.
__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t as_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

// 64 pieces of 16 bytes (one a lane) from memory to 1 KB of LDS at a wave-uniform
// address, lane after lane, without passing registers.  In assembly, so that the
// compiler does not wait for it before the next read of LDS; wait_loads does.
__device__ __forceinline__ void copy_to_lds(const uint8_t* from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(from), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// Until at most N (<= 63) loads of this wave are outstanding; they land in order, so
// loads that the compiler adds only make the wait longer.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N <= 63, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0f70);
  asm volatile("" ::: "memory");
}
// A barrier that waits for nothing but this wave's reads of LDS: what they read may be
// overwritten behind it.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Over the four lane groups (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float groups_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(as_bits(x), as_bits(x), false, false);
  x = fmaxf(as_float(a[0]), as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(as_bits(x), as_bits(x), false, false);
  return fmaxf(as_float(b[0]), as_float(b[1]));
}
__device__ __forceinline__ float groups_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The run of workgroup i of G: neighbouring runs on one XCD (workgroups go to the
// eight XCDs in turn).
__device__ __forceinline__ int run_of(int i, int G) {
  return (G & 7) == 0 ? (i & 7) * (G >> 3) + (i >> 3) : i;
}

// A request as the work split sees it.
struct Req {
  int start;        // its first element
  int n;            // elements that are visible to each other
  int rows;         // query rows to compute (elements within max_tokens, times heads a group)
  int ctx, total;   // positions before the segment, and with it
  int full;         // row tiles with all waves over rows
  int wr_last;      // waves over rows of the last one, 0 if there is none
  int units_full, units_last;   // units of a tile
  bool bad;
  __device__ __forceinline__ int64_t head_units() const {
    return (int64_t)full * units_full + units_last;
  }
};
// kTileCost in units of `unit` positions, at least one.
__device__ __forceinline__ int tile_cost(int unit) {
  return unit < kTileCost ? kTileCost / unit : 1;
}
template <int NT, int TOK, int WAVES, bool RING>
__device__ __forceinline__ Req request(const TreeAttnArgs& a, int r, int group, bool whole) {
  Req q;
  const int64_t s = a.cu[r], e = a.cu[r + 1];
  const int64_t n = s < 0 || e < s ? 0 : e - s;
  const int64_t here = n < a.max_tokens - s ? n : a.max_tokens - s;
  const int64_t ctx = a.ctx[r];
  const int64_t total = ctx + n;
  q.start = (int)s;
  q.n = (int)n;
  q.rows = here > 0 ? (int)here * group : 0;
  q.bad = ctx < 0 || total > 0x7fff0000LL || pages_of(total < 0 ? 0 : total, a.shift) > a.max_pages;
  if (a.mapped) q.bad |= total > a.mapped[r];   // what its row names there is not its own
  q.ctx = q.bad ? 0 : (int)ctx;
  q.total = q.bad ? 0 : (int)total;
  constexpr int kTile = 16 * NT * WAVES;
  q.full = q.rows / kTile;
  const int rest = q.rows - q.full * kTile;
  // (a ring needs at least two waves for each copy)
  q.wr_last = rest == 0 ? 0 : !RING && rest <= 16 * NT ? 1 : rest <= 32 * NT ? 2
              : rest <= 64 * NT ? 4 : WAVES;
  // Units of a tile: its cost, then its steps.
  const int steps = q.bad ? 1 : (q.total + TOK - 1) / TOK;
  q.units_full = tile_cost(TOK) + steps;
  const int wt = q.wr_last ? WAVES / q.wr_last : 1;
  q.units_last = q.wr_last ? tile_cost(TOK * wt) + (steps + wt - 1) / wt : 0;
  if (whole) {
    q.units_full = 1;
    q.units_last = q.wr_last ? 1 : 0;
  }
  return q;
}

// Steps of a ring of `slots` for each of `groups` of waves: at most four, so that the
// loads in flight stay countable.
constexpr int ring_steps(int slots, int groups) {
  return slots / groups < 4 ? slots / groups : 4;
}
// Waves of a SIMD that the registers of a tile allow.
constexpr int attn_waves(int nt, int d, bool ring) {
  return ring ? (d <= 128 ? 2 : 1) : nt * d <= 64 ? 4 : nt * d <= 96 ? 3 : nt * d <= 256 && d <= 128 ? 2 : 1;
}

// Launch with kThreads threads; a run of units per workgroup.
template <int DT, bool F8, int D, int NT, int kPage, bool kRing>
__global__ __launch_bounds__(64 * attn_group(D, kRing), attn_waves(NT, D, kRing)) void tree_attention_kernel(
    const TreeAttnArgs a, const bool whole, AttnCut* __restrict__ cuts,
    float* __restrict__ part_ml, float* __restrict__ part_o) {
  constexpr int kWaves = attn_group(D, kRing);
  constexpr int kThreads = 64 * kWaves;
  constexpr int kC = F8 ? 16 : 8;        // positions of a lane's 16 bytes of values
  constexpr int kTok = 4 * kC;           // positions of a step
  constexpr int kKT = kC / 4;            // key tiles of a step
  constexpr int kJ = F8 ? (D + 63) / 64 : D / 32;   // 16-byte key loads a tile
  constexpr int kMj = F8 ? 2 : 1;        // products a key load feeds
  constexpr int kU = kC / 8;             // products a value load feeds
  constexpr int kDT = D / 16;            // output tiles
  constexpr int kEl = F8 ? 1 : 2;
  constexpr int kPieces = D / kC;        // 16-byte pieces of a key row
  using E = El<DT>;
  // Where requests bring many rows the waves share positions (two or four of them)
  // and one copy of keys and values, in a ring of steps in LDS that is loaded up to
  // three steps ahead.  With few rows each wave loads its own positions into
  // registers, and the workgroups of a CU cover each other's waits.
  constexpr int kRingBytes = 128 * 1024;
  constexpr int kKB = kKT * kJ;          // 1 KB blocks of keys and of a step
  constexpr int kBlocks = kKB + kDT;
  constexpr int kSlots = kRingBytes / 1024 / kBlocks;

  constexpr int kBufs = kWaves / 2;      // tiles that wait for their join at once
  constexpr int kJoinBytes = kBufs * NT * kDT * 64 * 16;
  __shared__ __align__(16) uint8_t sh_mem[kRing && kRingBytes > kJoinBytes ? kRingBytes : kJoinBytes];
  f32x4(&sh_o)[kBufs][NT * kDT][64] = *reinterpret_cast<f32x4(*)[kBufs][NT * kDT][64]>(sh_mem);
  __shared__ float sh_ml[kBufs][NT][2][64];
  __shared__ int64_t sh_scan[kWaves];
  __shared__ int64_t sh_pos[2];          // request and unit within it of this run's first unit

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = uni(t >> 6);
  const int col = lane & 15;             // query row within a 16-row tile
  const int g = lane >> 4;               // lane group
  const int group = a.Hq / a.Hk;
  const int G = gridDim.x;
  const int b = run_of(blockIdx.x, G);

  // ---- where this run starts ----
  // With few units only the first workgroups take a run: every run between a tile's
  // first and last part holds a part.  Runs of waves that share a ring have two units
  // at least, their parts are as large as the keys and values of eight (2 trees of 20
  // to 30 over 500 and 2000 positions: 33 us, then 30; four units gain no more).  Other
  // runs may have one: with two, 1 and 6 elements over 8000 positions took 27.5 and
  // 30.6 us instead of 23.6 and 26.6.
  int64_t w, w_end, all, runs;
  {
    const int per = (a.R + kThreads - 1) / kThreads;
    const int r0 = min(t * per, a.R), r1 = min(r0 + per, a.R);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += a.Hk * request<NT, kTok, kWaves, kRing>(a, r, group, whole).head_units();
    int64_t inc = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t o = __shfl_up(inc, off);
      inc += lane >= off ? o : 0;
    }
    if (lane == 63) sh_scan[wave] = inc;
    __syncthreads();
    int64_t pre = 0;
    all = 0;
#pragma unroll
    for (int j = 0; j < kWaves; ++j) {
      pre += j < wave ? sh_scan[j] : 0;
      all += sh_scan[j];
    }
    const int64_t most = kRing && !whole && all > 1 ? all / 2 : all;
    runs = most < G ? most : G;
    w = b < runs ? all * b / runs : 0;
    w_end = b < runs ? all * (b + 1) / runs : 0;
    int64_t first = pre + inc - mine;
    if (w < w_end && w >= first && w < first + mine) {
      for (int r = r0; r < r1; ++r) {
        const int64_t u = a.Hk * request<NT, kTok, kWaves, kRing>(a, r, group, whole).head_units();
        if (w < first + u) {
          sh_pos[0] = r;
          sh_pos[1] = w - first;
          break;
        }
        first += u;
      }
    }
    __syncthreads();
  }
  if (w >= w_end) {
    if (t == 0 && !whole) cuts[b] = AttnCut{0, 0, 0, 0, 0, 0};
    return;
  }
  int r = uni((int)sh_pos[0]);
  AttnCut cut = {0, 0, 0, 0, 0, 0};
  Req rq = request<NT, kTok, kWaves, kRing>(a, r, group, whole);
  // the first tile by division, the others by counting
  int h, row_tile, s0;
  {
    const int64_t at = sh_pos[1], per_head = rq.head_units();
    h = uni((int)(at / per_head));
    const int64_t in_head = at - h * per_head;
    row_tile = uni(in_head < (int64_t)rq.full * rq.units_full ? (int)(in_head / rq.units_full) : rq.full);
    s0 = uni((int)(in_head - (int64_t)row_tile * rq.units_full));
  }

  while (w < w_end) {
    // ---- this segment: units s0 .. s1 of row tile `row_tile` of head h ----
    if (kRing) __syncthreads();            // the ring is free
    const bool full = row_tile < rq.full;
    const int units = uni(full ? rq.units_full : rq.units_last);
    const int wr = uni(full ? kWaves : rq.wr_last);
    const int64_t left = w_end - w;
    const int s1 = uni((int)(left < units - s0 ? s0 + left : units));
    const int wt = kWaves / wr;
    const int my_t = wave / wr, my_r = wave & (wr - 1);
    const int ctx = uni(rq.ctx), total = uni(rq.total);
    const int row0 = row_tile * (16 * NT * kWaves) + my_r * 16 * NT;
    const bool idle = row0 >= rq.rows;

    const float ks = a.k_scale ? a.k_scale[h] : 1.0f;
    float sc = a.scale2 * ks;
    const uint32_t flip = sc < 0.0f ? 0x80008000u : 0u;   // the sign goes to the queries
    sc = fabsf(sc);
    u32x4 qf[NT][kJ * kMj];
    int el[NT];                            // element (within the segment) of this lane's row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + nt * 16 + col;
      const bool in = row < rq.rows;
      el[nt] = in ? row / group : 0;
      const int y = in ? row - el[nt] * group : 0;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q) +
                           (int64_t)(rq.start + el[nt]) * a.q_stride + (h * group + y) * D;
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < kMj; ++i) {
          const int d = F8 ? (j * 4 + g) * 16 + i * 8 : (j * 4 + g) * 8;
          u32x4 x = {0, 0, 0, 0};
          if (in && d < D) x = *reinterpret_cast<const u32x4*>(qp + d);
          qf[nt][j * kMj + i] = x ^ flip;
        }
    }
    // Mask rows of up to 64 nodes are read here: a load among the steps would wait for
    // every copy to LDS before it.
    const bool short_mask = a.mask && a.mask_words <= 2;
    uint64_t mask64[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mask64[nt] = 0;
      if (short_mask) {
        const uint32_t* mw = a.mask + (int64_t)(rq.start + el[nt]) * a.mask_words;
        mask64[nt] = mw[0];
        if (a.mask_words == 2) mask64[nt] |= (uint64_t)mw[1] << 32;
      }
    }
    f32x4 o[NT][kDT];
    float m[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < kDT; ++dt) o[nt][dt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // the last position that a row of this wave sees, plus one
    int seen = total;
    if (!a.mask && !idle)
      seen = min(seen, ctx + (min(rq.rows, row0 + 16 * NT) - 1) / group + 1);
    bool bad = rq.bad;
    const int t_step = kTok * wt;
    const int cost = tile_cost(t_step);
    const int from = whole ? 0 : max(s0 - cost, 0) * wt * kTok;
    const int to = whole ? total : (s1 - cost) * t_step;
    int t0 = uni(from + my_t * kTok);
    const int t_end = uni(idle || bad ? 0 : min(seen, to));
    // the same of the whole tile: waves that share a ring take part to its end
    const int t0_tile = from;
    int seen_tile = total;
    if (!a.mask)
      seen_tile = min(seen_tile, ctx + (min(rq.rows, (row_tile * kWaves + wr) * 16 * NT) - 1) / group + 1);
    const int t_end_tile = uni(bad ? 0 : min(seen_tile, to));

    if (kRing ? t0_tile < t_end_tile : t0 < t_end) {
      const int shift = kPage ? kPage : a.shift;
      const int P = 1 << shift;
      const int last_page = (total - 1) >> shift;
      const int64_t page_bytes = ((int64_t)a.Hk * D << shift) * kEl;
      const uint8_t* kh = static_cast<const uint8_t*>(a.k_cache) + ((int64_t)h * D << shift) * kEl;
      const uint8_t* vh = static_cast<const uint8_t*>(a.v_cache) + ((int64_t)h * D << shift) * kEl;
      const int vb = kC * g;                // this lane's values start there within a step
      const int32_t* pages = a.table + (int64_t)r * a.max_pages;
      u32x4 kf[kKT][kJ], vf[kDT];
      // Pages of the step at tt, scalars; read two steps ahead of their use, keys and
      // values one or more.
      constexpr int kPk = kPage == 0 ? 1 : kTok >> kPage;
      struct Pages {
        uint64_t lo, hi;                   // pages 0 and 1, pages 2 and 3
        __device__ __forceinline__ int64_t at(int i) const {
          // no select between members, which would send them to memory
          const uint64_t two = kPk == 4 ? lo ^ ((lo ^ hi) & (0 - (uint64_t)((i >> 1) & 1))) : lo;
          return (int32_t)(two >> (32 * (i & 1)));
        }
      };
      auto entries = [&](int tt) __attribute__((always_inline)) {
        typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;
        const scalar_ptr row = (scalar_ptr)(uintptr_t)pages;
        const int i = tt >> shift;
        auto one = [&](int k) __attribute__((always_inline)) {
          return (uint64_t)(uint32_t)row[min(i + k, last_page)];
        };
        Pages e = {one(0), 0};
        if constexpr (kPk >= 2) e.lo |= one(1) << 32;
        if constexpr (kPk == 4) e.hi = one(2) | one(3) << 32;
        return e;
      };
      // A page outside the pool is not touched: page 0 stands in, and the rows are NaN.
      auto check = [&](Pages e) __attribute__((always_inline)) {
        auto one = [&](int k) __attribute__((always_inline)) {
          const bool ok = page_ok((int32_t)e.at(k), a.num_pages);
          bad |= !ok;
          return ok ? (uint64_t)(uint32_t)e.at(k) : (uint64_t)0;
        };
        Pages c = {one(0), 0};
        if constexpr (kPk >= 2) c.lo |= one(1) << 32;
        if constexpr (kPk == 4) c.hi = one(2) | one(3) << 32;
        return c;
      };
      // Addresses of this lane's 16 bytes of key block (kt, j) and of value block dt of
      // the step at tt.
      const uint32_t k_lane = (uint32_t)(col * 16 + g * (P * 16));
      auto k_block = [&](const Pages& e, int tt, int kt, int j) __attribute__((always_inline)) {
        const uint8_t* base = kh + e.at(kPage == 0 ? 0 : (16 * kt) >> kPage) * page_bytes +
                              ((tt + 16 * kt) & (P - 1)) * 16 + (int64_t)j * 4 * P * 16;
        // past the last piece: the first ones again, cleared where they are used
        return base + (kPieces % 4 != 0 && j * 4 + g >= kPieces ? (uint32_t)(col * 16) : k_lane);
      };
      auto v_base = [&](const Pages& e, int tt) __attribute__((always_inline)) {
        int64_t at = e.at(0) * page_bytes;
        if constexpr (kPk == 2) at = g & 2 ? e.at(1) * page_bytes : at;
        if constexpr (kPk == 4) {
          const int64_t lo = g & 1 ? e.at(1) * page_bytes : at;
          const int64_t hi = g & 1 ? e.at(3) * page_bytes : e.at(2) * page_bytes;
          at = g & 2 ? hi : lo;
        }
        return vh + at + (uint32_t)((col * P + ((tt + vb) & (P - 1))) * kEl);
      };
      auto k_tail = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
          if (kPieces % 4 != 0 && (kJ - 1) * 4 + g >= kPieces) kf[kt][kJ - 1] = u32x4{0, 0, 0, 0};
      };
      // Each wave's own loads.  Both caches are read once: non-temporal, except where
      // a step's values are parts of lines (long pages).
      auto load_k = [&](const Pages& e, int tt) __attribute__((always_inline)) {
#pragma unroll
        for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            kf[kt][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(k_block(e, tt, kt, j)));
      };
      auto load_v = [&](const Pages& e, int tt) __attribute__((always_inline)) {
        const uint8_t* base = v_base(e, tt);
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt) {
          const u32x4* q = reinterpret_cast<const u32x4*>(base + (int64_t)dt * 16 * P * kEl);
          vf[dt] = kPage == 0 ? *q : __builtin_nontemporal_load(q);
        }
      };
      // The positions of the step at t0 that this lane's rows see, as bits.
      typedef std::conditional_t<F8, uint64_t, uint32_t> Bits;
      auto below = [](int n) __attribute__((always_inline)) -> Bits {     // the first n positions
        return n >= kTok ? ~(Bits)0 : n <= 0 ? (Bits)0 : ((Bits)1 << n) - 1;
      };
      auto visible = [&](Bits (&vis)[NT]) __attribute__((always_inline)) {
        const int j0 = t0 - ctx;           // place of the first of them in the segment
        const Bits before = below(-j0);
        const Bits inside = below(rq.n - j0) & ~before;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Bits bits;
          if (a.mask) {
            const uint32_t* mw = a.mask + (int64_t)(rq.start + el[nt]) * a.mask_words;
            const int jj = j0 < 0 ? 0 : j0;
            const int w0 = jj >> 5, sh = jj & 31;
            uint64_t two;
            auto word = [&](int w) { return w < a.mask_words ? (uint64_t)mw[w] : (uint64_t)0; };
            if (short_mask) {
              two = jj < 64 ? mask64[nt] >> jj : 0;
            } else {
              two = (word(w0) | word(w0 + 1) << 32) >> sh;
              if (F8) two |= sh ? word(w0 + 2) << (64 - sh) : (uint64_t)0;
            }
            bits = (Bits)two;
            if (j0 < 0) bits = -j0 < kTok ? bits << -j0 : (Bits)0;
          } else {
            bits = below(el[nt] - j0 + 1);
          }
          vis[nt] = before | (bits & inside);
        }
      };
      // Bits of this lane's scores: those of tile kt in the lowest four.
      auto mine = [&](Bits v, int kt) __attribute__((always_inline)) { return (uint32_t)(v >> (16 * kt + 4 * g)); };
      // Values behind the last position become zeros, and so do others that are not
      // finite if `clear`.  Returns whether there were such.
      auto trim_values = [&](bool clear) __attribute__((always_inline)) {
        const int keep = total - (t0 + vb);
        uint32_t odd = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          constexpr int kPer = 4 / kEl;    // values a word
          const int c = keep - i * kPer;
          const uint32_t live = c >= kPer ? 0xffffffffu : c <= 0 ? 0u : (1u << (c * 8 * kEl)) - 1u;
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt) {
            uint32_t x = vf[dt][i] & live;
            const uint32_t flags = F8 ? bytes_nan(x) : halves_from(x, E::kExp);
            odd |= flags;
            if (clear) x &= ~(flags * (F8 ? 0xffu : 0xffffu));
            vf[dt][i] = x;
          }
        }
        return odd;
      };
      uint32_t specials = 0u;
      Pages ahead = entries(t0);
      const uint8_t* slot = sh_mem;        // kRing: the step's blocks

      auto step = [&](auto is_edge) __attribute__((always_inline)) {
        constexpr bool kEdge = decltype(is_edge)::value;
        // Past the last step the next loads read the last page again and are not used.
        const int next = t0 + t_step;
        Pages now;
        if constexpr (!kRing) {
          now = check(ahead);
          ahead = entries(next + t_step);
        } else {
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int j = 0; j < kJ; ++j)
              kf[kt][j] = *reinterpret_cast<const u32x4*>(slot + (kt * kJ + j) * 1024 + lane * 16);
        }
        k_tail();
        // ---- scores ----
        f32x4 s[NT][kKT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt) s[nt][kt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < kMj; ++i)
#pragma unroll
            for (int kt = 0; kt < kKT; ++kt) {
              const u32x4 kx = F8 ? widen8<DT>(kf[kt][j], i) : kf[kt][j];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                s[nt][kt] = E::mma(kx, qf[nt][j * kMj + i], s[nt][kt]);
            }
        if constexpr (!kRing) load_k(now, next);
        // ---- positions that rows do not see ----
        Bits vis[NT];
        if constexpr (kEdge) {
          visible(vis);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t on = spread(mine(vis[nt], kt), i);
                s[nt][kt][i] = as_float((as_bits(s[nt][kt][i]) & on) | (0xff800000u & ~on));
              }
        }
        if constexpr (kRing) {
          // read before the exponentials, so that they cover the latency
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt)
            vf[dt] = *reinterpret_cast<const u32x4*>(slot + (kKB + dt) * 1024 + lane * 16);
          asm volatile("" ::: "memory");
        }
        // ---- probabilities ----
        float top[NT];
        bool rise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float x = s[nt][0][0];
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt)
#pragma unroll
            for (int i = 0; i < 4; ++i) x = fmaxf(x, s[nt][kt][i]);
          top[nt] = groups_max(x) * sc;
          rise |= top[nt] > m[nt] + kSlack;
        }
        if (__any(rise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float nm = top[nt] > m[nt] + kSlack ? top[nt] : m[nt];
            const float f = m[nt] == nm ? 1.0f : pow2(m[nt] - nm);
            l[nt] *= f;
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) o[nt][dt] *= f;
            m[nt] = nm;
          }
        }
        u32x4 pf[NT][kU];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float base = m[nt] == -INFINITY ? 0.0f : m[nt];
          uint32_t lo[kKT], hi[kKT];   // a tile's four probabilities, packed
          // Rounded to the element type here, and only here: the second product's operand.
          // As two operands each they would keep twice the bits and double that product and
          // its registers.  The sum takes them unrounded.  Against 64 bits the
          // rounding takes the outputs' error (norm of it over theirs) from 0.0017 to 0.0022
          // in bf16 and from 0.00021 to 0.00029 in fp16; the outputs' own is the first.
          float sum = 0.0f;
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              p[i] = pow2(fmaf(s[nt][kt][i], sc, -base));
              // unseen: 0 whatever the line above made of -inf
              if (kEdge) p[i] = as_float(as_bits(p[i]) & spread(mine(vis[nt], kt), i));
            }
            sum += (p[0] + p[1]) + (p[2] + p[3]);
            lo[kt] = E::pack(p[0], p[1]);
            hi[kt] = E::pack(p[2], p[3]);
          }
          l[nt] += sum;
          regroup(lo);
          regroup(hi);
#pragma unroll
          for (int u = 0; u < kU; ++u)
            pf[nt][u] = u32x4{lo[2 * u], hi[2 * u], lo[2 * u + 1], hi[2 * u + 1]};
        }
        // ---- values ----
        if constexpr (kEdge) {
          // A value that is not finite must not meet the zero probability of a row that
          // does not see it: it leaves the product here and comes back below.
          specials |= trim_values(true);
        }
#pragma unroll
        for (int dt = 0; dt < kDT; ++dt)
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const u32x4 vx = F8 ? widen8<DT>(vf[dt], u) : vf[dt];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) o[nt][dt] = E::mma(vx, pf[nt][u], o[nt][dt]);
          }
        if constexpr (!kRing) load_v(now, next);
      };
      const int t_plain = min(t_end, ctx - kTok + 1);   // steps that end within the context
      int t_edge = max(t_plain, 0);
      t_edge = t0 >= t_edge ? t0 : t0 + (t_edge - t0 + t_step - 1) / t_step * t_step;
      if constexpr (!kRing) {
        const Pages first = check(ahead);
        load_k(first, t0);
        load_v(first, t0);
        ahead = entries(t0 + t_step);
        for (; t0 < t_plain; t0 += t_step) step(std::false_type{});
        for (; t0 < t_end; t0 += t_step) step(std::true_type{});
      } else {
        // Step x of this group of waves lies in slot x % n of its part of the ring.  The
        // loads of a step past the group's last one go to the last one again, so that
        // every wave issues the same number and a wait means the same for all.
        const int all_steps = (t_end_tile - t0_tile + t_step - 1) / t_step;
        const int t_last = t0 + max((t_end_tile - t0 + t_step - 1) / t_step - 1, 0) * t_step;
        int t_in = min(t0, t_last);
        int in = 0, out = 0;                 // slots that are loaded and used next
        const uint8_t* ring = sh_mem;
        auto fill = [&](auto wr_) __attribute__((always_inline)) {
          constexpr int kWr = decltype(wr_)::value;
          constexpr int kN = ring_steps(kSlots, kWaves / kWr);
          const Pages e = check(ahead);
          const int tt = t_in;
          t_in = min(t_in + t_step, t_last);
          ahead = entries(t_in);
          const uint32_t to = lds_address(ring) + in * (kBlocks * 1024);
#pragma unroll
          for (int i = 0; i < (kKB + kWr - 1) / kWr; ++i) {
            const int blk = min(my_r + i * kWr, kKB - 1);
            const int kt = blk / kJ;
            copy_to_lds(k_block(e, tt, kt, blk - kt * kJ), to + blk * 1024);
          }
          const uint8_t* vp = v_base(e, tt);
#pragma unroll
          for (int i = 0; i < (kDT + kWr - 1) / kWr; ++i) {
            const int dt = min(my_r + i * kWr, kDT - 1);
            copy_to_lds(vp + (int64_t)dt * 16 * P * kEl, to + (kKB + dt) * 1024);
          }
          in = in + 1 == kN ? 0 : in + 1;
        };
        auto begin = [&](auto wr_) __attribute__((always_inline)) {
          constexpr int kN = ring_steps(kSlots, kWaves / decltype(wr_)::value);
          ring = sh_mem + my_t * (kN * kBlocks * 1024);
#pragma unroll
          for (int i = 0; i < kN - 1; ++i) fill(wr_);
        };
        auto advance = [&](auto wr_) __attribute__((always_inline)) {
          constexpr int kWr = decltype(wr_)::value;
          constexpr int kN = ring_steps(kSlots, kWaves / kWr);
          constexpr int kLoads = (kKB + kWr - 1) / kWr + (kDT + kWr - 1) / kWr;
          static_assert(kN >= 2 && (kN - 1) * kLoads <= 63, "ring depth");
          wait_loads<(kN - 2) * kLoads>();
          // every wave's part of the step has landed, and the slot that is filled next
          // has been used up by all
          bare_barrier();
          fill(wr_);
          slot = ring + out * (kBlocks * 1024);
          out = out + 1 == kN ? 0 : out + 1;
        };
        typedef std::integral_constant<int, kWaves> Eight;   // or four, not used
        typedef std::integral_constant<int, 4> Four;
        typedef std::integral_constant<int, 2> Two;
        if (kWaves == 8 && wr == 8) begin(Eight{});
        else if (wr == 4) begin(Four{});
        else begin(Two{});
        int x = 0;
        auto next_step = [&](auto is_edge) __attribute__((always_inline)) {
          if (kWaves == 8 && wr == 8) advance(Eight{});
          else if (wr == 4) advance(Four{});
          else advance(Two{});
          if (t0 < t_end) step(is_edge);
          t0 += t_step;
          ++x;
        };
        while (x < all_steps && t0 < t_plain) next_step(std::false_type{});
        while (x < all_steps) next_step(std::true_type{});
        wait_loads<0>();
      }
      // Rows that see values that are not finite get them by products of indicators:
      // 1 where the value is +inf, -inf or NaN, with 1 where it is seen.
      if (__any(specials != 0u)) {
#pragma unroll 1
        for (t0 = t_edge; t0 < t_end; t0 += t_step) {
          load_v(check(entries(t0)), t0);
          if (!__any(trim_values(false) != 0u)) continue;
          Bits vis[NT];
          visible(vis);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            u32x4 sees[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t v = (uint32_t)(vis[nt] >> vb);   // this lane's values
                sees[nt][i] = (spread(v, 8 * u + 2 * i) & E::kOne) |
                              (spread(v, 8 * u + 2 * i + 1) & (E::kOne << 16));
              }
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) {
              const u32x4 x = F8 ? widen8<DT>(vf[dt], u) : vf[dt];
              u32x4 up, down, nan;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t is_nan = halves_from(x[i], E::kExp + 1u);
                const uint32_t inf = halves_from(x[i], E::kExp) & ~is_nan;
                const uint32_t minus = (x[i] >> 15) & 0x00010001u;
                nan[i] = is_nan * E::kOne;
                up[i] = (inf & ~minus) * E::kOne;
                down[i] = (inf & minus) * E::kOne;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                const f32x4 n_up = E::mma(up, sees[nt], zero);
                const f32x4 n_down = E::mma(down, sees[nt], zero);
                const f32x4 n_nan = E::mma(nan, sees[nt], zero);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float add = n_up[i] > 0.0f ? INFINITY : 0.0f;
                  add -= n_down[i] > 0.0f ? INFINITY : 0.0f;
                  o[nt][dt][i] += n_nan[i] > 0.0f ? NAN : add;
                }
              }
              __builtin_amdgcn_sched_barrier(0);   // one output tile at a time: few registers
            }
          }
        }
      }
    }
    // A bad page, length or table: every row of the wave is NaN.
    if (__any(bad)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) l[nt] = NAN;
    }

    // ---- join the waves over positions ----
    for (int half = wt >> 1; half >= 1; half >>= 1) {
      // buffers: wr * half <= kWaves / 2
      const int buf = (my_t & (half - 1)) * wr + my_r;
      __syncthreads();
      if (my_t >= half && my_t < 2 * half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          sh_ml[buf][nt][0][lane] = m[nt];
          sh_ml[buf][nt][1][lane] = l[nt];
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt) sh_o[buf][nt * kDT + dt][lane] = o[nt][dt];
        }
      }
      __syncthreads();
      if (my_t < half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float m2 = sh_ml[buf][nt][0][lane], l2 = sh_ml[buf][nt][1][lane];
          const float nm = fmaxf(m[nt], m2);
          const float base = nm == -INFINITY ? 0.0f : nm;
          const float f1 = pow2(m[nt] - base), f2 = pow2(m2 - base);
          m[nt] = nm;
          l[nt] = l[nt] * f1 + l2 * f2;
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt)
            o[nt][dt] = o[nt][dt] * f1 + sh_o[buf][nt * kDT + dt][lane] * f2;
        }
      }
    }

    // ---- out ----
    const bool complete = s0 == 0 && s1 == units;
    if (my_t == 0) {
      const float vs = a.v_scale ? a.v_scale[h] : 1.0f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + nt * 16 + col;
        const float sum = groups_sum(l[nt]);
        if (complete) {
          if (row < rq.rows) {
            const int y = h * group + row - el[nt] * group;
            const float f = sum == 0.0f ? 0.0f : vs / sum;
            uint16_t* op = static_cast<uint16_t*>(a.out) +
                           (int64_t)(rq.start + el[nt]) * a.out_stride + y * D + g * 4;
#pragma unroll
            for (int dt = 0; dt < kDT; ++dt) {
              uint2 x;
              x.x = E::pack(o[nt][dt][0] * f, o[nt][dt][1] * f);
              x.y = E::pack(o[nt][dt][2] * f, o[nt][dt][3] * f);
              *reinterpret_cast<uint2*>(op + dt * 16) = x;
            }
            if (a.lse && g == 0)
              a.lse[(int64_t)(rq.start + el[nt]) * a.Hq + y] =
                  (m[nt] + __log2f(sum)) * 0.69314718055994531f;
          }
        } else if (row0 + nt * 16 < rq.rows) {
          const int64_t slot = 2 * (int64_t)b + (s0 == 0 ? 1 : 0);
          const int64_t blk = slot * kWaves * NT + my_r * NT + nt;
          part_ml[(blk * 2) * 64 + lane] = m[nt];
          part_ml[(blk * 2 + 1) * 64 + lane] = sum;
          f32x4* po = reinterpret_cast<f32x4*>(part_o) + blk * kDT * 64;
#pragma unroll
          for (int dt = 0; dt < kDT; ++dt) po[dt * 64 + lane] = o[nt][dt];
        }
      }
    }
    if (!complete && s0 == 0) {
      // the tile's last unit belongs to the workgroup that ends the row of parts
      const int64_t last = w + (units - 1);
      int64_t owner = last * runs / all;
      while (all * (owner + 1) / runs <= last) ++owner;
      cut.parts = (int)(owner - b) + 1;
      cut.start = rq.start;
      cut.rows = rq.rows;
      cut.row0 = row_tile * (16 * NT * kWaves);
      cut.h = h;
    }
    w += s1 - s0;
    if (w >= w_end) break;
    // the next tile: of this head, of the next one, of the next request with rows
    s0 = 0;
    ++row_tile;
    if (row_tile >= rq.full + (rq.wr_last > 0 ? 1 : 0)) {
      row_tile = 0;
      ++h;
    }
    if (h >= a.Hk) {
      h = 0;
      do rq = request<NT, kTok, kWaves, kRing>(a, ++r, group, whole);
      while (rq.rows == 0);                // there is one: units are left
    }
  }
  if (t == 0 && !whole) cuts[b] = cut;
}

// Joins the parts of cut tiles.  Grid: (workgroups of the first launch, 16-row
// blocks of a tile).  A wave joins its share of the channels, kAhead parts' loads at
// a time: over all parts where a tile has few, over every second group of them
// where it has many (SPLIT = 2, one wave of each pair then adds the other's).  The
// order of the sums is fixed.
template <int DT, int D, int BLOCKS, int SPLIT>
__global__ __launch_bounds__(kJoinThreads * SPLIT) void tree_attention_join_kernel(
    const TreeAttnArgs a, const AttnCut* __restrict__ cuts, const float* __restrict__ part_ml,
    const float* __restrict__ part_o) {
  constexpr int kDT = D / 16;
  constexpr int kMine = (kDT + kJoinWaves - 1) / kJoinWaves;
  constexpr int kAhead = 4 * SPLIT;
  using E = El<DT>;
  __shared__ f32x4 sh_o[SPLIT > 1 ? kJoinWaves : 1][kMine][64];
  __shared__ float sh_ml[SPLIT > 1 ? kJoinWaves : 1][2][64];
  // In the order of the first launch: runs that tiles of equal length start in are a
  // multiple of eight apart, and in the grid's own order one XCD would join them all
  // (8 tiles of 33 parts: 57 us, so 15).
  const int b = run_of(blockIdx.x, gridDim.x);
  const int blk = blockIdx.y;
  const AttnCut cut = cuts[b];
  const int row0 = cut.row0 + blk * 16;
  if (cut.parts == 0 || row0 >= cut.rows) return;
  const int lane = threadIdx.x & 63;
  const int wave = uni((threadIdx.x >> 6) & (kJoinWaves - 1));
  const int share = uni(threadIdx.x >> 6) / kJoinWaves;   // of the parts
  const int dt0 = wave * kMine;          // (past the last channel there is no output)
  float m = -INFINITY, l = 0.0f;
  f32x4 o[kMine];
#pragma unroll
  for (int d = 0; d < kMine; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int p0 = share * kAhead; p0 < cut.parts; p0 += SPLIT * kAhead) {
    float m2[kAhead], l2[kAhead];
    f32x4 x[kAhead][kMine];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int p = min(p0 + u, cut.parts - 1);
      const int64_t slot = p == 0 ? 2 * (int64_t)b + 1 : 2 * (int64_t)(b + p);
      const int64_t at = slot * BLOCKS + blk;
      m2[u] = part_ml[(at * 2) * 64 + lane];
      l2[u] = part_ml[(at * 2 + 1) * 64 + lane];
      const f32x4* po = reinterpret_cast<const f32x4*>(part_o) + at * kDT * 64 + lane;
#pragma unroll
      for (int d = 0; d < kMine; ++d) x[u][d] = po[min(dt0 + d, kDT - 1) * 64];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (p0 + u >= cut.parts) continue;
      const float nm = fmaxf(m, m2[u]);
      const float base = nm == -INFINITY ? 0.0f : nm;
      const float f1 = pow2(m - base), f2 = pow2(m2[u] - base);
      m = nm;
      l = l * f1 + l2[u] * f2;
#pragma unroll
      for (int d = 0; d < kMine; ++d) o[d] = o[d] * f1 + x[u][d] * f2;
    }
  }
  if constexpr (SPLIT > 1) {
    if (share == 1) {
      sh_ml[wave][0][lane] = m;
      sh_ml[wave][1][lane] = l;
#pragma unroll
      for (int d = 0; d < kMine; ++d) sh_o[wave][d][lane] = o[d];
    }
    __syncthreads();
    if (share == 1) return;
    const float m2 = sh_ml[wave][0][lane];
    const float nm = fmaxf(m, m2);
    const float base = nm == -INFINITY ? 0.0f : nm;
    const float f1 = pow2(m - base), f2 = pow2(m2 - base);
    m = nm;
    l = l * f1 + sh_ml[wave][1][lane] * f2;
#pragma unroll
    for (int d = 0; d < kMine; ++d) o[d] = o[d] * f1 + sh_o[wave][d][lane] * f2;
  }
  const int col = lane & 15, g = lane >> 4;
  const int row = row0 + col;
  if (row >= cut.rows) return;
  const int group = a.Hq / a.Hk;
  const int el = row / group;
  const int y = cut.h * group + row - el * group;
  const float vs = a.v_scale ? a.v_scale[cut.h] : 1.0f;
  const float f = l == 0.0f ? 0.0f : vs / l;
  uint16_t* op = static_cast<uint16_t*>(a.out) + (int64_t)(cut.start + el) * a.out_stride + y * D + g * 4;
#pragma unroll
  for (int d = 0; d < kMine; ++d) {
    if (dt0 + d >= kDT) break;
    uint2 x;
    x.x = E::pack(o[d][0] * f, o[d][1] * f);
    x.y = E::pack(o[d][2] * f, o[d][3] * f);
    *reinterpret_cast<uint2*>(op + (dt0 + d) * 16) = x;
  }
  if (a.lse && g == 0 && dt0 == 0)
    a.lse[(int64_t)(cut.start + el) * a.Hq + y] = (m + __log2f(l)) * 0.69314718055994531f;
}

template <int DT, bool F8, int D, int NT, bool RING>
dspark_status go(const TreeAttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  AttnCut* cuts = static_cast<AttnCut*>(a.ws);
  float* ml = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + p.cut_bytes);
  float* po = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + p.cut_bytes + p.ml_bytes);
  // a step has 32 positions, 64 with an 8-bit cache
  auto kernel = a.shift == 4         ? &tree_attention_kernel<DT, F8, D, NT, 4, RING>
                : F8 && a.shift == 5 ? &tree_attention_kernel<DT, F8, D, NT, F8 ? 5 : 0, RING>
                                     : &tree_attention_kernel<DT, F8, D, NT, 0, RING>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)p.groups), dim3(64 * attn_group(D, RING)), 0, stream, a,
                     p.whole, cuts, ml, po);
  const dspark_status st = check_launch("tree_attention_kernel");
  if (st != DSPARK_OK || p.whole) return st;
  auto join = p.deep ? &tree_attention_join_kernel<DT, D, attn_group(D, RING) * NT, 2>
                     : &tree_attention_join_kernel<DT, D, attn_group(D, RING) * NT, 1>;
  hipLaunchKernelGGL(join, dim3((unsigned)p.groups, (unsigned)p.row_blocks),
                     dim3(kJoinThreads * (p.deep ? 2 : 1)), 0, stream, a, cuts, ml, po);
  return check_launch("tree_attention_join_kernel");
}
template <int DT, bool F8, int D>
dspark_status go(const TreeAttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if (p.ring) return go<DT, F8, D, 2, true>(a, p, stream);
  // (heads above 128 share a ring from two tiles on)
  if constexpr (D <= 128)
    if (p.nt == 2) return go<DT, F8, D, 2, false>(a, p, stream);
  return go<DT, F8, D, 1, false>(a, p, stream);
}

}  // namespace

template <int DT, bool F8>
dspark_status run_tree_attention(const TreeAttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  switch (a.D) {
    case 64: return go<DT, F8, 64>(a, p, stream);
    case 96: return go<DT, F8, 96>(a, p, stream);
    case 128: return go<DT, F8, 128>(a, p, stream);
    case 192: return go<DT, F8, 192>(a, p, stream);
    default: return go<DT, F8, 256>(a, p, stream);
  }
}

}  // namespace dspark
