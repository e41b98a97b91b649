// Matrix products in 16-bit types with fp32 accumulation on tcgen05 (kind::f16): the dense
// product with bias, activation and residual in its epilogue, the same product grouped by
// expert over ragged row ranges, and their two gradients.  (A dense forward product of a few rows:
// warp-level MMAs, lin_token_kernel.)
//
// Every product is written as out[j][i] = sum_c A[i][c] B[j][c], with i on the MMA's M (the
// TMEM lanes) and j on its N (the columns):
//   forward       i = output feature, j = token row, c = input feature   A = W,   B = x
//   input grad    i = input feature,  j = token row, c = output feature  A = W^T, B = dz
//   weight grad   i = input feature,  j = output feature, c = token row  A = x^T, B = dz^T
// The transposed operands are read as they lie in memory, as MN-major operands.  Token rows on
// N rather than M: a ragged expert's last tile then takes an MMA as narrow as its rows (in
// steps of 16), where a tile on M would always pay 128 rows, and a decode step's few tokens
// take an N of 16 under a weight tile of 128 rows that streams through once; and any row can be
// left out of the stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <atomic>
#include <mutex>

#include "linear_ptx.cuh"
#include "moe_linear.cuh"
#include "packed_math.cuh"
#include "row_blocks.h"

namespace moe {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s: a stuck pipeline, not a slow one
constexpr uint64_t kLandNs = 20000000ull;     // 20 ms: copies issued before a timeout have landed
constexpr int kBK = kBlockRows;                // contraction values per stage (a 128-byte row)

struct LinParams {
  int32_t rows, E, fn;
  int32_t I;             // extent of i (columns of out)
  int32_t J;             // extent of j (kWeightGrad: N; else the expert's rows)
  int32_t C;             // extent of c (kWeightGrad: the expert's rows)
  int32_t a_rows;        // kForward: rows of W per expert
  int32_t n_it;          // tiles along i
  int32_t nw_max;        // widest tile along j
  int32_t n_jt;          // kWeightGrad: tiles along j
  int32_t splits;        // CTAs of a cluster that share one tile's contraction
  int32_t win;           // kWeightGrad: rows of map 0's window
  float limit;
  const int32_t* offsets;
  uint16_t* out;
  int64_t ld_out;
  int64_t out_expert;    // kWeightGrad: elements of out per expert
  const float* bias;
  const uint16_t* residual;
  int64_t ld_res;
  uint16_t* z;
  int32_t* status;
  int32_t inject_timeout;
  const uint16_t* out_end;   // ends of out and z (bounds-checking builds)
  const uint16_t* z_end;
};

// One tile of the output: rows j0 .. j0 + nj - 1 (token rows of the buffer, or rows of dW) and
// columns i0 .. of expert e; the MMA's N is nw >= nj.
struct LinTile {
  int32_t e, i0, j0, nj, nw;
  int32_t c0, clen;      // contraction range (kWeightGrad: token rows c0 .. c0 + clen - 1)
  int32_t ok;
};

// ------------------------------------------------------------------------------ conversions
template <bool BF>
__device__ __forceinline__ uint16_t to16(float v) {
  return BF ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
template <bool BF>
__device__ __forceinline__ uint32_t to16x2(float lo, float hi) {   // lo in the low half
  if (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool BF>
__device__ __forceinline__ float from16(uint16_t v) {
  return BF ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

// ------------------------------------------------------------------------------ activations
// In fp32 with the hardware exponential: its relative error (a few 2^-23) and that of the
// approximate divide are far below the 16-bit rounding that follows.
// (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)) and (1 + erf v) / 2 = erfc(-v) / 2 keep their relative
// accuracy where the left sides cancel.  erfc by the Chebyshev fit of Press et al., Numerical
// Recipes, "erfcc" (relative error 1.2e-7 everywhere): one exponential and one divide, where erfcf
// set the time of products with a short contraction (16336 x 144 x 4384: 340 us).
// Of two values at once, in packed arithmetic.
__device__ __forceinline__ void normal_cdf2(float z0, float z1, float& c0, float& c1) {
  float x0, x1, t0, t1, q0, q1;
  mul2(x0, x1, fabsf(z0), fabsf(z1), 0.70710678f, 0.70710678f);
  fma2(t0, t1, x0, x1, 0.5f, 0.5f, 1.f, 1.f);
  t0 = __fdividef(1.f, t0);
  t1 = __fdividef(1.f, t1);
  fma2(q0, q1, t0, t1, 0.17087277f, 0.17087277f, -0.82215223f, -0.82215223f);
  fma2(q0, q1, t0, t1, q0, q1, 1.48851587f, 1.48851587f);
  fma2(q0, q1, t0, t1, q0, q1, -1.13520398f, -1.13520398f);
  fma2(q0, q1, t0, t1, q0, q1, 0.27886807f, 0.27886807f);
  fma2(q0, q1, t0, t1, q0, q1, -0.18628806f, -0.18628806f);
  fma2(q0, q1, t0, t1, q0, q1, 0.09678418f, 0.09678418f);
  fma2(q0, q1, t0, t1, q0, q1, 0.37409196f, 0.37409196f);
  fma2(q0, q1, t0, t1, q0, q1, 1.00002368f, 1.00002368f);
  fma2(q0, q1, t0, t1, q0, q1, -1.26551223f, -1.26551223f);
  fma2(q0, q1, -x0, -x1, x0, x1, q0, q1);
  mul2(t0, t1, t0, t1, 0.5f, 0.5f);
  mul2(q0, q1, t0, t1, __expf(q0), __expf(q1));   // erfc(|z| / sqrt 2) / 2
  c0 = z0 < 0.f ? q0 : 1.f - q0;
  c1 = z1 < 0.f ? q1 : 1.f - q1;
}
__device__ __forceinline__ float gelu_arg(float z) { return 0.79788456f * z * (1.f + 0.044715f * z * z); }

template <int FN>
__device__ __forceinline__ float act_fn(float z) {
  if (FN == MOE_FN_RELU) return z < 0.f ? 0.f : z;   // (NaN stays NaN)
  if (FN == MOE_FN_SILU) return __fdividef(z, 1.f + __expf(-z));
  if (FN == MOE_FN_GELU_TANH) return __fdividef(z, 1.f + __expf(-2.f * gelu_arg(z)));
  return z;
}

template <int FN>
__device__ __forceinline__ void act_pair(float& a, float& b) {
  if (FN == MOE_FN_GELU) {
    float ca, cb;
    normal_cdf2(a, b, ca, cb);
    mul2(a, b, a, b, ca, cb);
  } else {
    a = act_fn<FN>(a);
    b = act_fn<FN>(b);
  }
}

__device__ __forceinline__ float clamp_hi(float v, float L) { return v > L ? L : v; }    // NaN passes
__device__ __forceinline__ float clamp_both(float v, float L) { return v > L ? L : (v < -L ? -L : v); }

__device__ __forceinline__ float swiglu(float g, float u, float L) {
  const float gc = clamp_hi(g, L);
  return __fdividef(gc, 1.f + __expf(-gc)) * clamp_both(u, L);
}

// ------------------------------------------------------------------------------ ragged rows
// Range [a, b) of expert e, forced into [0, rows] and into order; bad offsets raise *bad.
__device__ __forceinline__ void expert_rows(const int32_t* off, int32_t rows, int e, int& a, int& b, bool& bad) {
  const int ra = __ldg(off + e), rb = __ldg(off + e + 1);
  a = min(max(ra, 0), rows);
  b = min(max(rb, a), rows);
  bad |= (a != ra) || (b != rb);
}

// Balanced tile width for cnt rows in tiles of at most nw_max, a multiple of `step`: the
// number of tiles stays ceil(cnt / nw_max).
__device__ __forceinline__ int tile_width(int cnt, int nt, int step) {
  return nt > 0 ? ((cnt + nt - 1) / nt + step - 1) / step * step : step;
}

// Tile `item` of a forward or input-gradient product, found by one warp (E <= 256: 8 experts
// per lane).  Tiles run expert by expert; within an expert its token tiles run fastest (CTAs that
// start together then share a weight tile in L2).
__device__ __forceinline__ LinTile find_row_tile(const LinParams& p, uint32_t item, int step, int iw) {
  const int lane = threadIdx.x & 31;
  LinTile t;
  t.ok = 0;
  t.c0 = 0;
  t.clen = p.C;
  if (!p.offsets) {
    const int nt = (p.rows + p.nw_max - 1) / p.nw_max, w = tile_width(p.rows, nt, step);
    if (item < (uint32_t)nt * (uint32_t)p.n_it) {
      const int it = item / (uint32_t)nt, jt = item - (uint32_t)it * nt;
      t.ok = 1;
      t.e = 0;
      t.i0 = it * iw;
      t.j0 = jt * w;
      t.nj = min(w, p.rows - t.j0);
      t.nw = (t.nj + step - 1) / step * step;
    }
    return t;
  }
  int a[8], cnt[8], sum = 0;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = 8 * lane + k;
    a[k] = 0;
    cnt[k] = 0;
    if (e < p.E) {
      int b;
      expert_rows(p.offsets, p.rows, e, a[k], b, bad);
      cnt[k] = b - a[k];
    }
    sum += (cnt[k] + p.nw_max - 1) / p.nw_max;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (__any_sync(0xffffffffu, bad) && item == 0 && lane == 0) set_status(p.status, MOE_ERR_INVALID_ARG);
  const uint32_t lo = (uint32_t)(incl - sum) * p.n_it, hi = (uint32_t)incl * p.n_it;
  const unsigned who = __ballot_sync(0xffffffffu, item >= lo && item < hi);
  if (!who) return t;
  const int src = __ffs(who) - 1;
  int fe = 0, fa = 0, fc = 0, floc = 0;
  if (lane == src) {
    uint32_t base = lo;
    bool found = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t n = (uint32_t)((cnt[k] + p.nw_max - 1) / p.nw_max) * p.n_it;
      if (!found && item < base + n) {
        found = true;
        fe = 8 * lane + k;
        fa = a[k];
        fc = cnt[k];
        floc = (int)(item - base);
      }
      base += n;
    }
  }
  fe = __shfl_sync(0xffffffffu, fe, src);
  fa = __shfl_sync(0xffffffffu, fa, src);
  fc = __shfl_sync(0xffffffffu, fc, src);
  floc = __shfl_sync(0xffffffffu, floc, src);
  const int nt = (fc + p.nw_max - 1) / p.nw_max, w = tile_width(fc, nt, step);
  const int it = floc / nt, jt = floc - it * nt;
  t.ok = 1;
  t.e = fe;
  t.i0 = it * iw;
  t.j0 = fa + jt * w;
  t.nj = min(w, fc - jt * w);
  t.nw = (t.nj + step - 1) / step * step;
  return t;
}

// Tile `item` of a weight gradient: every expert has the same tiles, its own contraction range.
__device__ __forceinline__ LinTile find_weight_tile(const LinParams& p, uint32_t item, int step, int iw) {
  LinTile t;
  const int per_e = p.n_it * p.n_jt;
  t.ok = item < (uint32_t)per_e * (uint32_t)p.E;
  if (!t.ok) return t;
  t.e = item / (uint32_t)per_e;
  const int loc = item - (uint32_t)t.e * per_e;
  const int w = tile_width(p.J, p.n_jt, step);
  t.i0 = (loc % p.n_it) * iw;
  t.j0 = (loc / p.n_it) * w;
  t.nj = min(w, p.J - t.j0);
  t.nw = (max(t.nj, 1) + step - 1) / step * step;
  t.c0 = 0;
  t.clen = p.rows;
  if (p.offsets) {
    int b;
    bool bad = false;
    expert_rows(p.offsets, p.rows, t.e, t.c0, b, bad);
    t.clen = b - t.c0;
    if (bad && loc == 0 && (threadIdx.x & 31) == 0) set_status(p.status, MOE_ERR_INVALID_ARG);
  }
  return t;
}

template <int MODE>
__device__ __forceinline__ LinTile find_tile(const LinParams& p, uint32_t item, int step, int iw) {
  if (MODE == kWeightGrad) return find_weight_tile(p, item, step, iw);
  return find_row_tile(p, item, step, iw);
}

// The experts' row ranges and tiles, kept in shared memory by kernels that take many tiles.
// Experts are ordered by the cost of one of their tiles, dearest first: the pairs take tiles in
// turn, so tiles that run side by side cost alike and the pairs end together (in the experts' own
// order some pairs drew the wide tiles of several: 7% longer at 32 experts of 512 +- 22 rows).
struct RowTable {
  uint32_t items;
  int32_t start[256], cnt[256];
  int32_t base[257];         // first tile (along j) of the expert of each rank
  uint8_t order[256];        // the expert of each rank
};

// Built by the whole block (at least 256 threads; contains block barriers).
template <int MODE>
__device__ __forceinline__ void build_table(const LinParams& p, RowTable* tab, int step) {
  const int th = threadIdx.x, lane = th & 31;
  bool bad = false;
  if (th < 256) {
    int a = 0, b = th < p.E ? p.rows : 0;
    if (p.offsets && th < p.E) expert_rows(p.offsets, p.rows, th, a, b, bad);
    tab->start[th] = a;
    tab->cnt[th] = b - a;
    tab->base[th] = 0;
  }
  if (bad && blockIdx.x == 0) set_status(p.status, MOE_ERR_INVALID_ARG);
  __syncthreads();
  // a tile's cost: its width, or the weight gradient's contraction length
  auto tiles_of = [&](int e) { return MODE == kWeightGrad ? p.n_jt : (tab->cnt[e] + p.nw_max - 1) / p.nw_max; };
  int cost = 0;
  if (th < p.E) cost = MODE == kWeightGrad ? tab->cnt[th] : tile_width(tab->cnt[th], tiles_of(th), step);
  if (th < p.E) tab->base[th] = cost;
  __syncthreads();
  if (th < p.E) {
    int rank = 0;
    for (int e = 0; e < p.E; ++e) {
      const int c = tab->base[e];
      rank += c > cost || (c == cost && e < th);
    }
    tab->order[rank] = (uint8_t)th;
  }
  __syncthreads();
  if (th < 32) {   // first tiles by rank, 8 ranks a lane
    int n[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      n[k] = 8 * lane + k < p.E ? tiles_of(tab->order[8 * lane + k]) : 0;
      sum += n[k];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int at = incl - sum;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      tab->base[8 * lane + k] = at;
      at += n[k];
    }
    if (lane == 31) {
      tab->base[256] = incl;
      tab->items = (uint32_t)incl * p.n_it;
    }
  }
}

// Tile `item` (< items) by the whole warp.  Tiles are listed expert by expert, dearest first, and
// within an expert along the axis with fewer tiles fastest: the tiles that run side by side then
// share the operand that is read once, and the other, smaller one stays in L2 (along i always:
// 4096 rows x 8 experts read 455 MB for 289 MB of operands, the weights again for each token tile;
// 301 MB so).  A weight gradient, bound by its writes, goes along i, so that whole rows of dW are
// written at one time (490 us, 520 along j).
template <int MODE>
__device__ __forceinline__ LinTile table_tile(const LinParams& p, const RowTable* tab, uint32_t item, int step, int iw) {
  const int lane = threadIdx.x & 31;
  const int q = item / (uint32_t)p.n_it;
  LinTile t;
  t.ok = 1;
  int rank = 0;
  if (p.E > 1) {   // the lane, then the rank of its eight, whose tiles hold q
    const unsigned m = __ballot_sync(0xffffffffu, tab->base[8 * lane] <= q && q < tab->base[8 * lane + 8]);
    const int r = 8 * (__ffs(m) - 1) + (lane & 7);
    const unsigned m8 = __ballot_sync(0xffffffffu, tab->base[r] <= q && q < tab->base[r + 1]);
    rank = 8 * (__ffs(m) - 1) + __ffs(m8) - 1;
  }
  t.e = p.E > 1 ? tab->order[rank] : 0;
  const int first = tab->base[rank], nt = tab->base[rank + 1] - first;
  const int cnt = tab->cnt[t.e], start = tab->start[t.e];
  int jt = q - first, it = item - (uint32_t)q * p.n_it;
  if (MODE != kWeightGrad && nt <= p.n_it) {
    const uint32_t loc = item - (uint32_t)first * p.n_it;
    it = loc / (uint32_t)nt;
    jt = loc - (uint32_t)it * nt;
  }
  t.i0 = it * iw;
  if (MODE == kWeightGrad) {
    const int w = tile_width(p.J, p.n_jt, step);
    t.j0 = jt * w;
    t.nj = min(w, p.J - t.j0);
    t.c0 = start;
    t.clen = cnt;
  } else {
    const int w = tile_width(cnt, (cnt + p.nw_max - 1) / p.nw_max, step);
    t.j0 = start + jt * w;
    t.nj = min(w, cnt - jt * w);
    t.c0 = 0;
    t.clen = p.C;
  }
  t.nw = (max(t.nj, 1) + step - 1) / step * step;
  return t;
}

// The tensor maps of a weight gradient's operands beside the first (row_blocks.h): windows of 8 rows
// and of one.
struct TailMaps {
  CUtensorMap a[2], b[2];
};
// Blocks of 64 along a tile's contraction.
template <int MODE>
__device__ __forceinline__ int tile_blocks(const LinParams& p, const LinTile& t) {
  return MODE == kWeightGrad ? weight_blocks(p.win, t.c0, t.clen) : (t.clen + kBK - 1) / kBK;
}

// ------------------------------------------------------------------------------ epilogue
// Four warps (128 threads, named barrier `bar`) finish 32 columns of a tile, held as matrix
// fragments: warp q has TMEM lanes 32 q ..; value (h, g, r), index 16 h + 4 g + r, of lane l is
// accumulator lane 32 q + 16 h + 8 (r / 2) + l / 4, column col0 + 8 g + 2 (l % 4) + r % 2.
// Accumulator lanes run along an output row: the 16-bit results are transposed into a shared
// buffer of output rows by stmatrix (8 x 8 values an instruction and matrix) and leave as 16-byte
// stores, 256 bytes of an output row by 16 threads.  (A lane per row with 2-byte stores to shared
// memory, 32 a thread, took 2.4 us of a 256 x 256 tile; with 2-byte stores to global memory, 5.)
// The buffer's rows are padded by 16 bytes, so that the 8 pieces of a matrix fall on other banks.
// SwiGLU: lanes 0-63 hold the gate and lanes 64-127 the up values of the tile's 64 features, the
// same fragment positions in warps q and q + 2.  The up warps hand their values of columns 0-15
// over, and take the gate values of columns 16-31, so that every thread finishes 16 columns.
constexpr int kEpiBytes = 9216;
constexpr int kPitch = 272, kPitchSw = 144;   // bytes per output row in the buffer: 128 or 64 values + 16

__device__ __forceinline__ void group_sync(int bar) { asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory"); }

// 32 accumulator columns of this warp's lanes as fragments (zeros where no contraction block was
// added).  taddr: the warp's first lane and the first column.
__device__ __forceinline__ void load_acc(uint32_t taddr, bool have, uint32_t (&v)[32]) {
  ptx::tmem_ld_16x256b_x4(taddr, v);
  ptx::tmem_ld_16x256b_x4(taddr + (16u << 16), v + 16);
  ptx::tmem_wait_ld();
  if (!have) {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = 0u;
  }
}

// Rows c < n of a buffer of W-value rows to dst (row c at dst + c ld), columns < lim.
template <int W>
__device__ __forceinline__ void store_rows(const LinParams& p, const uint8_t* buf, int pitch, uint16_t* dst, int64_t ld,
                                           int n, int lim, int th, const uint16_t* lo, const uint16_t* hi) {
  constexpr int V = W / 8;              // 16-byte pieces per row
  const int v = th % V;
  if (8 * v >= lim) return;             // (lim is a multiple of 8)
#pragma unroll
  for (int c = th / V; c < 32; c += 128 / V) {
    if (c < n) {
      uint4* q = reinterpret_cast<uint4*>(dst + c * ld + 8 * v);
      const uint4 val = *reinterpret_cast<const uint4*>(buf + c * pitch + 16 * v);
      if (in_bounds(q, lo, hi, p.status)) *q = val;
    }
  }
}

// This thread's pieces of the residual's 32 rows from col0 on.  They are fetched a step ahead, in
// registers, while the columns before them are finished: read where they were added, one after
// another, they made 16384 x 64 x 5760 258 us for 61 without a residual.
template <bool SW>
__device__ __forceinline__ void fetch_residual(const LinParams& p, const LinTile& t, int col0, int th, uint4 (&res)[4]) {
  constexpr int V = SW ? 8 : 16;        // pieces per row
  const int v = th % V;
  if (!p.residual || col0 >= t.nj || 8 * v >= p.I - t.i0) return;
  const uint16_t* src = p.residual + (int64_t)(t.j0 + col0) * p.ld_res + t.i0 + 8 * v;
#pragma unroll
  for (int k = 0; k < V / 4; ++k) {
    const int c = th / V + 128 / V * k;
    if (c < t.nj - col0) res[k] = *reinterpret_cast<const uint4*>(src + c * p.ld_res);
  }
}
template <bool SW>
__device__ __forceinline__ void place_residual(uint8_t* buf, int pitch, int th, const uint4 (&res)[4]) {
  constexpr int V = SW ? 8 : 16;
#pragma unroll
  for (int k = 0; k < V / 4; ++k)
    *reinterpret_cast<uint4*>(buf + (th / V + 128 / V * k) * pitch + 16 * (th % V)) = res[k];
}

// Column groups G0 .. G0 + NG - 1 of the fragments into the buffer (row 8 g + k, this warp's 32
// values at byte `at`), and back (added to v).
template <bool BF, int G0, int NG>
__device__ __forceinline__ void stage_frag(uint8_t* buf, int pitch, int at, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  const uint32_t base = ptx::smem_u32(buf) + (lane & 7) * pitch + at + 16 * (lane >> 3);
#pragma unroll
  for (int g = G0; g < G0 + NG; ++g)
    ptx::stmatrix_x4_trans(base + 8 * g * pitch, to16x2<BF>(v[4 * g], v[4 * g + 1]),
                           to16x2<BF>(v[4 * g + 2], v[4 * g + 3]), to16x2<BF>(v[16 + 4 * g], v[16 + 4 * g + 1]),
                           to16x2<BF>(v[16 + 4 * g + 2], v[16 + 4 * g + 3]));
}
template <bool BF, int G0, int NG>
__device__ __forceinline__ void add_frag(const uint8_t* buf, int pitch, int at, float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  const uint32_t base = ptx::smem_u32(buf) + (lane & 7) * pitch + at + 16 * (lane >> 3);
#pragma unroll
  for (int g = G0; g < G0 + NG; ++g) {
    uint32_t w[4];
    ptx::ldmatrix_x4_trans(base + 8 * g * pitch, w);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int i = 16 * (m >> 1) + 4 * g + 2 * (m & 1);
      v[i] += from16<BF>((uint16_t)w[m]);
      v[i + 1] += from16<BF>((uint16_t)(w[m] >> 16));
    }
  }
}

// SwiGLU of this thread's half of the columns (G0 = 0: gate warps, 2: up warps).
template <bool BF, int G0>
__device__ __forceinline__ void swiglu_half(const LinParams& p, float (&v)[32], const float4* theirs, int bar) {
  constexpr bool UP = G0 == 2;
#pragma unroll
  for (int k = 0; k < 4; ++k) {   // piece k: (h, g) = (k / 2, G0 + k % 2)
    const float4 o = theirs[64 * k];
    const int i = 16 * (k >> 1) + 4 * (G0 + (k & 1));
    const float other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      v[i + r] = UP ? swiglu(other[r], v[i + r], p.limit) : swiglu(v[i + r], other[r], p.limit);
  }
}

template <int FN, bool BF>
__device__ __forceinline__ void finish_cols(const LinParams& p, const LinTile& t, float (&v)[32], int col0, int th,
                                            uint8_t* buf, int bar, uint4 (&res)[4], int next) {
  const int n = min(32, t.nj - col0);   // valid columns
  const int64_t r0 = t.j0 + col0;
  uint16_t* out = p.out + t.e * p.out_expert + r0 * p.ld_out + t.i0;
  const int lim = p.I - t.i0;           // columns of out from i0 on
  const int q = th >> 5;
  group_sync(bar);                      // the buffer's last readers are done
  if (p.z) {
    stage_frag<BF, 0, 4>(buf, kPitch, 64 * q, v);
    group_sync(bar);
    if (FN == MOE_FN_SWIGLU) {   // gate lanes' 64 columns to z's first half, up lanes' to its second
      const int64_t ldz = 2 * (int64_t)p.I;
      const int h = th >> 6, w = th & 63, vv = w & 7;
      uint16_t* dst = p.z + r0 * ldz + h * (int64_t)p.I + t.i0;
      if (8 * vv < lim) {
#pragma unroll
        for (int c = w >> 3; c < 32; c += 8)
          if (c < n) {
            uint4* d = reinterpret_cast<uint4*>(dst + c * ldz + 8 * vv);
            const uint4 val = *reinterpret_cast<const uint4*>(buf + c * kPitch + 128 * h + 16 * vv);
            if (in_bounds(d, p.z, p.z_end, p.status)) *d = val;
          }
      }
    } else {
      store_rows<128>(p, buf, kPitch, p.z + r0 * p.I + t.i0, p.I, n, lim, th, p.z, p.z_end);
    }
    group_sync(bar);
  }
  if (FN == MOE_FN_SWIGLU) {
    const bool up = q >= 2;
    float4* ex = reinterpret_cast<float4*>(buf);   // [2][4][64] pieces: u of columns 0-15, g of columns 16-31
    float4* mine = ex + (up ? 0 : 256) + (th & 63);
    const float4* theirs = ex + (up ? 256 : 0) + (th & 63);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int a = 16 * (k >> 1) + 4 * (k & 1), b = a + 8;   // column groups k % 2 and 2 + k % 2
      mine[64 * k] = up ? make_float4(v[a], v[a + 1], v[a + 2], v[a + 3])
                        : make_float4(v[b], v[b + 1], v[b + 2], v[b + 3]);
    }
    group_sync(bar);
    if (up) swiglu_half<BF, 2>(p, v, theirs, bar);
    else swiglu_half<BF, 0>(p, v, theirs, bar);
    group_sync(bar);
    const int at = 64 * (q & 1);
    if (p.residual) {
      place_residual<true>(buf + 32 * kPitchSw, kPitchSw, th, res);
      fetch_residual<true>(p, t, next, th, res);
      group_sync(bar);
      if (up) add_frag<BF, 2, 2>(buf + 32 * kPitchSw, kPitchSw, at, v);
      else add_frag<BF, 0, 2>(buf + 32 * kPitchSw, kPitchSw, at, v);
    }
    if (up) stage_frag<BF, 2, 2>(buf, kPitchSw, at, v);
    else stage_frag<BF, 0, 2>(buf, kPitchSw, at, v);
    group_sync(bar);
    store_rows<64>(p, buf, kPitchSw, out, p.ld_out, n, lim, th, p.out, p.out_end);
  } else {
#pragma unroll
    for (int c = 0; c < 32; c += 2) act_pair<FN>(v[c], v[c + 1]);
    if (p.residual) {
      place_residual<false>(buf, kPitch, th, res);
      fetch_residual<false>(p, t, next, th, res);
      group_sync(bar);
      add_frag<BF, 0, 4>(buf, kPitch, 64 * q, v);   // (a warp reads and then overwrites its own values alone)
      __syncwarp();
    }
    stage_frag<BF, 0, 4>(buf, kPitch, 64 * q, v);
    group_sync(bar);
    store_rows<128>(p, buf, kPitch, out, p.ld_out, n, lim, th, p.out, p.out_end);
  }
}

// acc: the raw accumulator values; bias: of this thread's four accumulator lanes; th: the thread's
// number in its group, 32 q + lane; res: the residual's pieces of these columns, then those from
// column `next` on.
template <int MODE, bool SW, bool BF>
__device__ __forceinline__ void finish(const LinParams& p, const LinTile& t, const uint32_t (&acc)[32],
                                       const float (&bias)[4], int col0, int th, uint8_t* buf, int bar,
                                       uint4 (&res)[4], int next) {
  if (col0 >= t.nj) return;   // (the same for the whole group)
  float v[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    v[c] = __uint_as_float(acc[c]);
    if (MODE == kForward) v[c] += bias[2 * (c >> 4) + ((c >> 1) & 1)];
  }
  if (SW) return finish_cols<MOE_FN_SWIGLU, BF>(p, t, v, col0, th, buf, bar, res, next);
  if (MODE == kForward) {
    switch (p.fn) {
      case MOE_FN_RELU: return finish_cols<MOE_FN_RELU, BF>(p, t, v, col0, th, buf, bar, res, next);
      case MOE_FN_GELU: return finish_cols<MOE_FN_GELU, BF>(p, t, v, col0, th, buf, bar, res, next);
      case MOE_FN_GELU_TANH: return finish_cols<MOE_FN_GELU_TANH, BF>(p, t, v, col0, th, buf, bar, res, next);
      case MOE_FN_SILU: return finish_cols<MOE_FN_SILU, BF>(p, t, v, col0, th, buf, bar, res, next);
    }
  }
  finish_cols<MOE_FN_NONE, BF>(p, t, v, col0, th, buf, bar, res, next);
}

// The biases of this thread's accumulator lanes (SwiGLU: lanes 0-63 the gate's, 64-127 the up's).
template <int MODE, bool SW>
__device__ __forceinline__ void lane_bias(const LinParams& p, const LinTile& t, int th, float (&bias)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    bias[k] = 0.f;
    if (MODE == kForward && p.bias) {
      const int row = 32 * (th >> 5) + 8 * k + ((th & 31) >> 2);
      const int i = t.i0 + (SW ? row & 63 : row);
      if (i < p.I) bias[k] = __ldg(p.bias + (int64_t)t.e * p.a_rows + (SW && row >= 64 ? p.I : 0) + i);
    }
  }
}

// ------------------------------------------------------------------------------ split kernel
// One CTA (or a cluster of `splits` CTAs that share a tile's contraction) per output tile of
// 128 i x at most NB j (SwiGLU: 64 gate and the matching 64 up features), two CTAs per SM.
template <int MODE, int NB>
struct SplitCfg {
  static constexpr bool A_MN = MODE != kForward, B_MN = MODE == kWeightGrad;
  static constexpr int A_PANEL = 128 * 128;             // 128 i x 64 c of 2 bytes
  static constexpr int B_BYTES = NB * 128;
  static constexpr int STAGE = A_PANEL + B_BYTES;
  static constexpr int CPS = 2;                         // CTAs per SM
  static constexpr int S = 108 * 1024 / STAGE;
  static constexpr int TMEM_COLS = NB;
  // The stages are reused: the tile's fp32 partials, the received ones (splits x whole groups of
  // 8 columns: at most 7 more columns per split), the epilogue's buffer.
  static constexpr int SEND_BYTES = NB * 512, RED_BYTES = (NB + 32) * 512;
  static constexpr int EPI_OFF = SEND_BYTES + RED_BYTES;
  static constexpr int BAR_BYTES = 8 * (2 * S + 3) + 64;
  static constexpr int SMEM = S * STAGE + BAR_BYTES + 1024 /* align slack */;
  static constexpr int THREADS = 32 * 6;                // producer, MMA, four epilogue warps
  static_assert(EPI_OFF + kEpiBytes <= S * STAGE, "the partial tile and the epilogue's buffer fit the stages");
  static_assert(EPI_OFF + 32 * 512 <= S * STAGE, "a sum's reads past its share stay in the stages");
  static_assert((SMEM + 1024) * CPS <= 228 * 1024, "shared memory of the co-resident CTAs");
  static_assert((NB == 32 || NB == 64) && (!B_MN || NB % 64 == 0), "tile width");
};

template <int MODE, bool SW, int NB, bool BF>
__global__ void __launch_bounds__(SplitCfg<MODE, NB>::THREADS, SplitCfg<MODE, NB>::CPS)
    lin_split_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ TailMaps tails, const LinParams p) {
  using C = SplitCfg<MODE, NB>;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::S * C::STAGE);
  uint64_t* sfree = full + C::S;
  uint64_t* accf = sfree + C::S;
  uint64_t* drain = accf + 1;
  uint64_t* redf = drain + 1;        // the peers' partials have arrived
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(redf + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  LinTile* s_tile = reinterpret_cast<LinTile*>(s_tmem + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits;
  const int rank = S > 1 ? (int)ptx::cluster_ctarank() : 0;
  const uint32_t item = blockIdx.x / (unsigned)S;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < C::S; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&sfree[s], 1);
    }
    ptx::mbar_init(accf, 1);
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(redf, 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_a);
    ptx::prefetch_tensormap(&tm_b);
  }
  if (warp == 2) {
    const LinTile t = find_tile<MODE>(p, item, 16, SW ? 64 : 128);
    if (lane == 0) *s_tile = t;
  }
  // dz, in a backward call; what came before the call is complete without it.  Tensor memory is taken
  // after the wait: a CTA that held some while it waits for its predecessor could keep it from a CTA of
  // another stream whose own successor holds what that predecessor needs, and taking it has no bound.
  pdl_wait();
  if (warp == 1) {
    ptx::tmem_alloc(s_tmem, C::TMEM_COLS);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const LinTile t = *s_tile;
  const int kb_all = t.ok ? tile_blocks<MODE>(p, t) : 0;
  const int kb0 = (int)((int64_t)rank * kb_all / S), kb1 = (int)((int64_t)(rank + 1) * kb_all / S);

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    int g = 0;
    bool withheld = false;
    for (int kb = kb0; kb < kb1; ++kb, ++g) {
      const int s = g % C::S;
      bool ok = true;
      if (g >= C::S) ok = ptx::mbar_wait_bounded(&sfree[s], (uint32_t)(g / C::S - 1) & 1, s_abort, kWaitNs);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (p.inject_timeout && blockIdx.x == 0 && g == 0) {
        withheld = true;   // test hook: this stage never fills
        continue;
      }
      if (ptx::elect_one()) {
        uint8_t* a = smem + s * C::STAGE;
        uint8_t* b = a + C::A_PANEL;
        ptx::mbar_arrive_expect_tx(&full[s], C::STAGE);
        const int c = kb * kBK;
        if (MODE == kForward) {
          if (SW) ptx::tma_load_3d(a, &tm_a, c, t.i0, 2 * t.e, &full[s]);
          else ptx::tma_load_2d(a, &tm_a, c, t.e * p.a_rows + t.i0, &full[s]);
        } else if (MODE == kInputGrad) {
#pragma unroll
          for (int h = 0; h < 2; ++h) ptx::tma_load_3d(a + h * 8192, &tm_a, t.i0 + 64 * h, c, t.e, &full[s]);
        }
        if (MODE == kWeightGrad) {
          const RowBlock r = weight_block(p.win, t.c0, t.clen, kb);
          const CUtensorMap* map_a = r.map == 0 ? &tm_a : &tails.a[r.map - 1];
          const CUtensorMap* map_b = r.map == 0 ? &tm_b : &tails.b[r.map - 1];
#pragma unroll
          for (int h = 0; h < 2; ++h) ptx::tma_load_3d(a + h * 8192, map_a, t.i0 + 64 * h, r.d1, r.d2, &full[s]);
          ptx::tma_load_3d(b, map_b, t.j0, r.d1, r.d2, &full[s]);
        } else {
          ptx::tma_load_2d(b, &tm_b, c, t.j0, &full[s]);
        }
      }
      __syncwarp();
    }
    // no copies in flight when the CTA exits: wait (bounded) for the last fill of every slot
    volatile int local_abort = 0;
    for (int q = (g > C::S ? g - C::S : 0); q < g; ++q) {
      if (withheld && q == 0) continue;
      ptx::mbar_wait_bounded(&full[q % C::S], (uint32_t)(q / C::S) & 1, &local_abort, kWaitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t idesc = ptx::idesc_f16(BF, 128, t.nw, C::A_MN, C::B_MN);
    // a 16-wide step of c: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major box
    constexpr uint64_t kStepA = C::A_MN ? 2048 >> 4 : 32 >> 4, kStepB = C::B_MN ? 2048 >> 4 : 32 >> 4;
    int g = 0;
    bool stop = false;
    for (int kb = kb0; kb < kb1; ++kb, ++g) {
      const int s = g % C::S;
      if (!__all_sync(0xffffffffu,
                      ptx::mbar_wait_bounded(&full[s], (uint32_t)(g / C::S) & 1, s_abort, kWaitNs))) {
        stop = true;
        break;
      }
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
        const uint8_t* a = smem + s * C::STAGE;
        const uint8_t* b = a + C::A_PANEL;
        const uint64_t da = C::A_MN ? ptx::smem_desc_mn_sw128(a) : ptx::smem_desc_k_sw128(a);
        const uint64_t db = C::B_MN ? ptx::smem_desc_mn_sw128(b) : ptx::smem_desc_k_sw128(b);
#pragma unroll
        for (int k = 0; k < 4; ++k) ptx::mma_f16_ss(tmem, da + k * kStepA, db + k * kStepB, idesc, (g | k) != 0);
        ptx::tc_commit(&sfree[s]);
      }
      __syncwarp();
    }
    if (ptx::elect_one()) {
      if (!stop) ptx::tc_commit(accf);
      ptx::tc_commit(drain);
    }
    __syncwarp();
    volatile int local_abort = 0;
    ptx::mbar_wait_bounded(drain, 0, &local_abort, kWaitNs);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue warps
    const int q = warp & 3, row = 32 * q + lane;
    const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
    const bool have = kb1 > kb0;
    uint4 res[4] = {};
    if (MODE == kForward && S == 1 && t.ok) fetch_residual<SW>(p, t, 0, row, res);
    const bool ready = ptx::mbar_wait_bounded(accf, 0, s_abort, kWaitNs);
    if (!ptx::bar_or<1, 128>(!ready) && t.ok) {
      ptx::tc_fence_after();
      float bias[4];
      lane_bias<MODE, SW>(p, t, row, bias);
      if (S == 1) {
        for (int c0 = 0; c0 < t.nw; c0 += 32) {
          uint32_t v[32];
          load_acc(acc + c0, have, v);
          finish<MODE, SW, BF>(p, t, v, bias, c0, row, smem + C::EPI_OFF, 2, res, c0 + 32);
        }
      }
    }
  }

  __syncthreads();
  if (*s_abort && threadIdx.x == 0) set_status(p.status, MOE_ERR_TIMEOUT);
  if (S > 1) {
    // The cluster's partial tiles meet over distributed shared memory: CTA r finishes its share
    // of the columns, whose partials every CTA sends it by one bulk copy (loads or stores by the
    // threads took up to 30 us here).  The sum runs in rank order, so that it does not depend
    // on timing.
    const int row = 32 * (warp & 3) + lane;
    const int per = ((t.nw + S - 1) / S + 7) / 8 * 8;   // columns per CTA, in groups of 8
    auto share = [&](int r) { return max(0, min((r + 1) * per, (t.nj + 7) / 8 * 8) - r * per); };   // columns of CTA r
    // partials by column group and thread, 8 fragment values each: [nw / 8][2][128] and
    // [S][per / 8][2][128] pieces of 16 bytes
    float4* src = reinterpret_cast<float4*>(smem);
    float4* dst = reinterpret_cast<float4*>(smem + C::SEND_BYTES);
    if (warp >= 2 && t.ok) {
      const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
      for (int c0 = 0; c0 < t.nj; c0 += 32) {
        uint32_t v[32];
        load_acc(acc + c0, kb1 > kb0, v);
        const float* f = reinterpret_cast<const float*>(v);
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            src[((c0 / 8 + g) * 2 + h) * 128 + row] = make_float4(f[16 * h + 4 * g], f[16 * h + 4 * g + 1],
                                                                f[16 * h + 4 * g + 2], f[16 * h + 4 * g + 3]);
      }
      ptx::fence_proxy_async_smem();   // the copies read what the threads wrote
    }
    if (threadIdx.x == 0 && t.ok) ptx::mbar_arrive_expect_tx(redf, (uint32_t)(S * share(rank) * 512));
    ptx::cluster_sync();   // every CTA is done with its stages and expects its copies
    if (warp == 0 && t.ok) {
      if (ptx::elect_one()) {
        for (int r = 0; r < S; ++r) {
          const int n = share(r);
          if (n > 0)
            ptx::bulk_copy_cluster(ptx::mapa_shared(dst + rank * per * 32, r), src + r * per * 32, (uint32_t)n * 512,
                                   ptx::mapa_shared(redf, r));
        }
      }
      __syncwarp();
    }
    if (warp >= 2 && t.ok) {
      const int c1 = min((rank + 1) * per, t.nj);
      LinTile part = t;
      part.nj = c1;
      uint4 res[4] = {};
      if (MODE == kForward) fetch_residual<SW>(p, part, rank * per, row, res);
      // With a flag of its own: every CTA sends whether or not its pipeline timed out, and the copies
      // into this one have to have landed before the last barrier below lets it and its peers go.
      volatile int late = 0;
      ptx::mbar_wait_cluster_bounded(redf, 0, &late, kWaitNs);
      if (!ptx::bar_or<1, 128>(late || *s_abort)) {
        float bias[4];
        lane_bias<MODE, SW>(p, t, row, bias);
        for (int c0 = rank * per; c0 < c1; c0 += 32) {
          // One rank's 32 columns at a time, in straight-line code: a loop over the ranks inside
          // each column ran cold instructions column by column, 17 us for 32 of them.  Columns past
          // the share read what lies there and are not stored.
          float sum[32];
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) sum[c] = 0.f;
#pragma unroll 1
          for (int r = 0; r < S; ++r) {
            const float4* q = dst + ((r * per + c0 - rank * per) / 8) * 256 + row;
#pragma unroll
            for (int k = 0; k < 8; ++k) {   // (g, h) = (k / 2, k % 2)
              const float4 w = q[k * 128];
              const int i = 16 * (k & 1) + 4 * (k >> 1);
              sum[i] += w.x;
              sum[i + 1] += w.y;
              sum[i + 2] += w.z;
              sum[i + 3] += w.w;
            }
          }
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(sum[c]);
          finish<MODE, SW, BF>(p, part, v, bias, c0, row, smem + C::EPI_OFF, 2, res, c0 + 32);
        }
      } else {
        set_status(p.status, MOE_ERR_TIMEOUT);
      }
    }
    ptx::cluster_sync();   // no CTA leaves while its copies are under way
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------ pair kernel
// Large products: persistent CTA pairs (cta_group::2, one MMA of M = 256 over two SMs), tiles of
// 256 i x at most 256 j (SwiGLU: in each CTA 64 gate and the matching 64 up features).  Each CTA
// holds its 128 rows of A and half of B's rows, so a pair moves half the bytes into shared memory
// per multiply-add that two single CTAs would.  The
// accumulator is double-buffered in TMEM: the epilogue of a tile runs under the next tile's MMAs.
// B's maps with boxes of 32, 64, 96 and 128 rows (kWeightGrad: one map).
struct BMaps {
  CUtensorMap m[4];
};

template <int MODE>
struct PairCfg {
  static constexpr bool A_MN = MODE != kForward, B_MN = MODE == kWeightGrad;
  static constexpr int NB = 256;                        // widest tile along j
  static constexpr int A_PANEL = 128 * 128;
  static constexpr int B_BYTES = NB / 2 * 128;          // this CTA's half of B
  static constexpr int STAGE = A_PANEL + B_BYTES;
  static constexpr int S = 6;
  static constexpr int STEP = 32;                       // tile widths along j: two halves of 16 rows
  static constexpr int EPI_WARPS = 8;
  static constexpr int B_WARP = 2 + EPI_WARPS;          // A's copies, MMA, epilogue, B's copies
  static constexpr int THREADS = 32 * (3 + EPI_WARPS);
  static constexpr int BAR_BYTES = 8 * (2 * S + 5) + 16;
  static constexpr int SMEM = S * STAGE + 2 * kEpiBytes + BAR_BYTES + (int)sizeof(RowTable) + 1024 /* align slack */;
  static_assert(SMEM <= 227 * 1024 && S >= 4, "shared memory of one CTA per SM");
};

template <int MODE, bool SW, bool BF>
__global__ void __launch_bounds__(PairCfg<MODE>::THREADS, 1)
    lin_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ BMaps tm_b,
                    const __grid_constant__ TailMaps tails, const LinParams p) {
  using C = PairCfg<MODE>;
  pdl_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi = smem + C::S * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + 2 * kEpiBytes);   // (the leader's: both CTAs' copies landed)
  uint64_t* sfree = full + C::S;     // stage consumed
  uint64_t* accf = sfree + C::S;     // [2] accumulator ready
  uint64_t* acce = accf + 2;         // [2] (the leader's) accumulator read by both CTAs' epilogues
  uint64_t* drain = acce + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  RowTable* tab = reinterpret_cast<RowTable*>(s_tmem + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kIW = SW ? 128 : 256;   // columns of out per tile
  const int rank = (int)ptx::cluster_ctarank();
  const uint32_t unit0 = blockIdx.x / 2, units = gridDim.x / 2;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < C::S; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&sfree[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&accf[b], 1);
      ptx::mbar_init(&acce[b], 2 * C::EPI_WARPS);
    }
    ptx::mbar_init(drain, 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_a);
    for (int m = 0; m < (MODE == kWeightGrad ? 1 : 4); ++m) ptx::prefetch_tensormap(&tm_b.m[m]);
  }
  build_table<MODE>(p, tab, C::STEP);
  pdl_wait();   // (as in the split kernel, before the tensor memory)
  if (warp == 1) {
    ptx::tmem_alloc_pair(s_tmem, 512);
    ptx::tmem_relinquish_pair();
    ptx::tc_fence_before();
  }
  ptx::cluster_sync();   // the peer's copies, commits and arrivals find initialized barriers
  ptx::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t n_items = tab->items;

  if (warp == 0 || warp == C::B_WARP) {
    // ---------------------------------------------------------------- producers (each CTA its share)
    // One warp copies A, another B: a stage's copies are then issued side by side, each operand
    // by as few copies as its layout allows (B in boxes of 64 rows instead of 128: 8% slower).
    const bool is_a = warp == 0;
    int g = 0;
    bool stop = false, withheld = false;
    for (uint32_t item = unit0; item < n_items && !stop; item += units) {
      const LinTile t = table_tile<MODE>(p, tab, item, C::STEP, kIW);
      const int kb_all = tile_blocks<MODE>(p, t), half = t.nw / 2;
      const int boxes = (half + 31) / 32;   // B's rows in units of 32, as one copy
      const bool narrow = half <= 64;       // (kWeightGrad: one or two 64-wide copies)
      const uint32_t bytes = 2 * (C::A_PANEL + (MODE != kWeightGrad ? 4096 * boxes : narrow ? 8192 : 16384));
      const CUtensorMap* map_b = &tm_b.m[MODE == kWeightGrad ? 0 : boxes - 1];
      const int i0 = t.i0 + kIW / 2 * rank, j0 = t.j0 + half * rank;
      for (int kb = 0; kb < kb_all; ++kb, ++g) {
        const int s = g % C::S;
        bool ok = true;
        if (g >= C::S) ok = ptx::mbar_wait_bounded(&sfree[s], (uint32_t)(g / C::S - 1) & 1, s_abort, kWaitNs);
        if (!__all_sync(0xffffffffu, ok)) {
          stop = true;
          break;
        }
        if (p.inject_timeout && unit0 == 0 && g == 0) {
          withheld = true;   // test hook: this stage never fills
          continue;
        }
        if (ptx::elect_one()) {
          uint8_t* a = smem + s * C::STAGE;
          uint8_t* b = a + C::A_PANEL;
          const uint32_t bar = ptx::mapa_shared(&full[s], 0);
          const int c = kb * kBK;
          RowBlock r = {};
          if (MODE == kWeightGrad) r = weight_block(p.win, t.c0, t.clen, kb);
          if (is_a) {
            if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], bytes);
            if (MODE == kForward) {
              if (SW) ptx::tma_load_3d_pair(a, &tm_a, c, i0, 2 * t.e, bar);
              else ptx::tma_load_2d_pair(a, &tm_a, c, t.e * p.a_rows + i0, bar);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (MODE == kInputGrad) ptx::tma_load_3d_pair(a + h * 8192, &tm_a, i0 + 64 * h, c, t.e, bar);
                else ptx::tma_load_3d_pair(a + h * 8192, r.map == 0 ? &tm_a : &tails.a[r.map - 1], i0 + 64 * h, r.d1, r.d2, bar);
              }
            }
          } else if (MODE == kWeightGrad) {
            const CUtensorMap* map = r.map == 0 ? map_b : &tails.b[r.map - 1];
            ptx::tma_load_3d_pair(b, map, j0, r.d1, r.d2, bar);
            if (!narrow) ptx::tma_load_3d_pair(b + 8192, map, j0 + 64, r.d1, r.d2, bar);
          } else {
            ptx::tma_load_2d_pair(b, map_b, c, j0, bar);
          }
        }
        __syncwarp();
      }
    }
    // both CTAs' copies complete on the leader's barriers: it waits (bounded) for the last fill
    // of every slot, and the cluster barrier at the end holds the peer until it has
    if (rank == 0) {
      volatile int local_abort = 0;
      for (int q = (g > C::S ? g - C::S : 0); q < g; ++q) {
        if (withheld && q == 0) continue;
        ptx::mbar_wait_bounded(&full[q % C::S], (uint32_t)(q / C::S) & 1, &local_abort, kWaitNs);
      }
    } else if (stop) {
      // After a timeout the leader may have stopped at an earlier stage than this CTA, whose last
      // copies nobody then counts: it stays until they have long landed (they take microseconds).
      const uint64_t t0 = ptx::globaltimer_ns();
      while (ptx::globaltimer_ns() - t0 < kLandNs) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (the leader's)
    if (rank == 0) {
      constexpr uint64_t kStepA = C::A_MN ? 2048 >> 4 : 32 >> 4, kStepB = C::B_MN ? 2048 >> 4 : 32 >> 4;
      int g = 0;
      int li = 0;
      bool stop = false;
      for (uint32_t item = unit0; item < n_items && !stop; item += units, ++li) {
        const LinTile t = table_tile<MODE>(p, tab, item, C::STEP, kIW);
        const int kb_all = tile_blocks<MODE>(p, t), b2 = li & 1;
        const uint32_t idesc = ptx::idesc_f16(BF, 256, t.nw, C::A_MN, C::B_MN);
        if (li >= 2 && !__all_sync(0xffffffffu, ptx::mbar_wait_cluster_bounded(
                                                    &acce[b2], (uint32_t)((li >> 1) - 1) & 1, s_abort, kWaitNs)))
          break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + b2 * 256;
        for (int kb = 0; kb < kb_all; ++kb, ++g) {
          const int s = g % C::S;
          if (!__all_sync(0xffffffffu,
                          ptx::mbar_wait_bounded(&full[s], (uint32_t)(g / C::S) & 1, s_abort, kWaitNs))) {
            stop = true;
            break;
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint8_t* a = smem + s * C::STAGE;
            const uint8_t* b = a + C::A_PANEL;
            const uint64_t da = C::A_MN ? ptx::smem_desc_mn_sw128(a) : ptx::smem_desc_k_sw128(a);
            const uint64_t db = C::B_MN ? ptx::smem_desc_mn_sw128(b) : ptx::smem_desc_k_sw128(b);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_f16_ss_pair(d, da + k * kStepA, db + k * kStepB, idesc, (kb | k) != 0);
            ptx::tc_commit_pair(&sfree[s], (uint16_t)3);
          }
          __syncwarp();
        }
        if (!stop && ptx::elect_one()) ptx::tc_commit_pair(&accf[b2], (uint16_t)3);
        __syncwarp();
      }
      if (ptx::elect_one()) ptx::tc_commit_pair(drain, (uint16_t)3);
      __syncwarp();
    }
    volatile int local_abort = 0;
    ptx::mbar_wait_bounded(drain, 0, &local_abort, kWaitNs);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue warps
    const int q = warp & 3, row = 32 * q + lane, part = (warp - 2) >> 2;
    int li = 0;
    for (uint32_t item = unit0; item < n_items; item += units, ++li) {
      LinTile t = table_tile<MODE>(p, tab, item, C::STEP, kIW);
      t.i0 += kIW / 2 * rank;
      const int b2 = li & 1;
      const bool have = t.clen > 0;
      float bias[4];
      lane_bias<MODE, SW>(p, t, row, bias);
      uint4 res[4] = {};
      if (MODE == kForward) fetch_residual<SW>(p, t, 32 * part, row, res);
      const bool ready = !*s_abort && ptx::mbar_wait_bounded(&accf[b2], (uint32_t)(li >> 1) & 1, s_abort, kWaitNs);
      // (one answer for all epilogue warps: another role may raise the abort flag at any time)
      if (ptx::bar_or<1, 32 * C::EPI_WARPS>(!ready)) break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + b2 * 256;
      auto release = [&] {   // this warp's reads are done: one arrival on the leader's barrier
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(&acce[b2], 0));
      };
      if (32 * part >= t.nw) release();
      for (int c0 = 32 * part; c0 < t.nw; c0 += 64) {
        uint32_t v[32];
        load_acc(acc + c0, have, v);   // (an expert without rows: never written)
        if (c0 + 64 >= t.nw) release();
        finish<MODE, SW, BF>(p, t, v, bias, c0, row, epi + kEpiBytes * part, 2 + part, res, c0 + 64);
      }
    }
  }

  __syncthreads();
  if (*s_abort && threadIdx.x == 0) set_status(p.status, MOE_ERR_TIMEOUT);
  // the leader has seen every copy of both CTAs land and the MMAs complete before either CTA
  // frees its TMEM and exits
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------------------ token kernel
// A dense forward product of at most 16 rows: nothing but the weights' stream, where the set-up of
// the tiles (tensor memory, barriers, the cluster's join) took most of the time.  A block takes 16
// output features (SwiGLU: 8 gate and the 8 up), its 8 warps share the contraction in steps of 32,
// each lane loads 16 bytes of two weight rows and of NT token rows straight into the fragments of
// m16n8k16 MMAs, U steps at a time (what the registers of two blocks an SM hold; 4 steps at one
// token column took 5.9 us for 4096 x 4096, 6 took 6.7, 8 take 5.5), and the warps' sums meet in
// shared memory in warp order.  Lane l / 4 has a row, lane l % 4 the values 8 (l % 4) .. + 7 of a
// step: the first half of them stands for the fragments' k 2 (l % 4), + 1, + 8, + 9 of one MMA, the
// second half for the next; A and B permute k alike, which a sum does not see.
struct TokenParams {
  int32_t M, K, N, I, fn;
  float limit;
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* w;
  const float* bias;
  const uint16_t* residual;
  int64_t ld_res;
  uint16_t* y;
  int64_t ldy;
  uint16_t* z;
};

template <bool BF>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool SW, int NT, bool BF>
__global__ void __launch_bounds__(256, 2) lin_token_kernel(const TokenParams p) {
    constexpr int U = NT == 1 ? 8 : 4, TOK = 8 * NT;
  __shared__ float s_sum[8][16][TOK + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int f0 = blockIdx.x * (SW ? 8 : 16);
  const int rows = SW ? p.I : p.N;                     // output features
  const bool has0 = f0 + g < rows, has1 = SW ? has0 : f0 + 8 + g < rows;
  const uint16_t* w0 = p.w + (int64_t)(has0 ? f0 + g : 0) * p.K;
  const uint16_t* w1 = p.w + (int64_t)(has1 ? (SW ? p.I + f0 + g : f0 + 8 + g) : 0) * p.K;
  float c[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) c[t][r] = 0.f;
  const int steps = (p.K + 31) / 32;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int s0 = warp; s0 < steps; s0 += 8 * U) {
    uint4 a0[U], a1[U], b[U][NT];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = 32 * (s0 + 8 * i) + 8 * q;         // (K is a multiple of 8)
      const bool in = k < p.K;
      a0[i] = in && has0 ? __ldg(reinterpret_cast<const uint4*>(w0 + k)) : zero;
      a1[i] = in && has1 ? __ldg(reinterpret_cast<const uint4*>(w1 + k)) : zero;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        b[i][t] = in && 8 * t + g < p.M ? __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(8 * t + g) * p.ldx + k)) : zero;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_16816<BF>(c[t], a0[i].x, a1[i].x, a0[i].y, a1[i].y, b[i][t].x, b[i][t].y);
        mma_16816<BF>(c[t], a0[i].z, a1[i].z, a0[i].w, a1[i].w, b[i][t].z, b[i][t].w);
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    s_sum[warp][g][8 * t + 2 * q] = c[t][0];
    s_sum[warp][g][8 * t + 2 * q + 1] = c[t][1];
    s_sum[warp][g + 8][8 * t + 2 * q] = c[t][2];
    s_sum[warp][g + 8][8 * t + 2 * q + 1] = c[t][3];
  }
  __syncthreads();
  constexpr int F = SW ? 8 : 16;
  for (int i = threadIdx.x; i < F * TOK; i += 256) {
    const int f = i % F, tok = i / F, col = f0 + f;    // a token's features side by side
    if (col >= rows || tok >= p.M) continue;
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      v += s_sum[w][f][tok];
      if (SW) u += s_sum[w][f + 8][tok];
    }
    if (p.bias) {
      v += __ldg(p.bias + col);
      if (SW) u += __ldg(p.bias + p.I + col);
    }
    if (p.z) {
      uint16_t* z = p.z + (int64_t)tok * p.N + col;
      z[0] = to16<BF>(v);
      if (SW) z[p.I] = to16<BF>(u);
    }
    float y = v, other = 0.f;
    if (SW) {
      y = swiglu(v, u, p.limit);
    } else {
      switch (p.fn) {
        case MOE_FN_RELU: y = act_fn<MOE_FN_RELU>(v); break;
        case MOE_FN_GELU: act_pair<MOE_FN_GELU>(y, other); break;
        case MOE_FN_GELU_TANH: y = act_fn<MOE_FN_GELU_TANH>(v); break;
        case MOE_FN_SILU: y = act_fn<MOE_FN_SILU>(v); break;
      }
    }
    if (p.residual) y += from16<BF>(p.residual[(int64_t)tok * p.ld_res + col]);
    p.y[(int64_t)tok * p.ldy + col] = to16<BF>(y);
  }
}

// ------------------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// Map of 16-bit values, 128-byte swizzle, boxes of 64 values x box1 x box2; strides in values.
bool map16(CUtensorMap* m, bool bf16, const void* base, int rank, uint64_t d0, uint64_t d1, uint64_t s1, uint64_t d2,
           uint64_t s2, uint32_t box1, uint32_t box2 = 1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {2 * s1, 2 * s2};
  const cuuint32_t box[3] = {64, box1, box2}, es[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map `map` of a weight gradient's operand.
bool row_windows(CUtensorMap* m, bool bf16, const void* base, uint64_t values, int32_t rows, int64_t ld, int map) {
  const uint64_t w = window_rows(map, rows);
  return map16(m, bf16, base, 3, values, w, ld, (uint64_t)rows - w + 1, ld, kBK);
}
// (A dense product's only tail ends with the buffer: map 0 serves it.)
bool tail_maps(const LinArgs& a, TailMaps* t) {
  if (a.mode != kWeightGrad || !a.offsets) return true;
  const bool bf = a.bf16 != 0;
  for (int k = 0; k < 2; ++k)
    if (!row_windows(&t->a[k], bf, a.other, a.K, a.rows, a.ld_other, k + 1) ||
        !row_windows(&t->b[k], bf, a.tok, a.N, a.rows, a.ld_tok, k + 1))
      return false;
  return true;
}

// The map of A: 128 rows per copy of a K-major one (SwiGLU: 64 gate and the 64 matching up
// rows), 64 x 64 boxes of an MN-major one.
bool a_map(const LinArgs& a, CUtensorMap* m) {
  const bool bf = a.bf16 != 0;
  const uint64_t K = a.K, N = a.N, E = a.E, rows = a.rows;
  switch (a.mode) {
    case kForward:
      if (a.fn == MOE_FN_SWIGLU)   // W [E * 2][N / 2][K]
        return map16(m, bf, a.other, 3, K, N / 2, K, 2 * E, N / 2 * K, 64, 2);
      return map16(m, bf, a.other, 2, K, E * N, K, 1, 0, 128);   // W [E * N][K]
    case kInputGrad:   // W [E][N][K] (rows past an expert's N read zeros)
      return map16(m, bf, a.other, 3, K, N, K, E, N * K, 64);
    default:
      return row_windows(m, bf, a.other, K, a.rows, a.ld_other, 0);
  }
}

// The map of B, `box` rows per copy of a K-major one.
bool b_map(const LinArgs& a, uint32_t box, CUtensorMap* m) {
  const bool bf = a.bf16 != 0;
  const uint64_t rows = a.rows;
  if (a.mode == kWeightGrad) return row_windows(m, bf, a.tok, (uint64_t)a.N, a.rows, a.ld_tok, 0);
  return map16(m, bf, a.tok, 2, (uint64_t)(a.mode == kForward ? a.K : a.N), rows, a.ld_tok, 1, 0, box);
}

// Kernels' dynamic shared memory limit, set once per device.
template <class K>
bool allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev < 64) done.fetch_or(bit, std::memory_order_release);
  return true;
}

LinParams params_of(const LinArgs& a, int iw) {
  LinParams p = {};
  const int No = a.fn == MOE_FN_SWIGLU ? a.N / 2 : a.N;
  p.rows = a.rows;
  p.E = a.E;
  p.fn = a.fn;
  p.limit = a.limit;
  p.I = a.mode == kForward ? No : a.K;
  p.J = a.N;
  p.C = a.mode == kForward ? a.K : a.N;
  p.a_rows = a.N;
  p.win = window_rows(0, a.rows);
  p.n_it = (p.I + iw - 1) / iw;
  p.offsets = a.offsets;
  p.out = static_cast<uint16_t*>(a.out);
  p.ld_out = a.mode == kWeightGrad ? a.K : a.ld_out;
  p.out_expert = a.mode == kWeightGrad ? (int64_t)a.N * a.K : 0;
  p.bias = a.bias;
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.ld_res = a.ld_res;
  p.z = static_cast<uint16_t*>(a.z);
  p.status = a.status;
  p.inject_timeout = a.inject_timeout;
  const int64_t out_n = a.mode == kWeightGrad ? (int64_t)a.E * a.N * a.K : (int64_t)(a.rows - 1) * a.ld_out + p.I;
  p.out_end = p.out + out_n;
  p.z_end = p.z ? p.z + (int64_t)a.rows * a.N : nullptr;
  return p;
}

// Most token tiles of at most nw rows that `rows` rows of E experts can make.
int64_t row_tiles_bound(const LinArgs& a, int nw) {
  if (!a.offsets) return (a.rows + nw - 1) / nw;
  const int64_t used = std::min(a.E, a.rows);
  return (a.rows - used) / nw + used;
}

template <int MODE, bool SW, int NB, bool BF>
int launch_split_of(const LinArgs& a) {
  using C = SplitCfg<MODE, NB>;
  CUtensorMap ma, mb;
  TailMaps tails = {};
  if (!a_map(a, &ma) || !b_map(a, NB, &mb) || !tail_maps(a, &tails)) return -1;
  LinParams p = params_of(a, SW ? 64 : 128);
  p.nw_max = NB;
  p.n_jt = (a.N + NB - 1) / NB;
  const int64_t tiles = (MODE == kWeightGrad ? (int64_t)a.E * p.n_jt : row_tiles_bound(a, NB)) * p.n_it;
  // Fewer tiles than SMs: a cluster of up to four CTAs shares each tile's contraction (1 x 2880 x
  // 2880: 15.0 / 11.2 / 9.0 / 9.6 us with 1 / 2 / 4 / 6), each keeping at least five 64-wide blocks
  // of it (192-wide contractions: 5 us alone, 7 us shared), while the CTAs stay within 1.25 per
  // SM (128 x 2880 x 2880, 46 tiles: 12.7 us with 3, 19.4 us with 6: the clusters then queue).
  const int64_t blocks = MODE == kWeightGrad ? (a.rows / (a.offsets ? a.E : 1) + kBK - 1) / kBK : (p.C + kBK - 1) / kBK;
  const int64_t s = std::min<int64_t>(5 * (int64_t)multiprocessors() / (4 * tiles), blocks / 5);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(s, 4));
  auto kern = lin_split_kernel<MODE, SW, NB, BF>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(kern, C::SMEM, done)) return -1;
  const int64_t grid = tiles * p.splits;
  if (grid > 0x7fffffff) return -1;
  const dim3 g((unsigned)grid), b(C::THREADS);
  const cudaError_t err = p.splits == 1
      ? launch_kernel(kern, g, b, C::SMEM, a.stream, a.pdl != 0, ma, mb, tails, p)
      : launch_kernel_cluster(kern, g, b, C::SMEM, a.stream, a.pdl != 0, (unsigned)p.splits, ma, mb, tails, p);
  return err == cudaSuccess ? 1 : -1;
}

// Width of a pair's tiles along j: the one whose turns on `pairs` pairs take least.  A stage of a
// w-wide tile takes the longer of its MMAs (2 w cycles) and its copies (128 rows of A and w / 2 of
// B, 2 cycles a row), a turn about 96 cycles a stage more (its epilogue's share).  1024 x 2880 x
// 5760: 92 tiles of 256 are two turns of 74 pairs (33.6 us), 138 of 192 are two as well (30.6 us).
// Ragged rows: 256.
int pair_width(const LinArgs& a, int n_it, int pairs) {
  if (a.offsets && a.mode != kWeightGrad) return 256;
  const int64_t J = a.mode == kWeightGrad ? a.N : a.rows, experts = a.mode == kWeightGrad ? a.E : 1;
  int best = 256;
  int64_t least = -1;
  for (int w = 256; w >= 64; w -= 32) {
    const int64_t tiles = experts * ((J + w - 1) / w) * n_it, cost = (tiles + pairs - 1) / pairs * (std::max(2 * w, 256 + w) + 96);
    if (least < 0 || cost < least) {
      least = cost;
      best = w;
    }
  }
  return best;
}

// Clusters of two CTAs of `kern` that the device holds at once, remembered per device.
template <class K>
int pair_slots(K kern, int threads, int smem, std::atomic<int>* known) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_acquire)) > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * multiprocessors());
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (dev < 64) known[dev].store(n, std::memory_order_release);
  return n;
}

template <int MODE, bool SW, bool BF>
int launch_pair_of(const LinArgs& a) {
  using C = PairCfg<MODE>;
  CUtensorMap ma;
  BMaps mb;
  TailMaps tails = {};
  if (!a_map(a, &ma) || !tail_maps(a, &tails)) return -1;
  for (uint32_t m = 0; m < (MODE == kWeightGrad ? 1 : 4); ++m)
    if (!b_map(a, 32 * (m + 1), &mb.m[m])) return -1;
  LinParams p = params_of(a, SW ? 128 : 256);
  p.splits = 1;
  auto kern = lin_pair_kernel<MODE, SW, BF>;
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> slots[64];
  if (!allow_smem(kern, C::SMEM, done)) return -1;
  const int n = pair_slots(kern, C::THREADS, C::SMEM, slots);
  if (n <= 0) return -1;
  p.nw_max = pair_width(a, p.n_it, n);
  p.n_jt = (a.N + p.nw_max - 1) / p.nw_max;
  const int64_t tiles = (MODE == kWeightGrad ? (int64_t)a.E * p.n_jt : row_tiles_bound(a, p.nw_max)) * p.n_it;
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(tiles, n);
  return launch_kernel_cluster(kern, dim3(grid), dim3(C::THREADS), C::SMEM, a.stream, a.pdl != 0, 2u, ma, mb, tails,
                               p) ==
                 cudaSuccess ? 1 : -1;
}

template <int MODE, bool SW = false>
int launch_pair(const LinArgs& a) {
  return a.bf16 ? launch_pair_of<MODE, SW, true>(a) : launch_pair_of<MODE, SW, false>(a);
}
template <int MODE, bool SW, int NB>
int launch_split(const LinArgs& a) {
  return a.bf16 ? launch_split_of<MODE, SW, NB, true>(a) : launch_split_of<MODE, SW, NB, false>(a);
}

template <bool SW, int NT>
int launch_token(const LinArgs& a) {
  TokenParams p = {};
  p.M = a.rows;
  p.K = a.K;
  p.N = a.N;
  p.I = SW ? a.N / 2 : a.N;
  p.fn = a.fn;
  p.limit = a.limit;
  p.x = static_cast<const uint16_t*>(a.tok);
  p.ldx = a.ld_tok;
  p.w = static_cast<const uint16_t*>(a.other);
  p.bias = a.bias;
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.ld_res = a.ld_res;
  p.y = static_cast<uint16_t*>(a.out);
  p.ldy = a.ld_out;
  p.z = static_cast<uint16_t*>(a.z);
  auto kern = a.bf16 ? lin_token_kernel<SW, NT, true> : lin_token_kernel<SW, NT, false>;
  const int f = SW ? 8 : 16;
  return launch_kernel(kern, dim3((unsigned)((p.I + f - 1) / f)), dim3(256), 0, a.stream, false, p) == cudaSuccess ? 1 : -1;
}
template <bool SW>
int launch_tokens(const LinArgs& a) {
  return a.rows <= 8 ? launch_token<SW, 1>(a) : launch_token<SW, 2>(a);
}

// Tiles of 256 x 256 that the product makes (on average over the experts' counts).
int64_t pair_tiles(const LinArgs& a) {
  constexpr int nw = 256;
  const int64_t I = a.mode == kForward ? a.N : a.K;
  const int64_t j = a.mode == kWeightGrad ? a.E * (int64_t)((a.N + nw - 1) / nw)
                    : a.offsets           ? std::min<int64_t>(a.E, a.rows) * ((a.rows / a.E + nw - 1) / nw)
                                          : (a.rows + nw - 1) / nw;
  return j * ((I + 255) / 256);
}

}  // namespace

int launch_linear(const LinArgs& a) {
  const bool swiglu = a.mode == kForward && a.fn == MOE_FN_SWIGLU;
  // A few tokens: the kernel without tiles, until its many blocks cost more than the tiles' set-up.
  // Times in us, this kernel against the split tiles, weights K x N: 1 row 2880 x 2880 4.7 : 9.0,
  // 4096 x 16384 24 : 28, 2880 x 32768 36 : 33; 16 rows 2880 x 2880 6.3 : 9.2, 8192 x 8192 28 : 30,
  // 4096 x 16384 32 : 28; 24 rows 2880 x 2880 12 : 9.3.
  if (a.mode == kForward && !a.offsets && a.rows <= 16 && a.N <= (a.rows <= 8 ? 16384 : 8192))
    return swiglu ? launch_tokens<true>(a) : launch_tokens<false>(a);
  const bool narrow = a.rows / (a.offsets ? a.E : 1) <= 32;   // rows an expert: the weights' stream is the work
  // CTA pairs once their tiles fill about half of the SMs; fewer tiles: smaller ones on more SMs,
  // with clusters that share a contraction.
  const bool pair = pair_tiles(a) >= multiprocessors() / 4 && (a.mode == kWeightGrad || !narrow);
  switch (a.mode) {
    case kForward:
      if (swiglu)
        return pair     ? launch_pair<kForward, true>(a)
               : narrow ? launch_split<kForward, true, 32>(a)
                        : launch_split<kForward, true, 64>(a);
      return pair     ? launch_pair<kForward>(a)
             : narrow ? launch_split<kForward, false, 32>(a)
                      : launch_split<kForward, false, 64>(a);
    case kInputGrad:
      return pair     ? launch_pair<kInputGrad>(a)
             : narrow ? launch_split<kInputGrad, false, 32>(a)
                      : launch_split<kInputGrad, false, 64>(a);
    default:
      return pair ? launch_pair<kWeightGrad>(a) : launch_split<kWeightGrad, false, 64>(a);
  }
}

// ------------------------------------------------------------------------------ activation gradient
// dz = dy f'(z) and the column sums db of dz, in one pass over dy and z.  A block takes a chunk
// of kChunk rows of one expert and 256 columns of dy, 8 per lane; its 8 warps take rows in turn and
// add their column sums in a fixed order into one row of `partial`, which sum_chunks_kernel
// adds up per expert.  The sums take dz before its rounding to 16 bits.  GELU (two exponentials, a
// divide and a polynomial a value) runs on its arithmetic: 4099 x 4096 30 us with 67% of the issue
// slots and 28% of HBM's cycles in use; SwiGLU 4096 x 5760 25 us, 60% and 37%.
namespace {
constexpr int kChunk = 64;

__device__ __forceinline__ float from16r(uint16_t v, bool bf) { return bf ? from16<true>(v) : from16<false>(v); }

struct ActGradParams {
  int32_t rows, N, No, E, bf16, fn, chunks;
  float limit;
  const int32_t* offsets;
  const uint16_t* dy;
  int64_t ld_dy;
  const uint16_t* z;
  uint16_t* dz;
  float* partial;
  float* db;
  int32_t* status;
};

template <int FN>
__device__ __forceinline__ float act_grad(float z, float dy) {
  if (FN == MOE_FN_RELU) return z > 0.f ? dy : 0.f;
  if (FN == MOE_FN_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return dy * s * (1.f + z * (1.f - s));
  }
  if (FN == MOE_FN_GELU_TANH) {   // s = (1 + tanh v) / 2, (1 - tanh^2 v) / 2 = 2 s (1 - s)
    // (past 16 the second term is 0: there z^2 may overflow, and infinity times 0 is no slope)
    const float s = __fdividef(1.f, 1.f + __expf(-2.f * gelu_arg(z))), c = fminf(fmaxf(z, -16.f), 16.f);
    return dy * (s + 2.f * c * s * (1.f - s) * 0.79788456f * (1.f + 0.134145f * c * c));
  }
  return dy;
}

// Chunk q of the ragged rows -> (expert, first row, rows); one warp, as find_row_tile.
__device__ __forceinline__ bool find_chunk(const ActGradParams& p, int q, int& e, int& r0, int& n) {
  LinParams lp;
  lp.rows = p.rows;
  lp.E = p.E;
  lp.offsets = p.offsets;
  lp.n_it = 1;
  lp.nw_max = kChunk;
  lp.C = 0;
  lp.status = p.status;
  const LinTile t = find_row_tile(lp, q, kChunk, 0);
  e = t.e;
  r0 = t.j0;
  n = t.nj;
  return t.ok != 0;
}

// Eight values of dz from those of dy and z (SwiGLU: d_g and d_u from g and u).
template <int FN>
__device__ __forceinline__ void act_grad8(const ActGradParams& p, const float (&z)[8], const float (&u)[8],
                                          const float (&dy)[8], float (&o)[8], float (&ou)[8]) {
  if constexpr (FN == MOE_FN_GELU) {   // Phi(z) + z phi(z)
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float c0, c1, e0, e1;
      normal_cdf2(z[k], z[k + 1], c0, c1);
      mul2(e0, e1, z[k], z[k + 1], z[k], z[k + 1]);
      e0 = __expf(-0.5f * e0);
      e1 = __expf(-0.5f * e1);
      mul2(e0, e1, e0, e1, 0.39894228f, 0.39894228f);
      fma2(c0, c1, z[k], z[k + 1], e0, e1, c0, c1);
      mul2(o[k], o[k + 1], dy[k], dy[k + 1], c0, c1);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (FN == MOE_FN_SWIGLU) {
        const float g = clamp_hi(z[k], p.limit), uc = clamp_both(u[k], p.limit);
        const float s = __fdividef(1.f, 1.f + __expf(-g)), gs = g * s;
        o[k] = z[k] > p.limit ? 0.f : dy[k] * uc * (s + gs * (1.f - s));
        ou[k] = fabsf(u[k]) <= p.limit ? dy[k] * gs : 0.f;
      } else {
        o[k] = act_grad<FN>(z[k], dy[k]);
      }
    }
  }
}

__device__ __forceinline__ void widen(const uint4& q, bool bf, float (&f)[8]) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(&q);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = from16r(h[k], bf);
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8], bool bf) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = bf ? to16x2<true>(f[2 * k], f[2 * k + 1]) : to16x2<false>(f[2 * k], f[2 * k + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Threads: 32 lanes of 8 columns of dy (SwiGLU: the gate and the up column both), 8 warps of rows;
// two rows of a warp are loaded together.
template <int FN>
__global__ void __launch_bounds__(256) act_grad_kernel(const ActGradParams p) {
  constexpr int H = FN == MOE_FN_SWIGLU ? 2 : 1;
  __shared__ int s_t[3];
  __shared__ float s_sum[8][256];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int e = 0, r0 = 0, n = 0;
    const bool ok = find_chunk(p, blockIdx.x, e, r0, n);
    if (lane == 0) {
      s_t[0] = ok;
      s_t[1] = r0;
      s_t[2] = n;
    }
  }
  __syncthreads();
  if (!s_t[0]) return;
  const int r0 = s_t[1], r1 = r0 + s_t[2];
  const bool bf = p.bf16 != 0;
  const int col = blockIdx.y * 256 + 8 * lane;      // of dy's columns (a multiple of 8)
  float sum[H][8];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[h][k] = 0.f;
  if (col < p.No) {
    for (int r = r0 + warp; r < r1; r += 16) {
      uint4 dv[2], zv[2], uv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = r + 8 * i;
        if (row < r1) {
          dv[i] = __ldg(reinterpret_cast<const uint4*>(p.dy + row * p.ld_dy + col));
          if (FN != MOE_FN_NONE) zv[i] = __ldg(reinterpret_cast<const uint4*>(p.z + row * p.N + col));
          if (H == 2) uv[i] = __ldg(reinterpret_cast<const uint4*>(p.z + row * p.N + p.No + col));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t row = r + 8 * i;
        if (row < r1) {
          float dy[8], z[8], u[8], o[8], ou[8];
          widen(dv[i], bf, dy);
          if (FN != MOE_FN_NONE) widen(zv[i], bf, z);
          if (H == 2) widen(uv[i], bf, u);
          act_grad8<FN>(p, z, u, dy, o, ou);
          if (FN != MOE_FN_NONE) *reinterpret_cast<uint4*>(p.dz + row * p.N + col) = narrow(o, bf);
          if (H == 2) *reinterpret_cast<uint4*>(p.dz + row * p.N + p.No + col) = narrow(ou, bf);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sum[0][k] += o[k];
            if (H == 2) sum[H - 1][k] += ou[k];
          }
        }
      }
    }
  }
  if (!p.partial) return;
  for (int h = 0; h < H; ++h) {
    if (h) __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) s_sum[warp][8 * lane + k] = h == 0 ? sum[0][k] : sum[H - 1][k];
    __syncthreads();
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c < p.No) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += s_sum[w][threadIdx.x];
      p.partial[(int64_t)blockIdx.x * p.N + h * p.No + c] = v;
    }
  }
}

// db[e][n] = the sum of expert e's chunks (none: 0), in order: 8 warps take every eighth chunk
// and their sums are added in warp order.
__global__ void __launch_bounds__(256) sum_chunks_kernel(const ActGradParams p) {
  __shared__ float s_sum[8][32];
  __shared__ int s_first;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  int a = 0, b = p.rows;
  bool bad = false;
  if (p.offsets) {
    expert_rows(p.offsets, p.rows, e, a, b, bad);
    if (warp == 0) {   // first chunk of expert e: the chunks of the experts before it
      int n = 0;
      for (int q = lane; q < e; q += 32) {
        int qa, qb;
        expert_rows(p.offsets, p.rows, q, qa, qb, bad);
        n += (qb - qa + kChunk - 1) / kChunk;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane == 0) s_first = n;
    }
  } else if (threadIdx.x == 0) {
    s_first = 0;
  }
  __syncthreads();
  pdl_wait();
  // (offsets out of order could count past the rows of `partial`)
  const int first = s_first, n = min((b - a + kChunk - 1) / kChunk, p.chunks - first), c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < p.N)
    for (int q = warp; q < n; q += 8) v += p.partial[(int64_t)(first + q) * p.N + c];
  s_sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < p.N) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += s_sum[w][lane];
    p.db[(int64_t)e * p.N + c] = t;
  }
}
}  // namespace

int64_t act_grad_chunks(int32_t rows, int32_t E) {
  const int64_t used = std::min(E, rows);
  return used + (rows - used) / kChunk;   // the most that ragged counts can make
}

int launch_act_grad(const ActGradArgs& a) {
  ActGradParams p = {};
  p.rows = a.rows;
  p.N = a.N;
  p.No = a.fn == MOE_FN_SWIGLU ? a.N / 2 : a.N;
  p.E = a.E;
  p.bf16 = a.bf16;
  p.fn = a.fn;
  p.limit = a.limit;
  p.offsets = a.offsets;
  p.dy = static_cast<const uint16_t*>(a.dy);
  p.ld_dy = a.ld_dy;
  p.z = static_cast<const uint16_t*>(a.z);
  p.dz = static_cast<uint16_t*>(a.dz);
  p.partial = a.db ? a.partial : nullptr;
  p.db = a.db;
  p.status = a.status;
  p.chunks = (int)act_grad_chunks(a.rows, a.offsets ? a.E : 1);
  const dim3 grid((unsigned)p.chunks, (unsigned)((p.No + 255) / 256));
  auto kern = act_grad_kernel<MOE_FN_NONE>;
  switch (a.fn) {
    case MOE_FN_RELU: kern = act_grad_kernel<MOE_FN_RELU>; break;
    case MOE_FN_GELU: kern = act_grad_kernel<MOE_FN_GELU>; break;
    case MOE_FN_GELU_TANH: kern = act_grad_kernel<MOE_FN_GELU_TANH>; break;
    case MOE_FN_SILU: kern = act_grad_kernel<MOE_FN_SILU>; break;
    case MOE_FN_SWIGLU: kern = act_grad_kernel<MOE_FN_SWIGLU>; break;
  }
  if (launch_kernel(kern, grid, dim3(256), 0, a.stream, false, p) != cudaSuccess) return -1;
  if (!a.db) return 1;
  if (launch_kernel(sum_chunks_kernel, dim3((unsigned)((a.N + 31) / 32), (unsigned)a.E), dim3(256), 0, a.stream, true,
                    p) != cudaSuccess)
    return -1;
  return 2;
}

}  // namespace moe
