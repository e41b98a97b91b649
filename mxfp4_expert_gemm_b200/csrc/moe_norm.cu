// The norm of a row, forward and backward, with the reduction of the weight's gradient:
//   forward   m = mean(x) (RMSNorm: 0), r = 1 / sqrt(mean((x - m)^2) + eps), y = (x - m) r w + b
//   backward  xh = (x - m) r, g = dy w,
//             dx = r (g - xh mean(g xh) - [layer norm] mean(g)) [+ dres],
//             dw = sum over rows of dy xh, db = sum over rows of dy
// Both passes are bound by HBM: a row is read once into registers (16-byte loads), its
// statistics are taken from the registers in two passes (mean first, then centred squares:
// no cancellation), and the result is written.  Sums and statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "moe_linear.cuh"
#include "packed_math.cuh"

namespace moe {
namespace {

constexpr int kMaxPartialRows = 592;   // blocks of the backward pass that keep column sums (4 per SM)

struct BF16 { using Store = uint16_t; };
struct FP16 { using Store = uint16_t; };
struct FP32 { using Store = float; };

__device__ __forceinline__ float load1(uint16_t v, BF16) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float load1(uint16_t v, FP16) { return __half2float(__ushort_as_half(v)); }
__device__ __forceinline__ float load1(float v, FP32) { return v; }
__device__ __forceinline__ uint16_t store1(float v, BF16) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ uint16_t store1(float v, FP16) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ float store1(float v, FP32) { return v; }

// VEC consecutive values, as stored: 16 bytes, or 4 (two 16-bit values), or one value.
template <class DT, int VEC>
struct alignas(VEC * sizeof(typename DT::Store)) Pack {
  typename DT::Store v[VEC];
};

template <class DT, int VEC>
__device__ __forceinline__ Pack<DT, VEC> load_pack(const void* base, int64_t at) {
  return *reinterpret_cast<const Pack<DT, VEC>*>(static_cast<const typename DT::Store*>(base) + at);
}
template <class DT, int VEC>
__device__ __forceinline__ void store_pack(void* base, int64_t at, const Pack<DT, VEC>& p) {
  *reinterpret_cast<Pack<DT, VEC>*>(static_cast<typename DT::Store*>(base) + at) = p;
}

// A pack's values in fp32 and back: two 16-bit values per 32-bit word.
template <class DT, int VEC>
__device__ __forceinline__ void unpack(const Pack<DT, VEC>& p, float (&f)[VEC]) {
  if constexpr (VEC > 1 && sizeof(typename DT::Store) == 2) {
    uint32_t w[VEC / 2];
    if constexpr (VEC == 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(&p);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(&p);
    }
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (std::is_same<DT, BF16>::value) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = load1(p.v[j], DT{});
  }
}
template <class DT, int VEC>
__device__ __forceinline__ Pack<DT, VEC> pack(const float (&f)[VEC]) {
  Pack<DT, VEC> p;
  if constexpr (VEC > 1 && sizeof(typename DT::Store) == 2) {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (std::is_same<DT, BF16>::value) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(&p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint32_t*>(&p) = w[0];
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) p.v[j] = store1(f[j], DT{});
  }
  return p;
}

// Element-wise arithmetic of a pack's values, two per instruction (the packed fp32 operations of
// sm_100; with them, and the statistics loaded a step ahead, 16384 x 2880 backward 110 -> 93 us).
template <int N>   // d = a * b + c
__device__ __forceinline__ void vfma(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
  if constexpr (N == 1) d[0] = fmaf(a[0], b[0], c[0]);
  else
#pragma unroll
    for (int j = 0; j < N; j += 2) fma2(d[j], d[j + 1], a[j], a[j + 1], b[j], b[j + 1], c[j], c[j + 1]);
}
template <int N>   // d = a * b + c with scalars b and c
__device__ __forceinline__ void vfma(float (&d)[N], const float (&a)[N], float b, float c) {
  if constexpr (N == 1) d[0] = fmaf(a[0], b, c);
  else
#pragma unroll
    for (int j = 0; j < N; j += 2) fma2(d[j], d[j + 1], a[j], a[j + 1], b, b, c, c);
}
template <int N>   // d = a * b + c with a scalar b
__device__ __forceinline__ void vfma(float (&d)[N], const float (&a)[N], float b, const float (&c)[N]) {
  if constexpr (N == 1) d[0] = fmaf(a[0], b, c[0]);
  else
#pragma unroll
    for (int j = 0; j < N; j += 2) fma2(d[j], d[j + 1], a[j], a[j + 1], b, b, c[j], c[j + 1]);
}
template <int N>
__device__ __forceinline__ void vmul(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
  if constexpr (N == 1) d[0] = a[0] * b[0];
  else
#pragma unroll
    for (int j = 0; j < N; j += 2) mul2(d[j], d[j + 1], a[j], a[j + 1], b[j], b[j + 1]);
}
template <int N>
__device__ __forceinline__ void vadd(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
  if constexpr (N == 1) d[0] = a[0] + b[0];
  else
#pragma unroll
    for (int j = 0; j < N; j += 2) add2(d[j], d[j + 1], a[j], a[j + 1], b[j], b[j + 1]);
}

template <int N>
__device__ __forceinline__ void warp_sum(float (&v)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
}

// Sums of N values over the row's threads: a warp (blockDim.y rows per block), or the block.
// The N values' chains of shuffles overlap: summing four rows at once costs little more than one.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* s_red) {
  warp_sum(v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();   // the previous sums have been read
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s_red[i * 32 + warp] = v[i];
  }
  __syncthreads();
  if (nw <= 8) {   // few warps: every thread adds their sums itself (broadcast reads, no shuffles)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 a = *reinterpret_cast<const float4*>(s_red + i * 32), b = *reinterpret_cast<const float4*>(s_red + i * 32 + 4);
      float t = a.x + a.y;
      if (nw > 2) t += a.z;
      if (nw > 3) t += a.w;
      if (nw > 4) t += b.x;
      if (nw > 5) t += b.y;
      if (nw > 6) t += b.z;
      if (nw > 7) t += b.w;
      v[i] = t;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < nw ? s_red[i * 32 + lane] : 0.f;
  warp_sum(v);
}

// Asynchronous copies of a thread's own packs into its own slots of shared memory: rows come in
// D - 1 steps ahead without holding registers, and no barrier is needed to read them.
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct NormParams {
  int32_t T, d;
  float eps, inv_d;
  const void* x;
  int64_t ldx;
  const float* w;
  const float* b;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  const void* dy;
  int64_t lddy;
  const void* dres;
  int64_t lddres;
  void* dx;
  int64_t lddx;
  float* dw;
  float* db;
  float* partial;
  int32_t blocks;   // rows of `partial`
};

// VEC consecutive fp32 values (the packs of w, b and the column sums).
template <int VEC>
__device__ __forceinline__ void load_f32(const float* base, int at, float (&v)[VEC]) {
  if constexpr (VEC <= 2) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = __ldg(base + at + j);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(base + at + j));
      v[j] = q.x;
      v[j + 1 < VEC ? j + 1 : 0] = q.y;
      v[j + 2 < VEC ? j + 2 : 0] = q.z;
      v[j + 3 < VEC ? j + 3 : 0] = q.w;
    }
  }
}

// A warp per row, NV packs a lane: the row stays in registers and its sums need shuffles only.
// (With a row on 12 warps, whose reductions each of them repeats, 16384 x 2880 layer norm in bf16 took
// 63 us, with three quarters of the issue slots in use.)  It takes 44 us, with half of the issue slots
// and 38% of HBM's cycles: a row's loads and its two chains of shuffles follow one another, on a third
// of an SM's warps (80 registers).  RMS norm, with one chain: 36 us.  w and b come from L1 as 16-byte
// loads.
template <class DT, int VEC, int NV, bool LAYER>
__global__ void __launch_bounds__(128, 6) norm_warp_kernel(const NormParams p) {
  const int n = p.d / VEC, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.T) return;
  Pack<DT, VEC> xv[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (lane + 32 * k < n) xv[k] = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)(lane + 32 * k) * VEC);
  float s[1] = {0.f}, q[1] = {0.f};
  float acc[VEC], qcc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = qcc[j] = 0.f;
  if (LAYER) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (lane + 32 * k < n) {
        float f[VEC];
        unpack<DT, VEC>(xv[k], f);
        vadd(acc, acc, f);
      }
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += acc[j];
    warp_sum(s);
  }
  const float m = s[0] * p.inv_d;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (lane + 32 * k < n) {
      float f[VEC];
      unpack<DT, VEC>(xv[k], f);
      if (LAYER) vfma(f, f, 1.f, -m);
      vfma(qcc, f, f, qcc);
    }
#pragma unroll
  for (int j = 0; j < VEC; ++j) q[0] += qcc[j];
  warp_sum(q);
  const float r = 1.f / sqrtf(q[0] * p.inv_d + p.eps);
  if (lane == 0) {
    if (p.rstd) p.rstd[row] = r;
    if (LAYER && p.mean) p.mean[row] = m;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (lane + 32 * k < n) {
      float f[VEC], w[VEC], b[VEC];
      unpack<DT, VEC>(xv[k], f);
      load_f32<VEC>(p.w, (lane + 32 * k) * VEC, w);
      if (LAYER) vfma(f, f, 1.f, -m);
      vfma(f, f, r, 0.f);
      if (LAYER && p.b) {
        load_f32<VEC>(p.b, (lane + 32 * k) * VEC, b);
        vfma(f, f, w, b);
      } else {
        vmul(f, f, w);
      }
      store_pack<DT, VEC>(p.y, row * p.ldy + (int64_t)(lane + 32 * k) * VEC, pack<DT, VEC>(f));
    }
}

// A block per row (longer rows, and few rows: more loads in flight per row), NV packs a thread.
template <class DT, int VEC, int NV, bool LAYER>
__global__ void __launch_bounds__(512) norm_block_kernel(const NormParams p) {
  __shared__ __align__(16) float s_red[32];
  const int n = p.d / VEC, tid = threadIdx.x, step = blockDim.x;
  const int64_t row = blockIdx.x;
  Pack<DT, VEC> xv[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (tid + k * step < n) xv[k] = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)(tid + k * step) * VEC);
  float s[1] = {0.f}, q[1] = {0.f};
  if (LAYER) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (tid + k * step < n) {
        float f[VEC];
        unpack<DT, VEC>(xv[k], f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[0] += f[j];
      }
    row_sum<1>(s, s_red);
  }
  const float m = s[0] * p.inv_d;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (tid + k * step < n) {
      float f[VEC];
      unpack<DT, VEC>(xv[k], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float t = LAYER ? f[j] - m : f[j];
        q[0] += t * t;
      }
    }
  row_sum<1>(q, s_red);
  const float r = 1.f / sqrtf(q[0] * p.inv_d + p.eps);
  if (tid == 0) {
    if (p.rstd) p.rstd[row] = r;
    if (LAYER && p.mean) p.mean[row] = m;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (tid + k * step < n) {
      float f[VEC], w[VEC], b[VEC];
      unpack<DT, VEC>(xv[k], f);
      load_f32<VEC>(p.w, (tid + k * step) * VEC, w);
      if (LAYER && p.b) load_f32<VEC>(p.b, (tid + k * step) * VEC, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        f[j] = (LAYER ? (f[j] - m) * r : f[j] * r) * w[j];
        if (LAYER && p.b) f[j] += b[j];
      }
      store_pack<DT, VEC>(p.y, row * p.ldy + (int64_t)(tid + k * step) * VEC, pack<DT, VEC>(f));
    }
}

// Rows too long for the registers of a block: each pass reads the row again (from L2).
template <class DT, int VEC, bool LAYER>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormParams p) {
  __shared__ __align__(16) float s_red[64];
  const int64_t row = blockIdx.x;
  const int n = p.d / VEC, tid = threadIdx.x, step = blockDim.x;
  float m = 0.f;
  if (LAYER) {
    float s = 0.f;
    for (int c = tid; c < n; c += step) {
      const Pack<DT, VEC> v = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += load1(v.v[j], DT{});
    }
    float v[1] = {s};
    row_sum<1>(v, s_red);
    m = v[0] * p.inv_d;
  }
  float q = 0.f;
  for (int c = tid; c < n; c += step) {
    const Pack<DT, VEC> v = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float t = load1(v.v[j], DT{}) - m;
      q += t * t;
    }
  }
  float qs[1] = {q};
  row_sum<1>(qs, s_red);
  const float r = 1.f / sqrtf(qs[0] * p.inv_d + p.eps);
  if (tid == 0) {
    if (p.rstd) p.rstd[row] = r;
    if (LAYER && p.mean) p.mean[row] = m;
  }
  for (int c = tid; c < n; c += step) {
    const Pack<DT, VEC> v = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
    Pack<DT, VEC> o;
    float w[VEC], b[VEC];
    load_f32<VEC>(p.w, c * VEC, w);
    if (LAYER && p.b) load_f32<VEC>(p.b, c * VEC, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float t = (load1(v.v[j], DT{}) - m) * r * w[j];
      if (LAYER && p.b) t += b[j];
      o.v[j] = store1(t, DT{});
    }
    store_pack<DT, VEC>(p.y, row * p.ldy + (int64_t)c * VEC, o);
  }
}

// The backward pass: a block takes R rows at a time (R groups of rows with short rows:
// blockDim.y), and goes on to others; each thread keeps w and the column sums of its own columns
// (NV packs) over all its rows in registers.  The block's row groups meet in shared memory, and
// each block writes one row of `partial`.
// D > 0: rows come through a D-deep ring of asynchronous copies into each thread's own slots, and
// are read from there twice, which keeps the registers for the sums.  D = 0: loaded in place.
// 16384 x 2880 layer norm with dres in bf16: 89 us, 56% of the issue slots, 48% of HBM's cycles: three
// blocks an SM (96 registers, 74 KB of ring) leave 18 warps to cover two barriers every two rows.
template <class DT, int VEC, int NV, int R, int D, bool LAYER>
__global__ void __launch_bounds__(VEC < 4 ? 1024 : 576) norm_backward_kernel(const NormParams p) {
  pdl_trigger();
  __shared__ __align__(16) float s_red[2 * R * 32];
  extern __shared__ float4 s_dyn[];   // the ring, then the block's column sums (2 d floats)
  const int threads = blockDim.x * blockDim.y, self = threadIdx.y * blockDim.x + threadIdx.x;
  const int n = p.d / VEC, tid = threadIdx.x, step = blockDim.x;
  const int64_t stride = (int64_t)gridDim.x * blockDim.y * R;
  using S = typename DT::Store;
  float w[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[k][j] = ab[k][j] = 0.f;
    if (tid + k * step < n) load_f32<VEC>(p.w, (tid + k * step) * VEC, w[k]);
  }
  const int64_t first = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * R;
  auto slot = [&](int stage, int i, int k, int t) {
    return s_dyn + (((stage * R + i) * NV + k) * 3 + t) * threads + self;
  };
  auto bring = [&](int64_t row0, int stage) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = row0 + i;
      if (row < p.T) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (tid + k * step < n) {
            const int64_t col = (int64_t)(tid + k * step) * VEC;
            copy_async16(slot(stage, i, k, 0), static_cast<const S*>(p.x) + row * p.ldx + col);
            copy_async16(slot(stage, i, k, 1), static_cast<const S*>(p.dy) + row * p.lddy + col);
            if (p.dres) copy_async16(slot(stage, i, k, 2), static_cast<const S*>(p.dres) + row * p.lddres + col);
          }
      }
    }
    copy_commit();
  };
  int stage = 0;
  if (D > 0) {
#pragma unroll
    for (int s = 0; s < D - 1; ++s) bring(first + s * stride, s);
  }
  float rn[R], mn[R];   // the next rows' statistics, loaded a step ahead
  auto stats = [&](int64_t row0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = min(row0 + i, (int64_t)p.T - 1);
      rn[i] = __ldg(p.rstd + row);
      mn[i] = LAYER ? __ldg(p.mean + row) : 0.f;
    }
  };
  stats(first);
  for (int64_t row0 = first; row0 < p.T; row0 += stride) {
    Pack<DT, VEC> xv[R][NV] = {}, dv[R][NV] = {}, rv[R][NV] = {};   // (D = 0)
    if (D > 0) {
      bring(row0 + (D - 1) * stride, stage == 0 ? D - 1 : stage - 1);
      copy_wait<(D > 0 ? D - 1 : 0)>();
    }
    auto get = [&](int i, int k, int t) {
      if (D > 0) return *reinterpret_cast<const Pack<DT, VEC>*>(slot(stage, i, k, t));
      return t == 0 ? xv[i][k] : t == 1 ? dv[i][k] : rv[i][k];
    };
    // xh = (x - m) r, the mean subtracted first: x r - m r is off by 2^-24 of |m| r, which counts in
    // rows whose mean is far from their spread, and where the terms of dx cancel
    float m[R], r[R], c[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = min(row0 + i, (int64_t)p.T - 1);
      r[i] = rn[i];
      m[i] = mn[i];
      c[i] = c[R + i] = 0.f;
      if (D == 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (tid + k * step < n) {
            const int64_t col = (int64_t)(tid + k * step) * VEC;
            xv[i][k] = load_pack<DT, VEC>(p.x, row * p.ldx + col);
            dv[i][k] = load_pack<DT, VEC>(p.dy, row * p.lddy + col);
            if (p.dres) rv[i][k] = load_pack<DT, VEC>(p.dres, row * p.lddres + col);
          }
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (row0 + i < p.T) {
        float s1[VEC], s2[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) s1[j] = s2[j] = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (tid + k * step < n) {
            float x[VEC], dy[VEC], g[VEC];
            unpack<DT, VEC>(get(i, k, 0), x);
            unpack<DT, VEC>(get(i, k, 1), dy);
            if (LAYER) vfma(x, x, 1.f, -m[i]);
            vfma(x, x, r[i], 0.f);              // xh
            vmul(g, dy, w[k]);
            vfma(s1, g, x, s1);
            vfma(aw[k], dy, x, aw[k]);
            if (LAYER) {
              vadd(s2, s2, g);
              vadd(ab[k], ab[k], dy);
            }
          }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          c[i] += s1[j];
          c[R + i] += s2[j];
        }
      }
    }
    stats(row0 + stride);
    if (LAYER) {
      row_sum<2 * R>(c, s_red);
    } else {
      float c1[R];
#pragma unroll
      for (int i = 0; i < R; ++i) c1[i] = c[i];
      row_sum<R>(c1, s_red);
#pragma unroll
      for (int i = 0; i < R; ++i) c[i] = c1[i];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = row0 + i;
      if (row < p.T) {
        const float c1 = -r[i] * c[i] * p.inv_d, c2 = LAYER ? -r[i] * c[R + i] * p.inv_d : 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if (tid + k * step < n) {
            float x[VEC], dy[VEC];
            unpack<DT, VEC>(get(i, k, 0), x);
            unpack<DT, VEC>(get(i, k, 1), dy);
            // r g - r mean(g) - (x - m) r r mean(g xh)
            if (LAYER) vfma(x, x, 1.f, -m[i]);
            vmul(dy, dy, w[k]);
            vfma(dy, dy, r[i], c2);
            vfma(dy, x, c1 * r[i], dy);
            if (p.dres) {
              unpack<DT, VEC>(get(i, k, 2), x);
              vadd(dy, dy, x);
            }
            store_pack<DT, VEC>(p.dx, row * p.lddx + (int64_t)(tid + k * step) * VEC, pack<DT, VEC>(dy));
          }
      }
    }
    if (D > 0) stage = stage + 1 == D ? 0 : stage + 1;
  }
  if (!p.partial) return;
  float* s_col = reinterpret_cast<float*>(s_dyn + D * R * NV * 3 * threads);   // [blockDim.y > 1 ? 2 * d : 0]
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
  for (int g = 0; g < blockDim.y; ++g) {   // the block's row groups add up in order
    if (threadIdx.y == g) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (tid + k * step < n) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int col = (tid + k * step) * VEC + j;
            float vw = aw[k][j], vb = ab[k][j];
            if (g > 0) {
              vw += s_col[col];
              vb += s_col[p.d + col];
            }
            if (g + 1 < blockDim.y) {
              s_col[col] = vw;
              s_col[p.d + col] = vb;
            } else {
              out[col] = vw;
              out[p.d + col] = vb;
            }
          }
        }
    }
    if (g + 1 < blockDim.y) __syncthreads();
  }
}

// Rows too long for registers: dx with the row read twice, and the column sums on their own.
template <class DT, int VEC, bool LAYER>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormParams p) {
  __shared__ __align__(16) float s_red[64];
  const int64_t row = blockIdx.x;
  const int n = p.d / VEC, tid = threadIdx.x, step = blockDim.x;
  const float m = LAYER ? __ldg(p.mean + row) : 0.f, r = __ldg(p.rstd + row);
  float c1 = 0.f, c2 = 0.f;
  for (int c = tid; c < n; c += step) {
    const Pack<DT, VEC> xv = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
    const Pack<DT, VEC> dv = load_pack<DT, VEC>(p.dy, row * p.lddy + (int64_t)c * VEC);
    float w[VEC];
    load_f32<VEC>(p.w, c * VEC, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float xh = (load1(xv.v[j], DT{}) - m) * r, g = load1(dv.v[j], DT{}) * w[j];
      c1 += g * xh;
      c2 += g;
    }
  }
  float t[2] = {c1, c2};
  row_sum<2>(t, s_red);
  c1 = t[0] * p.inv_d;
  c2 = LAYER ? t[1] * p.inv_d : 0.f;
  for (int c = tid; c < n; c += step) {
    const Pack<DT, VEC> xv = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
    const Pack<DT, VEC> dv = load_pack<DT, VEC>(p.dy, row * p.lddy + (int64_t)c * VEC);
    Pack<DT, VEC> o, rv;
    if (p.dres) rv = load_pack<DT, VEC>(p.dres, row * p.lddres + (int64_t)c * VEC);
    float w[VEC];
    load_f32<VEC>(p.w, c * VEC, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float xh = (load1(xv.v[j], DT{}) - m) * r, g = load1(dv.v[j], DT{}) * w[j];
      float v = r * (g - xh * c1 - c2);
      if (p.dres) v += load1(rv.v[j], DT{});
      o.v[j] = store1(v, DT{});
    }
    store_pack<DT, VEC>(p.dx, row * p.lddx + (int64_t)c * VEC, o);
  }
}

template <class DT, bool LAYER>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormParams p) {
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (col >= p.d) return;
  const int64_t r0 = (int64_t)blockIdx.x * p.T / p.blocks, r1 = (int64_t)(blockIdx.x + 1) * p.T / p.blocks;
  float aw = 0.f, ab = 0.f;
  using S = typename DT::Store;
  for (int64_t row = r0; row < r1; ++row) {
    const float m = LAYER ? __ldg(p.mean + row) : 0.f, r = __ldg(p.rstd + row);
    const float dy = load1(static_cast<const S*>(p.dy)[row * p.lddy + col], DT{});
    aw += dy * ((load1(static_cast<const S*>(p.x)[row * p.ldx + col], DT{}) - m) * r);
    ab += dy;
  }
  p.partial[(int64_t)blockIdx.x * 2 * p.d + col] = aw;
  p.partial[(int64_t)blockIdx.x * 2 * p.d + p.d + col] = ab;
}

// dw and db: the rows of `partial` added up; 32 warps take every 32nd row, then meet in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const NormParams p) {
  __shared__ float s_sum[32][32];
  pdl_wait();   // `partial`
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;   // of [dw | db]
  float v = 0.f;
  if (c < 2 * (int64_t)p.d) {
#pragma unroll 16
    for (int b = warp; b < p.blocks; b += 32) v += p.partial[(int64_t)b * 2 * p.d + c];
  }
  s_sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < 2 * (int64_t)p.d) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) t += s_sum[w][lane];
    if (c < p.d) {
      if (p.dw) p.dw[c] = t;
    } else if (p.db) {
      p.db[c - p.d] = t;
    }
  }
}

NormParams params_of(const NormArgs& a) {
  NormParams p = {};
  p.T = a.T;
  p.d = a.d;
  p.eps = a.eps;
  p.inv_d = 1.f / (float)a.d;
  p.x = a.x;
  p.ldx = a.ldx;
  p.w = a.w;
  p.b = a.b;
  p.y = a.y;
  p.ldy = a.ldy;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.dy = a.dy;
  p.lddy = a.lddy;
  p.dres = a.dres;
  p.lddres = a.lddres;
  p.dx = a.dx;
  p.lddx = a.lddx;
  p.dw = a.dw;
  p.db = a.db;
  p.partial = (a.dw || a.db) ? a.partial : nullptr;
  return p;
}

bool vec_ok(const void* q, int64_t ld, int vec, int bytes) {
  return !q || ((reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0 && ld % vec == 0);
}

// A row's threads: whole warps, at most `nv` packs each; more than `most`: 0 (the row is long).
int row_threads(int packs, int nv, int most = 512) {
  const int t = ((packs + nv - 1) / nv + 31) / 32 * 32;
  return t <= most ? t : 0;
}

// The kernel's dynamic shared memory limit, raised to the most it can ask for once per device.
template <class K>
bool allow_smem(K kern, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) != cudaSuccess) return false;
  if (dev < 64) done.fetch_or(bit, std::memory_order_release);
  return true;
}

template <class DT, int VEC, bool LAYER>
int forward_vec(const NormArgs& a) {
  const NormParams p = params_of(a);
  const int packs = a.d / VEC, lane = (packs + 31) / 32;   // packs a lane
  void (*kern)(NormParams) = nullptr;
  dim3 grid, block;
  // A warp per row where the row fits a warp's registers (96 16-bit values a lane in packs, 48 32-bit
  // ones, 36 single ones) and the rows are many; few rows are spread over blocks (16 x 2880: 2.2 us
  // against 3 us).
  constexpr int U = VEC == 1 ? 6 : VEC == 2 ? 8 : VEC == 4 ? 2 : 2;   // packs a lane in steps of U, 2 U, 4 U, 6 U
  if (a.T >= 2 * multiprocessors() && lane <= 6 * U) {
    kern = lane <= U       ? norm_warp_kernel<DT, VEC, U, LAYER>
           : lane <= 2 * U ? norm_warp_kernel<DT, VEC, 2 * U, LAYER>
           : lane <= 4 * U ? norm_warp_kernel<DT, VEC, 4 * U, LAYER>
                           : norm_warp_kernel<DT, VEC, 6 * U, LAYER>;
    grid = dim3((unsigned)((a.T + 3) / 4));
    block = dim3(128);
  } else {
    constexpr int NV = 32 / VEC < 16 ? 32 / VEC : 16, N1 = VEC >= 4 ? 1 : 4;
    const int g1 = row_threads(packs, N1), g = g1 ? g1 : row_threads(packs, NV);
    kern = g1 ? norm_block_kernel<DT, VEC, N1, LAYER>
           : g ? norm_block_kernel<DT, VEC, NV, LAYER> : norm_long_kernel<DT, VEC, LAYER>;
    grid = dim3((unsigned)a.T);
    block = dim3(g ? g : 1024);
  }
  return launch_kernel(kern, grid, block, 0, a.stream, false, p) == cudaSuccess ? 1 : -1;
}

template <class DT, int VEC, bool LAYER>
int backward_vec(const NormArgs& a) {
  // 16-byte packs: two a thread (a row on half the warps, which each repeat its reductions) and
  // copies ahead.  Pairs and single values: eight values a thread, loaded in place, and as many
  // threads as the registers allow instead.
  constexpr int NV = VEC >= 4 ? 2 : 8 / VEC, R = VEC < 4 ? 1 : 2, D = VEC < 4 ? 0 : 2, most = VEC < 4 ? 1024 : 512;
  NormParams p = params_of(a);
  const int g = row_threads(a.d / VEC, NV, most);
  int n = 1;
  if (g) {
    const int y = g == 32 ? 8 : 1;   // short rows: a warp each, eight groups to a block
    // several rows at a time, and copies ahead, once every block has eight steps to take (the larger
    // code is cold until then; copies of 4 bytes ran slower than loads).  Blocks: those that are
    // resident at once, at most kMaxPartialRows.
    const int64_t fit = std::min<int64_t>(kMaxPartialRows,
                                          (int64_t)multiprocessors() * std::max(1, (VEC < 4 ? 1024 : 576) / (g * y)));
    const bool many = D > 0 && a.T >= 8 * R * fit * y;
    const int64_t rows = y * (many ? R : 1);
    p.blocks = (int)std::min(std::min<int64_t>((a.T + rows - 1) / rows, fit), norm_partial_rows(a.T, a.d));
    const size_t smem = (many ? (size_t)D * R * NV * 3 * 16 * g * y : 0) + (y > 1 ? 8 * (size_t)a.d : 0);
    auto kern = many ? norm_backward_kernel<DT, VEC, NV, R, D, LAYER> : norm_backward_kernel<DT, VEC, NV, 1, 0, LAYER>;
    static std::atomic<uint64_t> done{0};
    if (smem > 48 * 1024 && !allow_smem(norm_backward_kernel<DT, VEC, NV, R, D, LAYER>, done)) return -1;
    if (launch_kernel(kern, dim3((unsigned)p.blocks), dim3(g, y), smem, a.stream, false, p) != cudaSuccess) return -1;
  } else {
    p.blocks = (int)norm_partial_rows(a.T, a.d);
    // (the column sums first: dx may overwrite dy or x)
    if (p.partial) {
      if (launch_kernel(norm_columns_kernel<DT, LAYER>, dim3((unsigned)p.blocks, (unsigned)((a.d + 255) / 256)),
                        dim3(256), 0, a.stream, false, p) != cudaSuccess)
        return -1;
      ++n;
    }
    if (launch_kernel(norm_backward_long_kernel<DT, VEC, LAYER>, dim3((unsigned)a.T), dim3(1024), 0, a.stream, false,
                      p) != cudaSuccess)
      return -1;
  }
  if (!p.partial) return n;
  if (launch_kernel(norm_reduce_kernel, dim3((unsigned)(((a.layer ? 2 : 1) * (int64_t)a.d + 31) / 32)), dim3(1024), 0, a.stream, g != 0,
                    p) != cudaSuccess)
    return -1;
  return n + 1;
}

// Whether every row of the call is whole packs of VEC values at their alignment.
template <class DT, int VEC>
bool packs_ok(const NormArgs& a) {
  constexpr int bytes = VEC * (int)sizeof(typename DT::Store);
  return a.d % VEC == 0 && vec_ok(a.x, a.ldx, VEC, bytes) && vec_ok(a.y, a.ldy, VEC, bytes) &&
         vec_ok(a.dy, a.lddy, VEC, bytes) && vec_ok(a.dres, a.lddres, VEC, bytes) &&
         vec_ok(a.dx, a.lddx, VEC, bytes) && (VEC < 4 || (vec_ok(a.w, 4, 4, 16) && vec_ok(a.b, 4, 4, 16)));
}

template <class DT, int VEC, bool LAYER>
int run_vec(const NormArgs& a, bool backward) {
  return backward ? backward_vec<DT, VEC, LAYER>(a) : forward_vec<DT, VEC, LAYER>(a);
}

template <class DT, bool LAYER>
int dispatch_vec(const NormArgs& a, bool backward) {
  constexpr int VEC = 16 / (int)sizeof(typename DT::Store);
  if (packs_ok<DT, VEC>(a)) return run_vec<DT, VEC, LAYER>(a, backward);
  if constexpr (VEC == 8) {   // 16-bit rows of even length: pairs
    if (packs_ok<DT, 2>(a)) return run_vec<DT, 2, LAYER>(a, backward);
  }
  return run_vec<DT, 1, LAYER>(a, backward);
}

int dispatch(const NormArgs& a, bool backward) {
  switch (a.dtype) {
    case MOE_DTYPE_BF16: return a.layer ? dispatch_vec<BF16, true>(a, backward) : dispatch_vec<BF16, false>(a, backward);
    case MOE_DTYPE_F16: return a.layer ? dispatch_vec<FP16, true>(a, backward) : dispatch_vec<FP16, false>(a, backward);
    default: return a.layer ? dispatch_vec<FP32, true>(a, backward) : dispatch_vec<FP32, false>(a, backward);
  }
}

}  // namespace

int64_t norm_partial_rows(int32_t T, int32_t d) {
  (void)d;
  return std::min(T, kMaxPartialRows);
}
int launch_norm(const NormArgs& a) { return dispatch(a, false); }
int launch_norm_backward(const NormArgs& a) { return dispatch(a, true); }

}  // namespace moe
