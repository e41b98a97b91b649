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

#include "moe_linear.cuh"

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

// VEC consecutive values, as stored (16 bytes, or one value).
template <class DT, int VEC>
struct alignas(VEC == 1 ? sizeof(typename DT::Store) : 16) Pack {
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

// Sums of (a, b) over the row's threads: a warp (blockDim.y rows per block), or the block.
__device__ __forceinline__ float2 row_sum(float a, float b, float2* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();   // the previous sum has been read
  if (lane == 0) s_red[warp] = make_float2(a, b);
  __syncthreads();
  float2 t = lane < nw ? s_red[lane] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
  }
  return t;
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

// NV packs per thread in registers; NV = 0: the row does not fit, and each pass reads it again.
template <class DT, int VEC, int NV, bool LAYER>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
  __shared__ float2 s_red[32];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.T) return;   // (several rows per block only where a row is one warp: no block barrier)
  const int n = p.d / VEC;
  const int tid = threadIdx.x, step = blockDim.x;
  constexpr int R = NV > 0 ? NV : 1;
  Pack<DT, VEC> xv[R];
  float s = 0.f;
  if (NV > 0) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = tid + k * step;
      if (c < n) xv[k] = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
    }
  }
  auto each = [&](auto&& f) {   // f(k, pack index, pack)
    if (NV > 0) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int c = tid + k * step;
        if (c < n) f(c, xv[k]);
      }
    } else {
      for (int c = tid; c < n; c += step) {
        xv[0] = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
        f(c, xv[0]);
      }
    }
  };
  float m = 0.f;
  if (LAYER) {
    each([&](int, const Pack<DT, VEC>& v) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += load1(v.v[j], DT{});
    });
    m = row_sum(s, 0.f, s_red).x * p.inv_d;
  }
  float q = 0.f;
  each([&](int, const Pack<DT, VEC>& v) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float t = load1(v.v[j], DT{}) - m;
      q += t * t;
    }
  });
  const float r = 1.f / sqrtf(row_sum(q, 0.f, s_red).x * p.inv_d + p.eps);
  if (tid == 0) {
    if (p.rstd) p.rstd[row] = r;
    if (LAYER && p.mean) p.mean[row] = m;
  }
  each([&](int c, const Pack<DT, VEC>& v) {
    Pack<DT, VEC> o;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int col = c * VEC + j;
      float t = (load1(v.v[j], DT{}) - m) * r * __ldg(p.w + col);
      if (LAYER && p.b) t += __ldg(p.b + col);
      o.v[j] = store1(t, DT{});
    }
    store_pack<DT, VEC>(p.y, row * p.ldy + (int64_t)c * VEC, o);
  });
}

// Rows blockIdx.x * blockDim.y + threadIdx.y, + gridDim.x * blockDim.y, ...; each thread keeps
// the column sums of its own columns over its rows in registers, the block's rows meet in
// shared memory, and each block writes one row of `partial`.
template <class DT, int VEC, int NV, bool LAYER>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormParams p) {
  __shared__ float2 s_red[32];
  const int n = p.d / VEC, tid = threadIdx.x, step = blockDim.x;
  float aw[NV * VEC], ab[NV * VEC];
#pragma unroll
  for (int j = 0; j < NV * VEC; ++j) aw[j] = ab[j] = 0.f;
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < p.T; row += (int64_t)gridDim.x * blockDim.y) {
    Pack<DT, VEC> xv[NV], dv[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tid + k * step;
      if (c < n) {
        xv[k] = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
        dv[k] = load_pack<DT, VEC>(p.dy, row * p.lddy + (int64_t)c * VEC);
      }
    }
    const float m = LAYER ? __ldg(p.mean + row) : 0.f, r = __ldg(p.rstd + row);
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tid + k * step;
      if (c < n) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (load1(xv[k].v[j], DT{}) - m) * r, dy = load1(dv[k].v[j], DT{});
          const float g = dy * __ldg(p.w + c * VEC + j);
          c1 += g * xh;
          c2 += g;
          aw[k * VEC + j] += dy * xh;
          ab[k * VEC + j] += dy;
        }
      }
    }
    const float2 t = row_sum(c1, c2, s_red);
    c1 = t.x * p.inv_d;
    c2 = LAYER ? t.y * p.inv_d : 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = tid + k * step;
      if (c < n) {
        Pack<DT, VEC> o, rv;
        if (p.dres) rv = load_pack<DT, VEC>(p.dres, row * p.lddres + (int64_t)c * VEC);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (load1(xv[k].v[j], DT{}) - m) * r;
          const float g = load1(dv[k].v[j], DT{}) * __ldg(p.w + c * VEC + j);
          float v = r * (g - xh * c1 - c2);
          if (p.dres) v += load1(rv.v[j], DT{});
          o.v[j] = store1(v, DT{});
        }
        store_pack<DT, VEC>(p.dx, row * p.lddx + (int64_t)c * VEC, o);
      }
    }
  }
  if (!p.partial) return;
  extern __shared__ float s_col[];   // [blockDim.y > 1 ? 2 * d : 0]
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
  for (int g = 0; g < blockDim.y; ++g) {   // the block's row groups add up in order
    if (threadIdx.y == g) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = tid + k * step;
        if (c < n) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int col = c * VEC + j;
            float vw = aw[k * VEC + j], vb = ab[k * VEC + j];
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
    }
    if (g + 1 < blockDim.y) __syncthreads();
  }
}

// Rows too long for registers: dx with the row read twice, and the column sums on their own.
template <class DT, int VEC, bool LAYER>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormParams p) {
  __shared__ float2 s_red[32];
  const int64_t row = blockIdx.x;
  const int n = p.d / VEC, tid = threadIdx.x, step = blockDim.x;
  const float m = LAYER ? __ldg(p.mean + row) : 0.f, r = __ldg(p.rstd + row);
  float c1 = 0.f, c2 = 0.f;
  for (int c = tid; c < n; c += step) {
    const Pack<DT, VEC> xv = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
    const Pack<DT, VEC> dv = load_pack<DT, VEC>(p.dy, row * p.lddy + (int64_t)c * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float xh = (load1(xv.v[j], DT{}) - m) * r, g = load1(dv.v[j], DT{}) * __ldg(p.w + c * VEC + j);
      c1 += g * xh;
      c2 += g;
    }
  }
  const float2 t = row_sum(c1, c2, s_red);
  c1 = t.x * p.inv_d;
  c2 = LAYER ? t.y * p.inv_d : 0.f;
  for (int c = tid; c < n; c += step) {
    const Pack<DT, VEC> xv = load_pack<DT, VEC>(p.x, row * p.ldx + (int64_t)c * VEC);
    const Pack<DT, VEC> dv = load_pack<DT, VEC>(p.dy, row * p.lddy + (int64_t)c * VEC);
    Pack<DT, VEC> o, rv;
    if (p.dres) rv = load_pack<DT, VEC>(p.dres, row * p.lddres + (int64_t)c * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float xh = (load1(xv.v[j], DT{}) - m) * r, g = load1(dv.v[j], DT{}) * __ldg(p.w + c * VEC + j);
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

// dw and db: the rows of `partial` added up; 8 warps take every eighth row, then meet in order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormParams p) {
  __shared__ float s_sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;   // of [dw | db]
  float v = 0.f;
  if (c < 2 * (int64_t)p.d)
    for (int b = warp; b < p.blocks; b += 8) v += p.partial[(int64_t)b * 2 * p.d + c];
  s_sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < 2 * (int64_t)p.d) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += s_sum[w][lane];
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

bool vec_ok(const void* q, int64_t ld, int vec, int size) {
  return !q || ((reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % vec == 0 && vec * size == 16);
}

// A row's threads: whole warps, at most `nv` packs each; more than a block holds: 0.
int row_threads(int packs, int nv) {
  const int t = ((packs + nv - 1) / nv + 31) / 32 * 32;
  return t <= 1024 ? t : 0;
}

template <class DT, int VEC, bool LAYER>
int forward_vec(const NormArgs& a) {
  constexpr int NV = VEC == 1 ? 8 : 4;
  const NormParams p = params_of(a);
  const int g = row_threads(a.d / VEC, NV);
  const int rows = g == 32 ? 8 : 1;   // short rows: a warp each, eight to a block
  const dim3 block(g ? g : 1024, rows), grid((unsigned)((a.T + rows - 1) / rows));
  auto kern = g ? norm_kernel<DT, VEC, NV, LAYER> : norm_kernel<DT, VEC, 0, LAYER>;
  return launch_kernel(kern, grid, block, 0, a.stream, false, p) == cudaSuccess ? 1 : -1;
}

template <class DT, int VEC, bool LAYER>
int backward_vec(const NormArgs& a) {
  constexpr int NV = VEC == 8 ? 2 : VEC == 4 ? 4 : 8;
  NormParams p = params_of(a);
  const int g = row_threads(a.d / VEC, NV);
  int n = 1;
  if (g && g <= 512) {
    const int rows = g == 32 ? 8 : 1;
    p.blocks = (int)std::min<int64_t>((a.T + rows - 1) / rows, norm_partial_rows(a.T, a.d));
    if (launch_kernel(norm_backward_kernel<DT, VEC, NV, LAYER>, dim3((unsigned)p.blocks), dim3(g, rows),
                      rows > 1 ? 8 * (size_t)a.d : 0, a.stream, false, p) != cudaSuccess)
      return -1;
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
  if (launch_kernel(norm_reduce_kernel, dim3((unsigned)((2 * (int64_t)a.d + 31) / 32)), dim3(256), 0, a.stream, false,
                    p) != cudaSuccess)
    return -1;
  return n + 1;
}

template <class DT, bool LAYER>
int dispatch_vec(const NormArgs& a, bool backward) {
  constexpr int size = sizeof(typename DT::Store), VEC = 16 / size;
  const bool v = a.d % VEC == 0 && vec_ok(a.x, a.ldx, VEC, size) && vec_ok(a.y, a.ldy, VEC, size) &&
                 vec_ok(a.dy, a.lddy, VEC, size) && vec_ok(a.dres, a.lddres, VEC, size) &&
                 vec_ok(a.dx, a.lddx, VEC, size);
  if (backward) return v ? backward_vec<DT, VEC, LAYER>(a) : backward_vec<DT, 1, LAYER>(a);
  return v ? forward_vec<DT, VEC, LAYER>(a) : forward_vec<DT, 1, LAYER>(a);
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
