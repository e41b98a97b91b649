// C-ABI front end of the norms and the 16-bit products: argument checks, workspace, launches.
// Declarations and the contract of every entry point: include/moe_mxfp4.h.
#include <cmath>

#include "moe_linear.cuh"

namespace {

constexpr int32_t kMaxRows = 1 << 24;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// ------------------------------------------------------------------------------ norms
moe_status check_norm(int32_t kind, int32_t dtype, int32_t T, int32_t d) {
  if (kind != MOE_NORM_RMS && kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16 && dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (T < 0 || d <= 0) return MOE_ERR_INVALID_ARG;
  if (d > (1 << 16) || T > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

size_t norm_ws(int32_t T, int32_t d) {
  return round256(2 * sizeof(float) * (size_t)moe::norm_partial_rows(T, d) * (size_t)d);
}

// ------------------------------------------------------------------------------ products
moe_status check_linear(const moe_linear_dims* dm, int32_t rows, bool grouped) {
  if (!dm || rows < 0) return MOE_ERR_INVALID_ARG;
  if (dm->dtype != MOE_DTYPE_BF16 && dm->dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (dm->fn < MOE_FN_NONE || dm->fn > MOE_FN_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (dm->fn == MOE_FN_SWIGLU && (!(dm->limit > 0.f) || !std::isfinite(dm->limit))) return MOE_ERR_INVALID_ARG;
  if (dm->K <= 0 || dm->N <= 0 || dm->K % 8 || dm->N % 8 || dm->K > (1 << 16) || dm->N > (1 << 17))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (dm->fn == MOE_FN_SWIGLU && dm->N % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (dm->E < 1 || dm->E > 256 || (!grouped && dm->E != 1)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

int32_t out_features(const moe_linear_dims& dm) { return dm.fn == MOE_FN_SWIGLU ? dm.N / 2 : dm.N; }

bool rows_ok(const void* p, int64_t ld, int64_t width) {
  return p && aligned(p, 16) && ld >= width && ld % 8 == 0 && ld < (int64_t(1) << 38);
}

// Workspace of a backward pass: dz, then the column sums' chunks.
struct LinWs {
  size_t dz = 0, partial = 0, total = 0;
};
LinWs lin_ws(const moe_linear_dims& dm, int32_t rows) {
  LinWs w;
  size_t at = 0;
  if (dm.fn != MOE_FN_NONE) at = round256(2 * (size_t)rows * dm.N);
  w.partial = at;
  at += round256(sizeof(float) * (size_t)moe::act_grad_chunks(rows, dm.E) * dm.N);
  w.total = at;
  return w;
}

moe::LinArgs linear_args(const moe_linear_dims& dm, int32_t rows, int32_t* status, cudaStream_t stream) {
  moe::LinArgs a = {};
  a.rows = rows;
  a.K = dm.K;
  a.N = dm.N;
  a.E = dm.E;
  a.bf16 = dm.dtype == MOE_DTYPE_BF16;
  a.fn = dm.fn;
  a.limit = dm.limit;
  a.status = status;
  a.stream = stream;
  return a;
}

moe_status forward(const moe_linear_dims* dm, int32_t rows, bool grouped, const void* x, int64_t ldx, const void* w,
                   const int32_t* offsets, const float* bias, const void* residual, int64_t ldr, void* y, int64_t ldy,
                   void* z, int32_t* status_word, void* stream) {
  moe::note_launches(0);
  moe_status st = check_linear(dm, rows, grouped);
  if (st != MOE_OK || rows == 0) return st;
  const int64_t No = out_features(*dm);
  if (!rows_ok(x, ldx, dm->K) || !rows_ok(y, ldy, No) || !w || !aligned(w, 16)) return MOE_ERR_INVALID_ARG;
  if ((residual && !rows_ok(residual, ldr, No)) || (z && !aligned(z, 16))) return MOE_ERR_INVALID_ARG;
  if (grouped && (!offsets || !aligned(offsets, 4))) return MOE_ERR_INVALID_ARG;
  if ((bias && !aligned(bias, 4)) || (status_word && !aligned(status_word, 4))) return MOE_ERR_INVALID_ARG;
  if (y == x || z == x || y == w || (z && z == y) || (y == residual && ldy != ldr)) return MOE_ERR_INVALID_ARG;
  if ((st = moe::device_status()) != MOE_OK) return st;
  moe::LinArgs a = linear_args(*dm, rows, status_word, static_cast<cudaStream_t>(stream));
  a.mode = moe::kForward;
  a.offsets = grouped ? offsets : nullptr;
  a.tok = x;
  a.ld_tok = ldx;
  a.other = w;
  a.out = y;
  a.ld_out = ldy;
  a.bias = bias;
  a.residual = residual;
  a.ld_res = ldr;
  a.z = z;
  a.inject_timeout = moe::take_injected_timeout();
  const int n = moe::launch_linear(a);
  if (n < 0) return MOE_ERR_CUDA;
  moe::note_launches(n);
  return MOE_OK;
}

moe_status backward(const moe_linear_dims* dm, int32_t rows, bool grouped, const void* dy, int64_t lddy, const void* x,
                    int64_t ldx, const void* w, const int32_t* offsets, const void* z, void* dx, int64_t lddx, void* dw,
                    float* db, void* ws, size_t ws_bytes, int32_t* status_word, void* stream) {
  moe::note_launches(0);
  moe_status st = check_linear(dm, rows, grouped);
  if (st != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool act = dm->fn != MOE_FN_NONE;
  if ((dw && !aligned(dw, 16)) || (db && !aligned(db, 4)) || (status_word && !aligned(status_word, 4)))
    return MOE_ERR_INVALID_ARG;
  if (rows > 0) {
    if (!rows_ok(dy, lddy, out_features(*dm)) || (act && (!z || !aligned(z, 16)))) return MOE_ERR_INVALID_ARG;
    if (dx && (!rows_ok(dx, lddx, dm->K) || !w || !aligned(w, 16))) return MOE_ERR_INVALID_ARG;
    if (dw && !rows_ok(x, ldx, dm->K)) return MOE_ERR_INVALID_ARG;
    if (grouped && (!offsets || !aligned(offsets, 4))) return MOE_ERR_INVALID_ARG;
    if (dx && (dx == dy || dx == x || dx == w || dx == dw)) return MOE_ERR_INVALID_ARG;
    if (dw && (dw == w || dw == x || dw == dy)) return MOE_ERR_INVALID_ARG;
    if ((act || db) && (!ws || !aligned(ws, 16))) return MOE_ERR_INVALID_ARG;
    if ((act || db) && ws_bytes < lin_ws(*dm, rows).total) return MOE_ERR_WORKSPACE;
  }
  if (!dx && !dw && !db) return MOE_OK;
  if ((st = moe::device_status()) != MOE_OK) return st;
  if (rows == 0) {
    if (dw && cudaMemsetAsync(dw, 0, 2 * (size_t)dm->E * dm->N * dm->K, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, sizeof(float) * (size_t)dm->E * dm->N, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const LinWs L = lin_ws(*dm, rows);
  int launches = 0;
  const void* dz = dy;
  int64_t ld_dz = lddy;
  if (act || db) {
    moe::ActGradArgs g = {};
    g.rows = rows;
    g.N = dm->N;
    g.E = dm->E;
    g.bf16 = dm->dtype == MOE_DTYPE_BF16;
    g.fn = dm->fn;
    g.limit = dm->limit;
    g.offsets = grouped ? offsets : nullptr;
    g.dy = dy;
    g.ld_dy = lddy;
    g.z = act ? z : nullptr;
    g.dz = act ? static_cast<char*>(ws) + L.dz : nullptr;
    g.db = db;
    g.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + L.partial);
    g.status = status_word;
    g.stream = s;
    const int n = moe::launch_act_grad(g);
    if (n < 0) return MOE_ERR_CUDA;
    launches += n;
    if (act) {
      dz = g.dz;
      ld_dz = dm->N;
    }
  }
  moe::LinArgs a = linear_args(*dm, rows, status_word, s);
  a.fn = MOE_FN_NONE;
  a.offsets = grouped ? offsets : nullptr;
  a.tok = dz;
  a.ld_tok = ld_dz;
  a.inject_timeout = moe::take_injected_timeout();
  a.pdl = launches > 0;
  if (dx) {
    a.mode = moe::kInputGrad;
    a.other = w;
    a.out = dx;
    a.ld_out = lddx;
    const int n = moe::launch_linear(a);
    if (n < 0) return MOE_ERR_CUDA;
    launches += n;
    a.inject_timeout = 0;
    a.pdl = 1;
  }
  if (dw) {
    a.mode = moe::kWeightGrad;
    a.other = x;
    a.ld_other = ldx;
    a.out = dw;
    a.ld_out = dm->K;
    const int n = moe::launch_linear(a);
    if (n < 0) return MOE_ERR_CUDA;
    launches += n;
  }
  moe::note_launches(launches);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_norm(int32_t kind, int32_t dtype, int32_t T, int32_t d, const void* x, int64_t ldx, const float* w,
                    const float* b, float eps, void* y, int64_t ldy, float* mean, float* rstd, void* stream) {
  moe::note_launches(0);
  moe_status st = check_norm(kind, dtype, T, d);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps) || (b && kind == MOE_NORM_RMS)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const uintptr_t size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!x || !y || !w || !aligned(x, size) || !aligned(y, size) || ldx < d || ldy < d) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(b, 4) || !aligned(mean, 4) || !aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
  if (x == y && ldx != ldy) return MOE_ERR_INVALID_ARG;
  if ((st = moe::device_status()) != MOE_OK) return st;
  moe::NormArgs a = {};
  a.layer = kind == MOE_NORM_LAYER;
  a.dtype = dtype;
  a.T = T;
  a.d = d;
  a.eps = eps;
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.b = b;
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  a.stream = static_cast<cudaStream_t>(stream);
  const int n = moe::launch_norm(a);
  if (n < 0) return MOE_ERR_CUDA;
  moe::note_launches(n);
  return MOE_OK;
}

size_t moe_norm_workspace_bytes(int32_t T, int32_t d) {
  return check_norm(MOE_NORM_RMS, MOE_DTYPE_F32, T, d) == MOE_OK ? norm_ws(T, d) : 0;
}

moe_status moe_norm_backward(int32_t kind, int32_t dtype, int32_t T, int32_t d, const void* dy, int64_t lddy,
                             const void* x, int64_t ldx, const float* w, const float* mean, const float* rstd,
                             const void* dres, int64_t lddres, void* dx, int64_t lddx, float* dw, float* db, void* ws,
                             size_t ws_bytes, void* stream) {
  moe::note_launches(0);
  moe_status st = check_norm(kind, dtype, T, d);
  if (st != MOE_OK) return st;
  if (!aligned(dw, 4) || !aligned(db, 4) || (db && kind == MOE_NORM_RMS)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T > 0) {
    const uintptr_t size = dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (!dy || !x || !w || !rstd || !dx || (kind == MOE_NORM_LAYER && !mean)) return MOE_ERR_INVALID_ARG;
    if (!aligned(dy, size) || !aligned(x, size) || !aligned(dx, size) || !aligned(dres, size)) return MOE_ERR_INVALID_ARG;
    if (lddy < d || ldx < d || lddx < d || (dres && lddres < d)) return MOE_ERR_INVALID_ARG;
    if (!aligned(w, 4) || !aligned(mean, 4) || !aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
    if ((dx == dy && lddx != lddy) || (dx == x && lddx != ldx) || (dx == dres && lddx != lddres))
      return MOE_ERR_INVALID_ARG;
    if ((dw || db) && (!ws || !aligned(ws, 16))) return MOE_ERR_INVALID_ARG;
    if ((dw || db) && ws_bytes < norm_ws(T, d)) return MOE_ERR_WORKSPACE;
  }
  if ((st = moe::device_status()) != MOE_OK) return st;
  if (T == 0) {
    if (dw && cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)d, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, sizeof(float) * (size_t)d, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  moe::NormArgs a = {};
  a.layer = kind == MOE_NORM_LAYER;
  a.dtype = dtype;
  a.T = T;
  a.d = d;
  a.x = x;
  a.ldx = ldx;
  a.w = w;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.lddy = lddy;
  a.dres = dres;
  a.lddres = lddres;
  a.dx = dx;
  a.lddx = lddx;
  a.dw = dw;
  a.db = db;
  a.partial = static_cast<float*>(ws);
  a.stream = s;
  const int n = moe::launch_norm_backward(a);
  if (n < 0) return MOE_ERR_CUDA;
  moe::note_launches(n);
  return MOE_OK;
}

moe_status moe_linear(const moe_linear_dims* dims, int32_t M, const void* x, int64_t ldx, const void* w,
                      const float* bias, const void* residual, int64_t ldr, void* y, int64_t ldy, void* z,
                      int32_t* status_word, void* stream) {
  return forward(dims, M, false, x, ldx, w, nullptr, bias, residual, ldr, y, ldy, z, status_word, stream);
}

moe_status moe_linear_backward(const moe_linear_dims* dims, int32_t M, const void* dy, int64_t lddy, const void* x,
                               int64_t ldx, const void* w, const void* z, void* dx, int64_t lddx, void* dw, float* db,
                               void* ws, size_t ws_bytes, int32_t* status_word, void* stream) {
  return backward(dims, M, false, dy, lddy, x, ldx, w, nullptr, z, dx, lddx, dw, db, ws, ws_bytes, status_word, stream);
}

moe_status moe_grouped_linear(const moe_linear_dims* dims, int32_t P, const void* x, int64_t ldx, const void* w,
                              const int32_t* offsets, const float* bias, void* y, int64_t ldy, void* z,
                              int32_t* status_word, void* stream) {
  return forward(dims, P, true, x, ldx, w, offsets, bias, nullptr, 0, y, ldy, z, status_word, stream);
}

moe_status moe_grouped_linear_backward(const moe_linear_dims* dims, int32_t P, const void* dy, int64_t lddy,
                                       const void* x, int64_t ldx, const void* w, const int32_t* offsets,
                                       const void* z, void* dx, int64_t lddx, void* dw, float* db, void* ws,
                                       size_t ws_bytes, int32_t* status_word, void* stream) {
  return backward(dims, P, true, dy, lddy, x, ldx, w, offsets, z, dx, lddx, dw, db, ws, ws_bytes, status_word, stream);
}

size_t moe_linear_workspace_bytes(const moe_linear_dims* dims, int32_t rows) {
  if (check_linear(dims, rows, true) != MOE_OK) return 0;
  return lin_ws(*dims, rows).total;
}

}  // extern "C"
