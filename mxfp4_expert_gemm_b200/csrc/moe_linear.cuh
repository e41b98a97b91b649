// Internal interface of the 16-bit products (moe_linear.cu) and the row norm (moe_norm.cu).
#pragma once

#include "moe_internal.cuh"

namespace moe {

// What a product launch computes, for rows r of expert e (a dense product is one expert):
//   kForward:  y[r][i]    = f(sum_k x[r][k] W[e][i][k] + bias[e][i]) + residual[r][i]
//   kInputGrad:  dx[r][k] = sum_n dz[r][n] W[e][n][k]
//   kWeightGrad: dW[e][n][k] = sum_r dz[r][n] x[r][k]
enum LinMode { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

struct LinArgs {
  LinMode mode;
  int32_t rows;              // rows of the token buffers (M, or P of a grouped product)
  int32_t K, N, E;
  int32_t bf16;              // 1: bf16, 0: fp16
  int32_t fn;                // a moe_fn value (kForward)
  float limit;
  const int32_t* offsets;    // [E + 1] device, or null: one expert holding every row
  const void* tok;           // x (kForward), dz (kInputGrad, kWeightGrad)
  int64_t ld_tok;
  const void* other;         // W (kForward, kInputGrad), x (kWeightGrad)
  int64_t ld_other;          // (kWeightGrad) row stride of x
  void* out;                 // y, dx or dW
  int64_t ld_out;
  const float* bias;
  const void* residual;
  int64_t ld_res;
  void* z;                   // [rows][N] or null
  int32_t* status;
  int32_t inject_timeout;
  // The kernel before this one in the stream is of the same call (it was launched plainly or so
  // itself): this one may start its prologue under it.
  int32_t pdl;
  cudaStream_t stream;
};

// Each launch function returns the number of kernels launched, or -1 on a CUDA error.
int launch_linear(const LinArgs& a);

struct ActGradArgs {
  int32_t rows, N, E, bf16, fn;
  float limit;
  const int32_t* offsets;
  const void* dy;
  int64_t ld_dy;
  const void* z;             // [rows][N] (null with MOE_FN_NONE)
  void* dz;                  // [rows][N] (null with MOE_FN_NONE)
  float* db;                 // [E][N] or null
  float* partial;            // [act_grad_chunks(rows, E)][N] (db only)
  int32_t* status;
  cudaStream_t stream;
};
int64_t act_grad_chunks(int32_t rows, int32_t E);
int launch_act_grad(const ActGradArgs& a);

struct NormArgs {
  int32_t layer;             // 1: layer norm (mean subtracted, bias), 0: RMSNorm
  int32_t dtype;             // a moe_dtype value
  int32_t T, d;
  float eps;
  const void* x;
  int64_t ldx;
  const float* w;
  const float* b;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  // backward
  const void* dy;
  int64_t lddy;
  const void* dres;
  int64_t lddres;
  void* dx;
  int64_t lddx;
  float* dw;
  float* db;
  float* partial;            // [2][norm_partial_rows(T, d)][d]
  cudaStream_t stream;
};
int64_t norm_partial_rows(int32_t T, int32_t d);
int launch_norm(const NormArgs& a);
int launch_norm_backward(const NormArgs& a);

// Shared with moe_api.cu.
moe_status device_status();              // MOE_OK on an sm_100 device
void note_launches(int32_t n);           // moe_last_launch_count()
int32_t take_injected_timeout();         // the test hook, cleared by reading it
int multiprocessors();                   // of the current device (remembered per device)

}  // namespace moe
