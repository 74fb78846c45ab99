// Internal launcher interface of the training operators (include/moe_train.h)
// between the C ABI (train_api.cu) and their kernel translation units.
// Arguments are validated by the caller.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_train.h"

namespace moe {

// Device address of the current device's error word (MOE_DEVERR_* bits), as a status code.
int device_error_address(unsigned int** out);

struct NormArgs {
  const void* x;
  int64_t ldx;
  int T, D, dtype;
  const void* gamma;
  const void* beta;       // forward only; nullable
  int weight_dtype;
  float eps;              // forward only
  const int32_t* valid;
  void* y;                // forward: y; backward: dx
  float* mean;            // written by the forward (nullable), read by the backward
  float* rstd;
  const void* dy;         // backward only, as what follows
  const void* residual;   // nullable
  float* dgamma;
  float* dbeta;           // nullable
  void* ws;
  unsigned int* err;
};

size_t layer_norm_backward_workspace_bytes(int T, int D);
cudaError_t launch_layer_norm(const NormArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(const NormArgs& a, cudaStream_t s);

struct BalanceArgs {
  const void* scores;
  int dtype;
  int64_t stride_t, stride_e;
  int T, E, top_k, kind;
  float coefficient;
  const int32_t* valid;
  const int32_t* counts_in;
  int32_t* counts_out;
  float* mean_probs;
  float* loss;
  void* ws;
  const float* dloss;     // backward only, as what follows
  void* dscores;
  bool accumulate;
  unsigned int* err;
};

size_t balance_loss_workspace_bytes(int T, int E);
cudaError_t launch_balance_loss(const BalanceArgs& a, cudaStream_t s);
cudaError_t launch_balance_loss_backward(const BalanceArgs& a, cudaStream_t s);

struct CheckpointArgs {
  const void* x0;         // bf16 rows (pack: the only ones; SiLU*mul: the sigmoid's side)
  const void* x1;         // SiLU*mul only
  int64_t ld;
  int a, W;               // W: columns of one half
  const int32_t* valid;
  void* codes;
  uint8_t* exponents;
  const void* dz;         // SiLU*mul backward only
  void* out;              // unpack: x; SiLU*mul: z; its backward: dy
  void* z;                // SiLU*mul backward: nullable
  const int32_t* sum_counts;  // unpack: nullable; the row count is sum(sum_counts[0, E)) instead of *valid
  int E;
  unsigned int* err;
};

cudaError_t launch_checkpoint_pack(const CheckpointArgs& a, cudaStream_t s);
cudaError_t launch_checkpoint_unpack(const CheckpointArgs& a, cudaStream_t s);
cudaError_t launch_silu_mul_checkpoint(const CheckpointArgs& a, cudaStream_t s);
cudaError_t launch_silu_mul_backward(const CheckpointArgs& a, cudaStream_t s);

struct WeightGradArgs {
  const void* dy;
  const void* x;
  const uint8_t* exponents;  // nullable: x is bf16
  const int32_t* counts;
  int E, a_max, N, K;
  void* dw;
  int dw_dtype;
  bool accumulate;
  void* ws;
  unsigned int* err;
};

size_t weight_grad_workspace_bytes(int E, int a_max, int N, int K, bool packed);
cudaError_t launch_weight_grad(const WeightGradArgs& a, cudaStream_t s);

// The gated block: forward from x (writes y, z, out), backward from x = dout and y (writes dy, z, out = dx).
struct GatedArgs {
  const void* x;
  const void* w13;
  const void* w2;
  const int32_t* counts;
  int E, a_max, D, H, activation;
  void* y;                   // forward: nullable; backward: bf16, or codes with exponents
  const uint8_t* exponents;  // backward only
  void* dy;                  // backward only
  void* z;                   // backward: nullable
  void* out;
  unsigned int* err;
};

cudaError_t launch_gated_mlp(const GatedArgs& a, cudaStream_t s);
cudaError_t launch_gated_mlp_backward(const GatedArgs& a, cudaStream_t s);

struct OrthoArgs {
  const void* g;
  int64_t batch_stride, row_stride;
  int dtype, B, N, K;
  float* momentum;           // nullable
  float mu;
  int nesterov;
  int steps;
  float coef[3];
  float eps;
  bool update;               // out are weights: w = (1 - lr decay) w - lr scale X; else out = scale X, bf16
  void* out;
  int w_dtype;
  float scale, decay;
  const float* lr;           // nullable: 1
  void* ws;
  unsigned int* err;
};

size_t orthogonalize_workspace_bytes(int B, int N, int K);
cudaError_t launch_orthogonalize(const OrthoArgs& a, cudaStream_t s);
// Matrices that stay on the chip: no workspace.
bool orthogonalize_small_fits(int N, int K);
cudaError_t launch_orthogonalize_small(const OrthoArgs& a, cudaStream_t s);

}  // namespace moe
