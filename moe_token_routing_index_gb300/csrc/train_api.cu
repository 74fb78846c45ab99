// The C ABI of the training operators (declared in include/moe_train.h):
// argument checks on the host, then the launchers of the kernel translation units.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "train_launch.h"

namespace {

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int finish(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  if (e == cudaErrorNotSupported) return MOE_ERR_UNSUPPORTED;
  moe::record_cuda_error((int)e);
  return MOE_ERR_CUDA;
}

bool float_dtype(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F32; }
unsigned dtype_bytes(int dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }

constexpr int kMaxNormD = 16384;

int check_norm(const void* x, int64_t ldx, int T, int D, int dtype, const void* gamma, int weight_dtype) {
  if (T < 0 || D < 0) return MOE_ERR_INVALID;
  if (!float_dtype(dtype) || !float_dtype(weight_dtype)) return MOE_ERR_INVALID;
  if (T > 0 && (!x || ldx < D)) return MOE_ERR_INVALID;
  if (!gamma) return MOE_ERR_INVALID;
  if (D > kMaxNormD) return MOE_ERR_UNSUPPORTED;
  if (!aligned(x, dtype_bytes(dtype)) || !aligned(gamma, dtype_bytes(weight_dtype))) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_balance(const void* scores, int dtype, int64_t stride_t, int64_t stride_e, int T, int E, int top_k, int kind,
                  float coefficient) {
  if (T < 0 || E < 1 || top_k < 1 || top_k > E) return MOE_ERR_INVALID;
  if ((int64_t)T * top_k > INT32_MAX) return MOE_ERR_INVALID;
  if (kind != MOE_BALANCE_SCORES && kind != MOE_BALANCE_SOFTMAX && kind != MOE_BALANCE_SIGMOID) return MOE_ERR_INVALID;
  if (!float_dtype(dtype) || !isfinite(coefficient)) return MOE_ERR_INVALID;
  if (E > 1024) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!scores || stride_t < 0 || stride_e < 0)) return MOE_ERR_INVALID;
  if (!aligned(scores, dtype_bytes(dtype))) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Row matrices of the checkpoint operators: a rows of W columns.
int check_rows(int a, int W) {
  if (a < 0 || W < 0) return MOE_ERR_INVALID;
  if (W % 16 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The kernels add an expert's row tiles, 2^23 at most, to its rows in 32 bits.
constexpr int kMaxGatedRows = INT32_MAX - (1 << 24);

int check_gated(const void* x, const void* y, const void* w13, const void* w2, const int32_t* counts, int E, int a_max,
                int D, int H, int activation, const void* z, const void* out) {
  if (E < 1 || a_max < 0 || D < 1 || H < 1) return MOE_ERR_INVALID;
  if (activation != MOE_ACT_SILU && activation != MOE_ACT_GELU) return MOE_ERR_INVALID;
  if (E > 1024 || D % 16 != 0 || H % 16 != 0 || a_max > kMaxGatedRows) return MOE_ERR_UNSUPPORTED;
  if (!w13 || !w2 || !counts) return MOE_ERR_INVALID;
  if (a_max > 0 && (!x || !out)) return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(z, 16) ||
      !aligned(out, 16))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

constexpr int kMaxOrthoSide = 65535, kMaxOrthoBatch = 65535, kMaxOrthoSteps = 16;
constexpr float kOrthoDefaults[3] = {3.4445f, -4.7750f, 2.0315f};

// Whether the iteration s -> (a + p(s)) s, p(s) = b s^2 + c s^4, keeps every singular value of [0, 1] in the
// range of the kernels' fp16.  It is odd and takes [0, top] onto an interval around 0, whose sizes are [0, the
// next top]: the largest value at top and at the extrema below it.  (Starting points on a grid miss what escapes
// between them: of 3.0000002 s - 0.9427371 s^3 all of 1025 points stay below 4 for 16 steps, while some between
// them pass it in 10.)
bool coefficients_fit(const float* coef, int steps) {
  const double a = coef[0], b = coef[1], c = coef[2];
  if (!isfinite(a) || !isfinite(b) || !isfinite(c)) return false;
  // s^2 at the extrema, of p and of the iterate: p' = 0 and a + 3 b s^2 + 5 c s^4 = 0, in the form that
  // does not cancel (0, infinity or NaN where there is none)
  const double of_p = -b / (2.0 * c);
  const double root = sqrt(9.0 * b * b - 20.0 * a * c), q = -0.5 * (3.0 * b + (b < 0.0 ? -root : root));
  const double of_f[2] = {q / (5.0 * c), a / q};
  const auto p = [&](double t) { return (b + c * t) * t; };
  const auto f = [&](double t) { return fabs((a + p(t)) * sqrt(t)); };
  double top = 1.0;
  for (int k = 0; k < steps; ++k) {
    const double t = top * top;
    double largest = fabs(p(t)), next = f(t);
    if (of_p > 0.0 && of_p < t) largest = fmax(largest, fabs(p(of_p)));
    for (const double e : of_f)
      if (e > 0.0 && e < t) next = fmax(next, f(e));
    if (!(largest < 32.0) || !(next < 4.0)) return false;
    top = next;
  }
  return true;
}

// Fills what both entry points share; g's sizes are set.
int check_ortho(moe::OrthoArgs* g, int steps, const float* coefficients, float eps, void* ws, size_t ws_bytes) {
  size_t need;
  const int rc = moe_orthogonalize_workspace_size(g->B, g->N, g->K, &need);
  if (rc != MOE_OK) return rc;
  if (!float_dtype(g->dtype) || steps < 1 || steps > kMaxOrthoSteps) return MOE_ERR_INVALID;
  if (!(eps >= 1e-12f) || !isfinite(eps)) return MOE_ERR_INVALID;
  for (int i = 0; i < 3; ++i) g->coef[i] = coefficients ? coefficients[i] : kOrthoDefaults[i];
  if (!coefficients_fit(g->coef, steps)) return MOE_ERR_INVALID;
  g->steps = steps;
  g->eps = eps;
  if (need == 0) return MOE_OK;
  if (!ws) return MOE_ERR_INVALID;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_INVALID;
  g->ws = ws;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_layer_norm(const void* x, int64_t ldx, int T, int D, int dtype, const void* gamma, const void* beta,
                   int weight_dtype, float eps, const int32_t* num_valid_tokens, void* y, float* mean, float* rstd,
                   cudaStream_t stream) {
  if (T == 0 || D == 0) return MOE_OK;
  int rc = check_norm(x, ldx, T, D, dtype, gamma, weight_dtype);
  if (rc != MOE_OK) return rc;
  if (!y || !(eps >= 0.0f) || !isfinite(eps)) return MOE_ERR_INVALID;
  if (!aligned(y, dtype_bytes(dtype)) || !aligned(beta, dtype_bytes(weight_dtype))) return MOE_ERR_UNSUPPORTED;
  moe::NormArgs g{};
  g.x = x;
  g.ldx = ldx;
  g.T = T;
  g.D = D;
  g.dtype = dtype;
  g.gamma = gamma;
  g.beta = beta;
  g.weight_dtype = weight_dtype;
  g.eps = eps;
  g.valid = num_valid_tokens;
  g.y = y;
  g.mean = mean;
  g.rstd = rstd;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_layer_norm(g, stream));
}

int moe_layer_norm_backward_workspace_size(int T, int D, size_t* bytes) {
  if (!bytes || T < 0 || D < 0) return MOE_ERR_INVALID;
  if (D > kMaxNormD) return MOE_ERR_UNSUPPORTED;
  *bytes = moe::layer_norm_backward_workspace_bytes(T, D);
  return MOE_OK;
}

int moe_layer_norm_backward(const void* dy, const void* x, int64_t ldx, int T, int D, int dtype, const void* gamma,
                            int weight_dtype, const float* mean, const float* rstd, const int32_t* num_valid_tokens,
                            const void* residual_grad, void* dx, float* dgamma, float* dbeta, void* ws,
                            size_t ws_bytes, cudaStream_t stream) {
  size_t need;
  int rc = moe_layer_norm_backward_workspace_size(T, D, &need);
  if (rc != MOE_OK) return rc;
  if (D == 0) return MOE_OK;
  rc = check_norm(x, ldx, T, D, dtype, gamma, weight_dtype);
  if (rc != MOE_OK) return rc;
  if (!dgamma) return MOE_ERR_INVALID;
  if (T > 0 && (!dy || !mean || !rstd || !dx)) return MOE_ERR_INVALID;
  if (need > 0 && !ws) return MOE_ERR_INVALID;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return MOE_ERR_INVALID;
  const unsigned b = dtype_bytes(dtype);
  if (!aligned(dy, b) || !aligned(dx, b) || !aligned(residual_grad, b)) return MOE_ERR_UNSUPPORTED;
  moe::NormArgs g{};
  g.x = x;
  g.ldx = ldx;
  g.T = T;
  g.D = D;
  g.dtype = dtype;
  g.gamma = gamma;
  g.weight_dtype = weight_dtype;
  g.valid = num_valid_tokens;
  g.y = dx;
  g.mean = const_cast<float*>(mean);
  g.rstd = const_cast<float*>(rstd);
  g.dy = dy;
  g.residual = residual_grad;
  g.dgamma = dgamma;
  g.dbeta = dbeta;
  g.ws = ws;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_layer_norm_backward(g, stream));
}

int moe_balance_loss_workspace_size(int T, int E, size_t* bytes) {
  if (!bytes || T < 0 || E < 1) return MOE_ERR_INVALID;
  if (E > 1024) return MOE_ERR_UNSUPPORTED;
  *bytes = moe::balance_loss_workspace_bytes(T, E);
  return MOE_OK;
}

int moe_balance_loss(const void* scores, int scores_dtype, int64_t stride_t, int64_t stride_e, int T, int E, int top_k,
                     int kind, float coefficient, const int32_t* num_valid_tokens, const int32_t* counts_in,
                     int32_t* counts_out, float* mean_probs, float* loss, void* ws, size_t ws_bytes,
                     cudaStream_t stream) {
  int rc = check_balance(scores, scores_dtype, stride_t, stride_e, T, E, top_k, kind, coefficient);
  if (rc != MOE_OK) return rc;
  const size_t need = moe::balance_loss_workspace_bytes(T, E);
  if (!mean_probs || !loss || (!counts_in && !counts_out) || (need > 0 && !ws)) return MOE_ERR_INVALID;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return MOE_ERR_INVALID;
  moe::BalanceArgs g{};
  g.scores = scores;
  g.dtype = scores_dtype;
  g.stride_t = stride_t;
  g.stride_e = stride_e;
  g.T = T;
  g.E = E;
  g.top_k = top_k;
  g.kind = kind;
  g.coefficient = coefficient;
  g.valid = num_valid_tokens;
  g.counts_in = counts_in;
  g.counts_out = counts_out;
  g.mean_probs = mean_probs;
  g.loss = loss;
  g.ws = ws;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_balance_loss(g, stream));
}

int moe_balance_loss_backward(const void* scores, int scores_dtype, int64_t stride_t, int64_t stride_e, int T, int E,
                              int top_k, int kind, float coefficient, const int32_t* num_valid_tokens,
                              const int32_t* counts, const float* dloss, void* dscores, int accumulate,
                              cudaStream_t stream) {
  int rc = check_balance(scores, scores_dtype, stride_t, stride_e, T, E, top_k, kind, coefficient);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  if (!counts || !dscores) return MOE_ERR_INVALID;
  if (!aligned(dscores, dtype_bytes(scores_dtype))) return MOE_ERR_UNSUPPORTED;
  moe::BalanceArgs g{};
  g.scores = scores;
  g.dtype = scores_dtype;
  g.stride_t = stride_t;
  g.stride_e = stride_e;
  g.T = T;
  g.E = E;
  g.top_k = top_k;
  g.kind = kind;
  g.coefficient = coefficient;
  g.valid = num_valid_tokens;
  g.counts_in = counts;
  g.dloss = dloss;
  g.dscores = dscores;
  g.accumulate = accumulate != 0;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_balance_loss_backward(g, stream));
}

int moe_checkpoint_pack(const void* x, int64_t ld, int a, int W, const int32_t* valid_rows, void* codes,
                        uint8_t* exponents, cudaStream_t stream) {
  int rc = check_rows(a, W);
  if (rc != MOE_OK) return rc;
  if (a == 0 || W == 0) return MOE_OK;
  if (!x || !codes || !exponents || ld < W) return MOE_ERR_INVALID;
  if (ld % 8 != 0 || !aligned(x, 16) || !aligned(codes, 16)) return MOE_ERR_UNSUPPORTED;
  moe::CheckpointArgs g{};
  g.x0 = x;
  g.ld = ld;
  g.a = a;
  g.W = W;
  g.valid = valid_rows;
  g.codes = codes;
  g.exponents = exponents;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_checkpoint_pack(g, stream));
}

int moe_checkpoint_unpack(const void* codes, const uint8_t* exponents, int a, int W, const int32_t* valid_rows,
                          void* x, cudaStream_t stream) {
  int rc = check_rows(a, W);
  if (rc != MOE_OK) return rc;
  if (a == 0 || W == 0) return MOE_OK;
  if (!x || !codes || !exponents) return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(codes, 16)) return MOE_ERR_UNSUPPORTED;
  moe::CheckpointArgs g{};
  g.a = a;
  g.W = W;
  g.valid = valid_rows;
  g.codes = const_cast<void*>(codes);
  g.exponents = const_cast<uint8_t*>(exponents);
  g.out = x;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_checkpoint_unpack(g, stream));
}

int moe_silu_mul_checkpoint(const void* x0, const void* x1, int64_t ld, int a, int H, const int32_t* valid_rows,
                            void* z, void* codes, uint8_t* exponents, cudaStream_t stream) {
  int rc = check_rows(a, H);
  if (rc != MOE_OK) return rc;
  if (a == 0 || H == 0) return MOE_OK;
  if (!x0 || !x1 || !z || !codes || !exponents || ld < H) return MOE_ERR_INVALID;
  if (ld % 8 != 0 || !aligned(x0, 16) || !aligned(x1, 16) || !aligned(z, 16) || !aligned(codes, 16))
    return MOE_ERR_UNSUPPORTED;
  moe::CheckpointArgs g{};
  g.x0 = x0;
  g.x1 = x1;
  g.ld = ld;
  g.a = a;
  g.W = H;
  g.valid = valid_rows;
  g.codes = codes;
  g.exponents = exponents;
  g.out = z;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_silu_mul_checkpoint(g, stream));
}

int moe_silu_mul_backward(const void* codes, const uint8_t* exponents, const void* dz, int a, int H,
                          const int32_t* valid_rows, void* dy, void* z, cudaStream_t stream) {
  int rc = check_rows(a, H);
  if (rc != MOE_OK) return rc;
  if (a == 0 || H == 0) return MOE_OK;
  if (!codes || !exponents || !dz || !dy) return MOE_ERR_INVALID;
  if (!aligned(codes, 16) || !aligned(dz, 16) || !aligned(dy, 16) || !aligned(z, 16)) return MOE_ERR_UNSUPPORTED;
  moe::CheckpointArgs g{};
  g.a = a;
  g.W = H;
  g.valid = valid_rows;
  g.codes = const_cast<void*>(codes);
  g.exponents = const_cast<uint8_t*>(exponents);
  g.dz = dz;
  g.out = dy;
  g.z = z;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_silu_mul_backward(g, stream));
}

int moe_grouped_weight_grad_workspace_size(int E, int a_max, int N, int K, int x_dtype, size_t* bytes) {
  if (!bytes || E < 1 || a_max < 0 || N < 0 || K < 0) return MOE_ERR_INVALID;
  if (x_dtype != MOE_DTYPE_BF16 && x_dtype != MOE_DTYPE_E4M3) return MOE_ERR_INVALID;
  if (E > 1024 || N % 16 != 0 || K % 16 != 0) return MOE_ERR_UNSUPPORTED;
  *bytes = moe::weight_grad_workspace_bytes(E, a_max, N, K, x_dtype == MOE_DTYPE_E4M3);
  return MOE_OK;
}

int moe_grouped_weight_grad(const void* dy, const void* x, const uint8_t* x_exponents, const int32_t* counts, int E,
                            int a_max, int N, int K, void* dw, int dw_dtype, int accumulate, void* ws, size_t ws_bytes,
                            cudaStream_t stream) {
  size_t need;
  int rc = moe_grouped_weight_grad_workspace_size(E, a_max, N, K, x_exponents ? MOE_DTYPE_E4M3 : MOE_DTYPE_BF16, &need);
  if (rc != MOE_OK) return rc;
  if (!float_dtype(dw_dtype) || (accumulate && dw_dtype != MOE_DTYPE_F32)) return MOE_ERR_INVALID;
  if (N == 0 || K == 0) return MOE_OK;
  if (!counts || !dw || (a_max > 0 && (!dy || !x)) || (need > 0 && !ws)) return MOE_ERR_INVALID;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_INVALID;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16)) return MOE_ERR_UNSUPPORTED;
  moe::WeightGradArgs g{};
  g.dy = dy;
  g.x = x;
  g.exponents = x_exponents;
  g.counts = counts;
  g.E = E;
  g.a_max = a_max;
  g.N = N;
  g.K = K;
  g.dw = dw;
  g.dw_dtype = dw_dtype;
  g.accumulate = accumulate != 0;
  g.ws = ws;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_weight_grad(g, stream));
}

int moe_gated_mlp(const void* x, const void* w13, const void* w2, const int32_t* counts, int E, int a_max, int D, int H,
                  int activation, void* y, void* z, void* out, cudaStream_t stream) {
  int rc = check_gated(x, y, w13, w2, counts, E, a_max, D, H, activation, z, out);
  if (rc != MOE_OK) return rc;
  if (a_max == 0) return MOE_OK;
  if (!z) return MOE_ERR_INVALID;
  moe::GatedArgs g{};
  g.x = x;
  g.w13 = w13;
  g.w2 = w2;
  g.counts = counts;
  g.E = E;
  g.a_max = a_max;
  g.D = D;
  g.H = H;
  g.activation = activation;
  g.y = y;
  g.z = z;
  g.out = out;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_gated_mlp(g, stream));
}

int moe_gated_mlp_backward(const void* dout, const void* y, const uint8_t* y_exponents, const void* w13, const void* w2,
                           const int32_t* counts, int E, int a_max, int D, int H, int activation, void* dy, void* z,
                           void* dx, cudaStream_t stream) {
  int rc = check_gated(dout, y, w13, w2, counts, E, a_max, D, H, activation, z, dx);
  if (rc != MOE_OK) return rc;
  if (a_max == 0) return MOE_OK;
  if (!y || !dy) return MOE_ERR_INVALID;
  if (!aligned(dy, 16)) return MOE_ERR_UNSUPPORTED;
  moe::GatedArgs g{};
  g.x = dout;
  g.w13 = w13;
  g.w2 = w2;
  g.counts = counts;
  g.E = E;
  g.a_max = a_max;
  g.D = D;
  g.H = H;
  g.activation = activation;
  g.y = const_cast<void*>(y);
  g.exponents = y_exponents;
  g.dy = dy;
  g.z = z;
  g.out = dx;
  rc = moe::device_error_address(&g.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_gated_mlp_backward(g, stream));
}

int moe_orthogonalize_workspace_size(int B, int N, int K, size_t* bytes) {
  if (!bytes || B < 0 || N < 0 || K < 0) return MOE_ERR_INVALID;
  if (B > kMaxOrthoBatch || N > kMaxOrthoSide || K > kMaxOrthoSide) return MOE_ERR_UNSUPPORTED;
  *bytes = B == 0 || N == 0 || K == 0 ? 0 : moe::orthogonalize_workspace_bytes(B, N, K);
  return MOE_OK;
}

int moe_orthogonalize(const void* g, int dtype, int64_t batch_stride, int64_t row_stride, int B, int N, int K, int steps,
                      const float* coefficients, float eps, float scale, void* out, void* ws, size_t ws_bytes,
                      cudaStream_t stream) {
  moe::OrthoArgs a{};
  a.g = g;
  a.dtype = dtype;
  a.batch_stride = batch_stride;
  a.row_stride = row_stride;
  a.B = B;
  a.N = N;
  a.K = K;
  int rc = check_ortho(&a, steps, coefficients, eps, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (!isfinite(scale)) return MOE_ERR_INVALID;
  if (B == 0 || N == 0 || K == 0) return MOE_OK;
  if (!g || !out || row_stride < 0 || batch_stride < 0) return MOE_ERR_INVALID;
  if (!aligned(g, dtype_bytes(dtype)) || !aligned(out, 2)) return MOE_ERR_UNSUPPORTED;
  a.out = out;
  a.scale = scale;
  rc = moe::device_error_address(&a.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_orthogonalize(a, stream));
}

int moe_muon_update(void* w, int w_dtype, const void* grad, int grad_dtype, float* momentum, int B, int N, int K,
                    float mu, int nesterov, float lr, const float* lr_scale, float weight_decay, int steps,
                    const float* coefficients, float eps, void* ws, size_t ws_bytes, cudaStream_t stream) {
  moe::OrthoArgs a{};
  a.g = grad;
  a.dtype = grad_dtype;
  a.batch_stride = (int64_t)N * K;
  a.row_stride = K;
  a.B = B;
  a.N = N;
  a.K = K;
  int rc = check_ortho(&a, steps, coefficients, eps, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (!float_dtype(w_dtype) || !isfinite(lr) || !isfinite(weight_decay) || !(mu >= 0.0f && mu < 1.0f))
    return MOE_ERR_INVALID;
  if (B == 0 || N == 0 || K == 0) return MOE_OK;
  if (!w || !grad || !momentum) return MOE_ERR_INVALID;
  if (!aligned(w, dtype_bytes(w_dtype)) || !aligned(grad, dtype_bytes(grad_dtype)) || !aligned(momentum, 4))
    return MOE_ERR_UNSUPPORTED;
  a.momentum = momentum;
  a.mu = mu;
  a.nesterov = nesterov != 0;
  a.update = true;
  a.out = w;
  a.w_dtype = w_dtype;
  a.scale = lr;
  a.decay = lr * weight_decay;
  a.lr = lr_scale;
  rc = moe::device_error_address(&a.err);
  if (rc != MOE_OK) return rc;
  return finish(moe::launch_orthogonalize(a, stream));
}

}  // extern "C"
