// Layer norm of the token rows and its gradient (include/moe_train.h).
//
// A block owns a row; the weights' gradients are column sums over the rows.
#include "common.cuh"
#include "launch.h"
#include "train_launch.h"

namespace moe {
namespace {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }

constexpr int kThreads = 256;

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float s[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += s[i];
  return t;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs g) {
  const int n = read_count(g.valid, g.T, g.err);
  const W* gamma = static_cast<const W*>(g.gamma);
  const W* beta = static_cast<const W*>(g.beta);
  for (int t = blockIdx.x; t < n; t += gridDim.x) {
    const T* x = static_cast<const T*>(g.x) + t * g.ldx;
    T* y = static_cast<T*>(g.y) + (int64_t)t * g.D;
    float s = 0.0f;
    for (int d = threadIdx.x; d < g.D; d += kThreads) s += to_f32(x[d]);
    const float mean = block_sum(s) / g.D;
    s = 0.0f;
    for (int d = threadIdx.x; d < g.D; d += kThreads) {
      const float c = to_f32(x[d]) - mean;
      s += c * c;
    }
    const float rstd = 1.0f / sqrtf(block_sum(s) / g.D + g.eps);
    for (int d = threadIdx.x; d < g.D; d += kThreads)
      store_f32(y + d, (to_f32(x[d]) - mean) * rstd * to_f32(gamma[d]) + (beta ? to_f32(beta[d]) : 0.0f));
    if (threadIdx.x == 0) {
      if (g.mean) g.mean[t] = mean;
      if (g.rstd) g.rstd[t] = rstd;
    }
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(const NormArgs g) {
  const int n = read_count(g.valid, g.T, g.err);
  const W* gamma = static_cast<const W*>(g.gamma);
  for (int t = blockIdx.x; t < n; t += gridDim.x) {
    const T* x = static_cast<const T*>(g.x) + t * g.ldx;
    const T* dy = static_cast<const T*>(g.dy) + (int64_t)t * g.D;
    const T* res = g.residual ? static_cast<const T*>(g.residual) + (int64_t)t * g.D : nullptr;
    T* dx = static_cast<T*>(g.y) + (int64_t)t * g.D;
    const float mean = g.mean[t], rstd = g.rstd[t];
    float s0 = 0.0f, s1 = 0.0f;
    for (int d = threadIdx.x; d < g.D; d += kThreads) {
      const float gd = to_f32(dy[d]) * to_f32(gamma[d]);
      s0 += gd;
      s1 += gd * ((to_f32(x[d]) - mean) * rstd);
    }
    const float m0 = block_sum(s0) / g.D, m1 = block_sum(s1) / g.D;
    for (int d = threadIdx.x; d < g.D; d += kThreads) {
      const float xh = (to_f32(x[d]) - mean) * rstd;
      const float v = rstd * (to_f32(dy[d]) * to_f32(gamma[d]) - m0 - xh * m1);
      store_f32(dx + d, v + (res ? to_f32(res[d]) : 0.0f));
    }
  }
}

// Column sums: a block of 32 columns x 8 row lanes, each lane's rows in ascending order.
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_kernel(const NormArgs g) {
  __shared__ float sg[8][33], sb[8][33];
  const int n = read_count(g.valid, g.T, g.err);
  const int c = threadIdx.x & 31, l = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + c;
  float dg = 0.0f, db = 0.0f;
  if (d < g.D)
    for (int t = l; t < n; t += 8) {
      const float dy = to_f32(static_cast<const T*>(g.dy)[(int64_t)t * g.D + d]);
      dg += dy * ((to_f32(static_cast<const T*>(g.x)[t * g.ldx + d]) - g.mean[t]) * g.rstd[t]);
      db += dy;
    }
  sg[l][c] = dg;
  sb[l][c] = db;
  __syncthreads();
  if (l == 0 && d < g.D) {
    for (int i = 1; i < 8; ++i) {
      dg += sg[i][c];
      db += sb[i][c];
    }
    g.dgamma[d] = dg;
    if (g.dbeta) g.dbeta[d] = db;
  }
}

template <typename F>
cudaError_t by_types(const NormArgs& g, F f) {
  const bool xf = g.dtype == MOE_DTYPE_F32, wf = g.weight_dtype == MOE_DTYPE_F32;
  if (xf && wf) f(float{}, float{});
  else if (xf) f(float{}, __nv_bfloat16{});
  else if (wf) f(__nv_bfloat16{}, float{});
  else f(__nv_bfloat16{}, __nv_bfloat16{});
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const NormArgs& g, cudaStream_t s) {
  const int cap = device_sm_count() * 8, grid = g.T < cap ? g.T : cap;
  return by_types(g, [&](auto t, auto w) { norm_kernel<decltype(t), decltype(w)><<<grid, kThreads, 0, s>>>(g); });
}

size_t layer_norm_backward_workspace_bytes(int, int) { return 0; }

cudaError_t launch_layer_norm_backward(const NormArgs& g, cudaStream_t s) {
  const int cap = device_sm_count() * 8, grid = g.T < cap ? g.T : cap;
  return by_types(g, [&](auto t, auto w) {
    if (grid > 0) norm_dx_kernel<decltype(t), decltype(w)><<<grid, kThreads, 0, s>>>(g);
    norm_dw_kernel<decltype(t)><<<(g.D + 31) / 32, 256, 0, s>>>(g);
  });
}

}  // namespace moe
