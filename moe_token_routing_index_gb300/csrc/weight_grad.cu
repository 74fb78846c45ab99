// The experts' weight gradients dW[e] = dY_e^T X_e (include/moe_train.h).
//
// One block per 64 x 64 tile of an expert's dW; 256 threads hold 4 x 4 fp32 sums
// each and walk the expert's rows 16 at a time through shared memory.  8-bit rows
// are unpacked to bf16 in the workspace first, which loses nothing.
#include "common.cuh"
#include "launch.h"
#include "train_launch.h"

namespace moe {
namespace {

constexpr int kTile = 64, kRows = 16, kThreads = 256;

__global__ void __launch_bounds__(kThreads) weight_grad_kernel(const WeightGradArgs g, const __nv_bfloat16* x) {
  __shared__ float sa[kRows][kTile], sb[kRows][kTile];
  __shared__ int s_row[2];
  const int e = blockIdx.z, n0 = blockIdx.y * kTile, k0 = blockIdx.x * kTile;
  if (threadIdx.x < 32) {
    // rows of the experts before e, and of e, cut at a_max
    int64_t before = 0;
    bool bad = false;
    for (int i = threadIdx.x; i < g.E; i += 32) {
      const int c = __ldg(g.counts + i);
      bad |= c < 0;
      if (i < e) before += max(c, 0);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (threadIdx.x == 0) {
      const int64_t end = before + max(__ldg(g.counts + e), 0);
      s_row[0] = (int)min(before, (int64_t)g.a_max);
      s_row[1] = (int)min(end, (int64_t)g.a_max);
      bad |= end > g.a_max;
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) flag_error(g.err, MOE_DEVERR_BAD_COUNT);
  }
  __syncthreads();
  const int r0 = s_row[0], r1 = s_row[1];
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(g.dy);
  const int tn = threadIdx.x >> 4, tk = threadIdx.x & 15;
  float acc[4][4] = {};
  for (int r = r0; r < r1; r += kRows) {
    for (int i = threadIdx.x; i < kRows * kTile; i += kThreads) {
      const int rr = i / kTile, c = i % kTile;
      const bool row = r + rr < r1;
      sa[rr][c] = row && n0 + c < g.N ? __bfloat162float(dy[(int64_t)(r + rr) * g.N + n0 + c]) : 0.0f;
      sb[rr][c] = row && k0 + c < g.K ? __bfloat162float(x[(int64_t)(r + rr) * g.K + k0 + c]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int rr = 0; rr < kRows; ++rr)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[rr][tn * 4 + i] * sb[rr][tk * 4 + j];
    __syncthreads();
  }
  if (g.accumulate && r0 == r1) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tn * 4 + i, k = k0 + tk * 4 + j;
      if (n >= g.N || k >= g.K) continue;
      const int64_t at = ((int64_t)e * g.N + n) * g.K + k;
      if (g.dw_dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16*>(g.dw)[at] = __float2bfloat16_rn(acc[i][j]);
      else if (g.accumulate) static_cast<float*>(g.dw)[at] += acc[i][j];
      else static_cast<float*>(g.dw)[at] = acc[i][j];
    }
}

}  // namespace

size_t weight_grad_workspace_bytes(int, int a_max, int, int K, bool packed) {
  return packed ? ((size_t)a_max * K * 2 + 255) / 256 * 256 : 0;
}

cudaError_t launch_weight_grad(const WeightGradArgs& g, cudaStream_t s) {
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(g.x);
  if (g.exponents && g.a_max > 0) {
    CheckpointArgs c{};
    c.a = g.a_max;
    c.W = g.K;
    c.codes = const_cast<void*>(g.x);
    c.exponents = const_cast<uint8_t*>(g.exponents);
    c.out = g.ws;
    c.sum_counts = g.counts;
    c.E = g.E;
    c.err = g.err;
    cudaError_t e = launch_checkpoint_unpack(c, s);
    if (e != cudaSuccess) return e;
    x = static_cast<const __nv_bfloat16*>(g.ws);
  }
  const dim3 grid((g.K + kTile - 1) / kTile, (g.N + kTile - 1) / kTile, g.E);
  weight_grad_kernel<<<grid, kThreads, 0, s>>>(g, x);
  return cudaGetLastError();
}

}  // namespace moe
