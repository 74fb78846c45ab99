// The router's load-balance loss, per-expert counts and its gradient
// (include/moe_train.h).  A warp owns a token; lane l holds experts l, l + 32, ...
#include "common.cuh"
#include "launch.h"
#include "train_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 304;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// sigmoid(a) and 1 - sigmoid(a) = sigmoid(-a), each to full relative precision: from
// e^-|a|, which neither overflows nor cancels.
__device__ __forceinline__ void sigmoid_both(float a, float* s, float* rest) {
  const float e = __expf(-fabsf(a)), r = __fdividef(1.0f, 1.0f + e), er = e * r;
  *s = a >= 0.0f ? r : er;
  *rest = a >= 0.0f ? er : r;
}

// The token's row a[V] (padding: 0) becomes unnormalised weights in place, rest[V] (SIGMOID)
// what each sigmoid lacks to 1; returns 1 / the sum of the weights, or 0.
template <int V, int KIND>
__device__ __forceinline__ float weights(float* a, float* rest, int E, int lane) {
  if (KIND == MOE_BALANCE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 32 * i < E) m = fmaxf(m, a[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.0f;  // every expert masked: all weights are 0
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = lane + 32 * i < E ? __expf(a[i] - m) : 0.0f;
  } else if (KIND == MOE_BALANCE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sigmoid_both(a[i], a + i, rest + i);
      if (lane + 32 * i >= E) a[i] = 0.0f;
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += a[i];
  s = warp_sum(s);
  return s == 0.0f ? 0.0f : 1.0f / s;
}

template <int V, int KIND, bool SELECT>
__global__ void __launch_bounds__(kThreads) balance_kernel(const BalanceArgs g, float* psum, int* csum) {
  extern __shared__ float sh[];  // [kWarps][E] p sums, then [kWarps][E] counts
  const int n = read_count(g.valid, g.T, g.err);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = g.E;
  float ps[V];
  int cs[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ps[i] = 0.0f;
    cs[i] = 0;
  }
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < n; t += (int64_t)gridDim.x * kWarps) {
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      a[i] = e < E ? load_score(g.scores, g.dtype, t * g.stride_t + e * g.stride_e) : 0.0f;
    }
    if (SELECT) {
      uint32_t key[V];
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < E ? route_order_key(a[i]) : 0u;
      for (int k = 0; k < g.top_k; ++k) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, key[i]);
        m = __reduce_max_sync(0xffffffffu, m);
        unsigned at = 0xffffffffu;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (key[i] == m) at = lane + 32 * i;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at == (unsigned)(lane + 32 * i)) {
            key[i] = 0u;
            ++cs[i];
          }
      }
    }
    float rest[V];
    const float inv = weights<V, KIND>(a, rest, E, lane);
#pragma unroll
    for (int i = 0; i < V; ++i) ps[i] += a[i] * inv;
  }
  int* shc = reinterpret_cast<int*>(sh + kWarps * E);
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (lane + 32 * i < E) {
      sh[warp * E + lane + 32 * i] = ps[i];
      if (SELECT) shc[warp * E + lane + 32 * i] = cs[i];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float p = 0.0f;
    int c = 0;
    for (int w = 0; w < kWarps; ++w) {
      p += sh[w * E + e];
      if (SELECT) c += shc[w * E + e];
    }
    psum[(int64_t)blockIdx.x * E + e] = p;
    if (SELECT) csum[(int64_t)blockIdx.x * E + e] = c;
  }
}

__global__ void __launch_bounds__(1024) balance_finish_kernel(const BalanceArgs g, int blocks, const float* psum,
                                                              const int* csum) {
  __shared__ float s_loss[32];
  const int n = read_count(g.valid, g.T, nullptr), E = g.E, e = threadIdx.x;
  float part = 0.0f;
  if (e < E) {
    float p = 0.0f;
    int c = 0;
    for (int b = 0; b < blocks; ++b) {
      p += psum[(int64_t)b * E + e];
      if (!g.counts_in) c += csum[(int64_t)b * E + e];
    }
    if (g.counts_in) c = g.counts_in[e];
    else g.counts_out[e] = c;
    p = n > 0 ? p / n : 0.0f;
    g.mean_probs[e] = p;
    if (n > 0) part = (float)c * ((float)E / ((float)g.top_k * n)) * p;
  }
  part = warp_sum(part);
  if ((threadIdx.x & 31) == 0) s_loss[threadIdx.x >> 5] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float l = 0.0f;
    for (int i = 0; i < 32; ++i) l += s_loss[i];
    *g.loss = g.coefficient * l;
    if (!g.counts_in) g.counts_out[E] = n * g.top_k;
  }
}

template <int V, int KIND>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(const BalanceArgs g) {
  const int n = read_count(g.valid, g.T, g.err);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = g.E;
  if (n == 0) return;
  const float w = g.coefficient / n * (g.dloss ? *g.dloss : 1.0f);
  // f_e - 1 for f_e: the p of a token add up to 1, so the differences f_e - q are the
  // same, and near balance they keep their digits (c E - k Tv is exact in integers)
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    const int64_t kt = (int64_t)g.top_k * n;
    f[i] = e < E ? (float)((int64_t)g.counts_in[e] * E - kt) / (float)kt : 0.0f;
  }
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < n; t += (int64_t)gridDim.x * kWarps) {
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      a[i] = e < E ? load_score(g.scores, g.dtype, t * g.stride_t + e * g.stride_e) : 0.0f;
    }
    float rest[V];
    const float inv = weights<V, KIND>(a, rest, E, lane);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) q += f[i] * a[i];
    q = warp_sum(q) * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e >= E) continue;
      float d = w * (f[i] - q) * inv;
      if (KIND == MOE_BALANCE_SOFTMAX) d *= a[i];
      if (KIND == MOE_BALANCE_SIGMOID) d *= a[i] * rest[i];
      const int64_t at = t * E + e;
      if (g.dtype == MOE_DTYPE_F32) {
        float* o = static_cast<float*>(g.dscores) + at;
        *o = g.accumulate ? *o + d : d;
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.dscores) + at;
        *o = __float2bfloat16_rn(g.accumulate ? __bfloat162float(*o) + d : d);
      }
    }
  }
}

template <int V>
struct Values {
  static constexpr int v = V;
};

// f(Values<V>, Kind) for the least V in 1, 2, 4, .. 32 with 32 V >= E.
template <typename F>
void by_experts(int E, F f) {
  if (E <= 32) f(Values<1>{});
  else if (E <= 64) f(Values<2>{});
  else if (E <= 128) f(Values<4>{});
  else if (E <= 256) f(Values<8>{});
  else if (E <= 512) f(Values<16>{});
  else f(Values<32>{});
}

template <typename F>
void by_kind(int kind, F f) {
  if (kind == MOE_BALANCE_SCORES) f(Values<MOE_BALANCE_SCORES>{});
  else if (kind == MOE_BALANCE_SOFTMAX) f(Values<MOE_BALANCE_SOFTMAX>{});
  else f(Values<MOE_BALANCE_SIGMOID>{});
}

int blocks_for(int T) {
  const int64_t b = ((int64_t)T + kWarps - 1) / kWarps;
  return (int)(b < kMaxBlocks ? b : kMaxBlocks);
}

}  // namespace

size_t balance_loss_workspace_bytes(int T, int E) { return 16 + (size_t)blocks_for(T) * E * 8; }

cudaError_t launch_balance_loss(const BalanceArgs& g, cudaStream_t s) {
  const int blocks = blocks_for(g.T);
  float* psum = reinterpret_cast<float*>(static_cast<char*>(g.ws) + 16);
  int* csum = reinterpret_cast<int*>(psum + (size_t)blocks * g.E);
  const size_t smem = (size_t)kWarps * g.E * 8;
  cudaError_t e = cudaSuccess;
  if (blocks > 0)
    by_experts(g.E, [&](auto v) {
      by_kind(g.kind, [&](auto k) {
        auto kern = g.counts_in ? balance_kernel<decltype(v)::v, decltype(k)::v, false>
                                : balance_kernel<decltype(v)::v, decltype(k)::v, true>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) {
          kern<<<blocks, kThreads, smem, s>>>(g, psum, csum);
          e = cudaGetLastError();
        }
      });
    });
  if (e != cudaSuccess) return e;
  balance_finish_kernel<<<1, 1024, 0, s>>>(g, blocks, psum, csum);
  return cudaGetLastError();
}

cudaError_t launch_balance_loss_backward(const BalanceArgs& g, cudaStream_t s) {
  const int64_t b = ((int64_t)g.T + kWarps - 1) / kWarps, cap = (int64_t)device_sm_count() * 8;
  by_experts(g.E, [&](auto v) {
    by_kind(g.kind, [&](auto k) {
      balance_grad_kernel<decltype(v)::v, decltype(k)::v><<<(int)(b < cap ? b : cap), kThreads, 0, s>>>(g);
    });
  });
  return cudaGetLastError();
}

}  // namespace moe
