// The router's load-balance loss, per-expert counts and its gradient
// (include/moe_train.h).
//
// LANES lanes of a warp own a token, V experts each (4 in 4 lanes for 16 experts up to 32 in
// 32 for 1024), so a lane's experts stay the same from token to token and their sums of p
// and counts stay in registers.  Blocks leave partial sums; one block adds them in order.
// A batch that one block gets through is a single launch.
//
// The top_k largest of a token: up to 8 from 8 or more values a lane come from sorted lists of
// 8 that are merged in a lane and across lanes (largest_8).  Otherwise each lane sorts its
// values, and top_k rounds take the largest of the lanes' heads, whose lanes move on.  The
// last one is the threshold.  Of bf16 inputs the key carries the expert below the value, so
// that keys differ and ties fall to the lower expert; fp32 inputs that tie are noticed by
// the count above the threshold and selected again one by one.
//
// The selection binds the forward, not memory.  65536 tokens of 128 experts in fp32, top 8:
// 33.6 us looking for the next smaller value in every round, 28.3 with sorted lanes, 25.4 with
// merged lists, 23.0 without a test of each expert against E, 19.9 with the next token's
// values loaded under this one's work, 19.4 with a kernel for each kind; the integer pipe is
// then the busiest.
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "train_launch.h"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kMaxWarps = 32;
constexpr int warps_of(int V) { return V <= 8 ? kMaxWarps : V <= 16 ? 16 : 8; }  // of a forward block
constexpr int kOneBlockTurns = 4;  // turns of a block's tokens up to which it does a batch alone

// How the selection is made: the counts are given, or by keys of bf16 or fp32 inputs.
enum Select { kGiven, kBf16Keys, kF32Keys };
constexpr int kAnyKind = -1;  // of a kernel that takes the kind from its arguments

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (LANES == 32) {
    return __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
  }
}
template <int LANES>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return ~group_max<LANES>(~v);
}
template <int LANES>
__device__ __forceinline__ int group_count(int v) {
  if constexpr (LANES == 32) {
    return __reduce_add_sync(kAll, v);
  } else {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  }
}

// The expert of a lane's value i; e0: that of value 0.  A lane has 4 neighbouring experts of
// every 4 LANES, so that neighbouring lanes read neighbouring pieces of a row.
template <int LANES>
__device__ __forceinline__ int expert(int e0, int i) {
  return e0 + i % 4 + i / 4 * (4 * LANES);
}

// A lane's V values of token t as they lie in memory: nothing waits for them before
// values_of.  wide: they are whole 8- or 16-byte pieces of a dense row.
// Past E, and where the token is not live: -inf, whose weight is 0 and whose key is the least
// (a NaN's is the largest), so that such values are chosen after all others, by ties
// going to the lower expert.
constexpr uint32_t kMinusInf = 0xff800000u, kMinusInf2 = 0xff80ff80u;
template <int V, int LANES>
__device__ __forceinline__ void load_raw(const BalanceArgs& g, int dtype, int64_t t, bool live, int e0, bool wide,
                                         uint32_t* raw) {
  const int E = live ? g.E : 0;
  if (wide) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int64_t at = t * g.stride_t + expert<LANES>(e0, i);
      const bool in = expert<LANES>(e0, i) < E;
      if (dtype == MOE_DTYPE_F32) {
        uint4 v = make_uint4(kMinusInf, kMinusInf, kMinusInf, kMinusInf);
        if (in) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(g.scores) + at));
        raw[i] = v.x;
        raw[i + 1] = v.y;
        raw[i + 2] = v.z;
        raw[i + 3] = v.w;
      } else {
        uint2 v = make_uint2(kMinusInf2, kMinusInf2);
        if (in) v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(g.scores) + at));
        raw[i] = v.x;
        raw[i + 1] = v.y;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert<LANES>(e0, i);
    const int64_t at = t * g.stride_t + e * g.stride_e;
    if (dtype == MOE_DTYPE_F32) raw[i] = e < E ? __ldg(static_cast<const uint32_t*>(g.scores) + at) : kMinusInf;
    else raw[i] = e < E ? __ldg(static_cast<const uint16_t*>(g.scores) + at) : kMinusInf2;
  }
}
template <int V>
__device__ __forceinline__ void values_of(const uint32_t* raw, int dtype, bool wide, float* a) {
  if (dtype == MOE_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = __uint_as_float(raw[i]);
  } else if (wide) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = bf16x2_bits_to_f32(raw[i / 4 * 4 + i % 4 / 2]);
      a[i] = v.x;
      a[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = __uint_as_float(raw[i] << 16);
  }
}

// sigmoid(a) and 1 - sigmoid(a) = sigmoid(-a), each to full relative precision: from
// e^-|a|, which neither overflows nor cancels.
__device__ __forceinline__ void sigmoid_both(float a, float* s, float* rest) {
  const float e = __expf(-fabsf(a)), r = __fdividef(1.0f, 1.0f + e), er = e * r;
  *s = a >= 0.0f ? r : er;
  *rest = a >= 0.0f ? er : r;
}

// 2^x, 0 below the normal numbers: next to the largest weight of a row, which is 1.
constexpr float kLog2E = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The order of scores as in routing (route_order_key), -0 folded onto +0 by an addition.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Whether any live group's lanes all say so.
template <int LANES>
__device__ __forceinline__ bool any_whole_group(bool in) {
  if constexpr (LANES == 32) {
    return __all_sync(kAll, in);
  } else {
    uint32_t b = __ballot_sync(kAll, in);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) b &= b >> o;  // bit i: lanes i .. i + 2 o - 1
    constexpr uint32_t first = LANES == 4 ? 0x11111111u : LANES == 8 ? 0x01010101u : 0x00010001u;
    return (b & first) != 0;
  }
}

// Logits below which a sigmoid is its exponential to fp32, and those of a masked row: the
// sigmoid of one is 0 in 64 bits, too.
constexpr float kSmallLogit = -32.0f, kMaskedLogit = -700.0f;
// Sums of scores whose reciprocal fp32 does not hold, or that it does not hold themselves, are
// taken of scores times a power of two.
constexpr float kTinySum = 0x1p-100f, kHugeSum = 0x1p+100f;

// The token's values become unnormalised weights in place (0 past E), rest[V] what each
// sigmoid lacks to 1; returns 1 / the sum of the weights, or 0.  top: their largest value
// (softmax only).  *scale: what the scores were multiplied by.
//
// A row of sigmoids may add up to less than fp32 holds although each expert's share is an
// ordinary number.  Where all of its logits are below kSmallLogit the weights are so taken
// relative to the largest one's, which is a softmax.
template <int V, int LANES>
__device__ __forceinline__ float weights(float* a, float* rest, int kind, int E, int e0, float top, bool live,
                                         float* scale) {
  *scale = 1.0f;
  if (kind == MOE_BALANCE_SOFTMAX) {
    if (top == -INFINITY) top = 0.0f;  // every expert masked: all weights are 0
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = exp2_ftz((a[i] - top) * kLog2E);
  } else if (kind == MOE_BALANCE_SIGMOID) {
    float most = a[0];
#pragma unroll
    for (int i = 1; i < V; ++i) most = fmaxf(most, a[i]);
    if (any_whole_group<LANES>(live && most < kSmallLogit)) {
      most = group_max<LANES>(most);
      const bool small = most < kSmallLogit;
      if (most < kMaskedLogit) most = 0.0f;  // all weights are 0
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float relative = exp2_ftz((a[i] - most) * kLog2E);
        sigmoid_both(a[i], a + i, rest + i);
        if (small) a[i] = relative;  // (and rest is 1)
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) sigmoid_both(a[i], a + i, rest + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert<LANES>(e0, i) >= E) a[i] = 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) s += a[i];
  s = group_sum<LANES>(s);
  if (kind == MOE_BALANCE_SCORES && __any_sync(kAll, live && ((s > 0.0f && s < kTinySum) || s > kHugeSum))) {
    if (s < kTinySum) *scale = kHugeSum;
    if (s > kHugeSum) *scale = kTinySum;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += a[i] *= *scale;
    s = group_sum<LANES>(s);
  }
  return s == 0.0f ? 0.0f : 1.0f / s;
}

template <int V, int LANES>
__device__ __forceinline__ float largest(const float* a) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, a[i]);
  return group_max<LANES>(m);
}

// Sorts keys descending (odd-even merge network; V a power of two).
template <int V>
__device__ __forceinline__ void sort_descending(uint32_t* k) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int d = p; d > 0; d /= 2)
#pragma unroll
      for (int j = d % p; j + d < V; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i)
          if (j + i + d < V && (j + i) / (2 * p) == (j + i + d) / (2 * p)) {
            const uint32_t a = k[j + i], b = k[j + i + d];
            k[j + i] = max(a, b);
            k[j + i + d] = min(a, b);
          }
}

// Of two descending lists of 8, the larger of h[i] and the other's [7 - i] are the 8 largest of
// both, rising and falling once: this sorts them.
__device__ __forceinline__ void sort_merged(uint32_t* h) {
#pragma unroll
  for (int d = 4; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) {
        const uint32_t a = h[i], b = h[i + d];
        h[i] = max(a, b);
        h[i + d] = min(a, b);
      }
}
// The 8 largest keys of the group's lanes, descending.
template <int V, int LANES>
__device__ __forceinline__ void largest_8(const uint32_t* key, uint32_t* h) {
#pragma unroll
  for (int b = 0; b < V; b += 8) {
    uint32_t own[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) own[i] = key[b + i];
    sort_descending<8>(own);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = b ? max(h[i], own[7 - i]) : own[i];
    if (b) sort_merged(h);
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    uint32_t other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kAll, h[7 - i], o);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = max(h[i], other[i]);
    sort_merged(h);
  }
}

// Adds 1 to the counts cs[V] of the lane's values that are among the token's k largest, where
// the token is live; *top: the largest value.
template <int V, int LANES, int SELECT>
__device__ __forceinline__ void choose(const float* a, int k, int E, int e0, bool live, int* cs, float* top) {
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = order_key(a[i]);
    // a bf16 value's order is in the upper half of its key; the lower expert is the larger key
    if (SELECT == kBf16Keys) key[i] = (key[i] & 0xffff0000u) | (uint32_t)(0xffff - expert<LANES>(e0, i));
  }
  uint32_t limit = 0u;
  if (V >= 8 && k <= 8) {
    uint32_t h[8];
    largest_8<V < 8 ? 8 : V, LANES>(key, h);
    *top = key_value(h[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) limit = max(limit, k <= i + 1 ? h[i] : 0u);
  } else if constexpr (V <= 16) {
    uint32_t head[V];
#pragma unroll
    for (int i = 0; i < V; ++i) head[i] = key[i];
    sort_descending<V>(head);
    for (int r = 0; r < k; ++r) {
      limit = group_max<LANES>(head[0]);
      if (r == 0) *top = key_value(limit);
      if (head[0] == limit) {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) head[i] = head[i + 1];
        head[V - 1] = 0u;
      }
    }
  } else {
    limit = kAll;
    for (int r = 0; r < k; ++r) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < V; ++i) m = max(m, key[i] < limit ? key[i] : 0u);
      limit = group_max<LANES>(m);
      if (r == 0) *top = key_value(limit);
    }
  }
  limit = live ? limit : kAll;
  if (SELECT == kBf16Keys) *top = __uint_as_float(__float_as_uint(*top) & 0xffff0000u);
  int n = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int in = key[i] >= limit ? 1 : 0;
    cs[i] += in;
    n += in;
  }
  if (SELECT == kF32Keys) {
    n = group_count<LANES>(n);
    if (__any_sync(kAll, live && n != k)) {
#pragma unroll
      for (int i = 0; i < V; ++i) cs[i] -= key[i] >= limit ? 1 : 0;
      // equal values among them: one at a time, the lowest expert of the largest value
      for (int r = 0; r < k; ++r) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, key[i]);
        m = group_max<LANES>(m);
        uint32_t at = kAll;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (key[i] == m && expert<LANES>(e0, i) < E) at = (uint32_t)expert<LANES>(e0, i);
        at = group_min<LANES>(at);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at == (uint32_t)expert<LANES>(e0, i)) {
            key[i] = 0u;
            cs[i] += live ? 1 : 0;
          }
      }
    }
  }
}

// The loss, mean_probs and counts from each expert's sum of p and count: threads e < E hold
// them, all threads of a block of up to 1024 call it.
__device__ __forceinline__ void finish(const BalanceArgs& g, int n, int e, float p, int c) {
  __shared__ float s_loss[kMaxWarps];
  float part = 0.0f;
  if (e < g.E) {
    if (g.counts_in) c = __ldg(g.counts_in + e);
    else g.counts_out[e] = c;
    p = n > 0 ? p / n : 0.0f;
    g.mean_probs[e] = p;
    if (n > 0) part = (float)c * ((float)g.E / ((float)g.top_k * n)) * p;
  }
  part = group_sum<32>(part);
  if ((threadIdx.x & 31) == 0) s_loss[threadIdx.x >> 5] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float l = 0.0f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) l += s_loss[i];
    *g.loss = g.coefficient * l;
    if (!g.counts_in) g.counts_out[g.E] = n * g.top_k;
  }
}

// partial: [blocks][2][E], p sums and (as int) counts; unused by a single block.
template <int V, int LANES, int SELECT, int KIND>
__global__ void __launch_bounds__(32 * warps_of(V))
    balance_kernel(const BalanceArgs g, bool wide, float* partial) {
  const int kind = KIND == kAnyKind ? g.kind : KIND;
  extern __shared__ float sh[];  // [warps][E] p sums, then [warps][E] counts
  pdl_launch_dependents();
  constexpr int TOKENS = 32 / LANES;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32, E = g.E;
  const int e0 = (lane & (LANES - 1)) * 4;
  const int dtype = SELECT == kGiven ? g.dtype : SELECT == kBf16Keys ? MOE_DTYPE_BF16 : MOE_DTYPE_F32;
  const int64_t stride = (int64_t)gridDim.x * warps * TOKENS;
  int64_t t0 = ((int64_t)blockIdx.x * warps + warp) * TOKENS, t = t0 + lane / LANES;
  uint32_t raw[V];
  const int n = read_count(g.valid, g.T, g.err);
  load_raw<V, LANES>(g, dtype, t, t < n, e0, wide, raw);
  float ps[V];
  int cs[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ps[i] = 0.0f;
    cs[i] = 0;
  }
  for (; t0 < n; t0 += stride, t += stride) {
    const bool live = t < n;
    float a[V], rest[V], scale;
    values_of<V>(raw, dtype, wide, a);
    load_raw<V, LANES>(g, dtype, t + stride, t + stride < n, e0, wide, raw);  // the next token's, under this one's work
    float top = 0.0f;
    if (SELECT != kGiven) choose<V, LANES, SELECT>(a, g.top_k, E, e0, live, cs, &top);
    else if (kind == MOE_BALANCE_SOFTMAX) top = largest<V, LANES>(a);
    const float inv = weights<V, LANES>(a, rest, kind, E, e0, top, live, &scale);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (live) ps[i] += a[i] * inv;
  }
  // the warp's groups, then the block's warps, in order
  int* shc = reinterpret_cast<int*>(sh + warps * E);
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
      ps[i] += __shfl_xor_sync(kAll, ps[i], o);
      if (SELECT != kGiven) cs[i] += __shfl_xor_sync(kAll, cs[i], o);
    }
    const int e = expert<LANES>(e0, i);
    if (lane < LANES && e < E) {
      sh[warp * E + e] = ps[i];
      if (SELECT != kGiven) shc[warp * E + e] = cs[i];
    }
  }
  __syncthreads();
  const bool alone = gridDim.x == 1 && E <= (int)blockDim.x;
  for (int e = threadIdx.x; e < E || (alone && e < (int)blockDim.x); e += blockDim.x) {
    float p = 0.0f;
    int c = 0;
    if (e < E)
      for (int w = 0; w < warps; ++w) {
        p += sh[w * E + e];
        if (SELECT != kGiven) c += shc[w * E + e];
      }
    if (alone) {
      finish(g, n, e, p, c);
      return;
    }
    partial[(int64_t)blockIdx.x * 2 * E + e] = p;
    if (SELECT != kGiven) partial[((int64_t)blockIdx.x * 2 + 1) * E + e] = __int_as_float(c);
  }
}

// Adds the blocks' partial sums: 1024 / width threads of each expert (width: a power of two,
// at least E) take every so manieth block's, and are added in order.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const BalanceArgs g, const float* __restrict__ partial,
                                                              int blocks, int width) {
  __shared__ float s_p[1024];
  __shared__ int s_c[1024];
  pdl_wait();
  const int n = read_count(g.valid, g.T, nullptr), E = g.E;
  const int e = threadIdx.x & (width - 1), part = threadIdx.x / width, parts = 1024 / width;
  float p = 0.0f;
  int c = 0;
  constexpr int kAtOnce = 5;  // loads under way together
  if (e < E)
    for (int b = part; b < blocks; b += kAtOnce * parts) {
      float vp[kAtOnce], vc[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t at = (int64_t)(b + i * parts) * 2 * E + e;
        const bool in = b + i * parts < blocks;
        vp[i] = in ? partial[at] : 0.0f;
        vc[i] = in && !g.counts_in ? partial[at + E] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        p += vp[i];
        c += __float_as_int(vc[i]);
      }
    }
  s_p[threadIdx.x] = p;
  s_c[threadIdx.x] = c;
  __syncthreads();
  if (part == 0)
    for (int i = 1; i < parts; ++i) {
      p += s_p[i * width + e];
      c += s_c[i * width + e];
    }
  finish(g, n, part == 0 ? e : E, p, c);
}

// The gradient's blocks of an SM, all of them resident, with the next tokens' values on their
// way.  65536 tokens of 128 experts, softmax in fp32 (4 values a lane): 15.5 us, with three 17.0;
// 11000 in bf16, sigmoid: 5.4 both.  65536 of 256 (8 values) 24.4 us, with three 25.5.
constexpr int grad_each(int V) { return V <= 8 ? 4 : V <= 16 ? 2 : 1; }
template <int V, int LANES, int KIND>
__global__ void __launch_bounds__(256, grad_each(V))
    balance_grad_kernel(const BalanceArgs g, bool wide, bool wide_out) {
  constexpr int kind = KIND;
  constexpr int TOKENS = 32 / LANES;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32, E = g.E;
  const int e0 = (lane & (LANES - 1)) * 4;
  const int64_t stride = (int64_t)gridDim.x * warps * TOKENS;
  int64_t t0 = ((int64_t)blockIdx.x * warps + warp) * TOKENS, t = t0 + lane / LANES;
  int count[V];
#pragma unroll
  for (int i = 0; i < V; ++i) count[i] = expert<LANES>(e0, i) < E ? __ldg(g.counts_in + expert<LANES>(e0, i)) : 0;
  const int n = read_count(g.valid, g.T, g.err);
  if (n == 0) return;
  uint32_t raw[V];
  load_raw<V, LANES>(g, g.dtype, t, t < n, e0, wide, raw);
  const float w = g.coefficient / n * (g.dloss ? __ldg(g.dloss) : 1.0f);
  // f_e - 1 for f_e: the p of a token add up to 1, so the differences f_e - q are the
  // same, and near balance they keep their digits (c E - k Tv is exact in integers)
  float f[V];
  const int64_t kt = (int64_t)g.top_k * n;
#pragma unroll
  for (int i = 0; i < V; ++i)
    f[i] = expert<LANES>(e0, i) < E ? (float)((int64_t)count[i] * E - kt) / (float)kt : 0.0f;
  for (; t0 < n; t0 += stride, t += stride) {
    const bool live = t < n;
    float a[V], rest[V], scale;
    values_of<V>(raw, g.dtype, wide, a);
    load_raw<V, LANES>(g, g.dtype, t + stride, t + stride < n, e0, wide, raw);
    const float top = kind == MOE_BALANCE_SOFTMAX ? largest<V, LANES>(a) : 0.0f;
    const float inv = weights<V, LANES>(a, rest, kind, E, e0, top, live, &scale);
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) q += f[i] * a[i];
    q = group_sum<LANES>(q) * inv;
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      d[i] = w * (f[i] - q) * inv * scale;
      if (kind == MOE_BALANCE_SOFTMAX) d[i] *= a[i];
      if (kind == MOE_BALANCE_SIGMOID) d[i] *= a[i] * rest[i];
    }
    if (!live) continue;
    if (wide_out) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        if (expert<LANES>(e0, i) >= E) continue;
        const int64_t at = t * E + expert<LANES>(e0, i);
        if (g.dtype == MOE_DTYPE_F32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.dscores) + at);
          float4 v = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
          if (g.accumulate) {
            const float4 b = *o;
            v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
          }
          *o = v;
        } else {
          uint2* o = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(g.dscores) + at);
          float v[4] = {d[i], d[i + 1], d[i + 2], d[i + 3]};
          if (g.accumulate) {
            const uint2 b = *o;
            const float2 lo = bf16x2_bits_to_f32(b.x), hi = bf16x2_bits_to_f32(b.y);
            v[0] += lo.x;
            v[1] += lo.y;
            v[2] += hi.x;
            v[3] += hi.y;
          }
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
          *o = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = expert<LANES>(e0, i);
        if (e >= E) continue;
        const int64_t at = t * E + e;
        if (g.dtype == MOE_DTYPE_F32) {
          float* o = static_cast<float*>(g.dscores) + at;
          *o = g.accumulate ? *o + d[i] : d[i];
        } else {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.dscores) + at;
          *o = __float2bfloat16_rn(g.accumulate ? __bfloat162float(*o) + d[i] : d[i]);
        }
      }
    }
  }
}

template <int V_, int LANES_>
struct Layout {
  static constexpr int V = V_, LANES = LANES_;
};

// f(Layout) for E experts.  4 experts a lane keep small batches short and 16 take fewer
// instructions a token.  Softmax in fp32, top 8: of 61 experts 4096 tokens take 6.3 us with 4 in 16
// lanes and 7.4 with 16 in 4, 65536 17.0 and 14.3; of 128 experts 500 tokens 5.4 and 6.3,
// 65536 20.6 and 19.2; of 32 experts 1024 tokens 5.1 and (16 in 2) 8.7, 65536 10.2 and 8.9; of
// 256 experts 1024 tokens 9.0 with 8 in 32 lanes and 7.4 with 16 in 16, 65536 46 and 35.  The
// gradient has nothing to select: 65536 tokens of 256 experts 24.2 with 8, 25.7 with 16.
constexpr int kManyTokens = 8192;
template <bool FORWARD, typename F>
void by_experts(int E, int T, F f) {
  if constexpr (FORWARD) {
    if (E > 32 && E <= 128 && T > kManyTokens) return E <= 64 ? f(Layout<16, 4>{}) : f(Layout<16, 8>{});
  }
  if (E <= 16) f(Layout<4, 4>{});
  else if (E <= 32) f(Layout<4, 8>{});
  else if (E <= 64) f(Layout<4, 16>{});
  else if (E <= 128) f(Layout<4, 32>{});
  else if (E <= 256) f(std::conditional_t<FORWARD, Layout<16, 16>, Layout<8, 32>>{});
  else if (E <= 512) f(Layout<16, 32>{});
  else f(Layout<32, 32>{});
}

// f(kind as a type): a kernel for each, without the others' code (65536 tokens of 128 experts in
// fp32 from L2, softmax: 19.4 us and 15.7 backward with one for all, 18.7 and 13.7).  Given the
// counts there is one for all (from HBM 13.9 us, 15.3 with one for each).
template <typename F>
auto by_kind(int kind, F f) {
  return kind == MOE_BALANCE_SOFTMAX   ? f(std::integral_constant<int, MOE_BALANCE_SOFTMAX>{})
         : kind == MOE_BALANCE_SIGMOID ? f(std::integral_constant<int, MOE_BALANCE_SIGMOID>{})
                                       : f(std::integral_constant<int, MOE_BALANCE_SCORES>{});
}

// A forward launch: whether a single block does it all; warps of a block; blocks.
struct Plan {
  bool alone;
  int warps, blocks;
};
// One block while it gets through the tokens in a few turns and has a thread for each expert,
// which then finishes by itself; else up to one a SM.
Plan plan(int T, int E) {
  Plan p = {};
  by_experts<true>(E, T, [&](auto l) {
    p.warps = warps_of(l.V);
    const int64_t turn = (int64_t)p.warps * (32 / l.LANES);
    p.alone = T <= kOneBlockTurns * turn && E <= p.warps * 32;
    const int64_t need = (T + turn - 1) / turn;
    p.blocks = p.alone ? 1 : (int)(need < kNumSmsGB300 ? need : kNumSmsGB300);
  });
  return p;
}

// Whether rows of `stride` elements hold experts by fours as whole aligned pieces.
bool whole_pieces(const void* base, int dtype, int64_t stride, int E) {
  const int piece = dtype == MOE_DTYPE_F32 ? 16 : 8;  // 4 values
  return E % 4 == 0 && stride % 4 == 0 && (reinterpret_cast<uintptr_t>(base) & (piece - 1)) == 0;
}

}  // namespace

size_t balance_loss_workspace_bytes(int T, int E) {
  const Plan p = plan(T, E);
  return p.alone ? 0 : (size_t)p.blocks * 2 * E * sizeof(float);
}

cudaError_t launch_balance_loss(const BalanceArgs& g, cudaStream_t s) {
  const Plan p = plan(g.T, g.E);
  const size_t smem = (size_t)p.warps * g.E * 8;  // at most 64 KB
  const bool wide = g.stride_e == 1 && whole_pieces(g.scores, g.dtype, g.stride_t, g.E);
  float* partial = static_cast<float*>(g.ws);
  cudaError_t e = cudaSuccess;
  if (p.blocks > 0) by_experts<true>(g.E, g.T, [&](auto l) {
    constexpr int V = decltype(l)::V, LANES = decltype(l)::LANES;
    auto kern = by_kind(g.kind, [&](auto kind) {
      constexpr int KIND = decltype(kind)::value;
      return g.counts_in ? balance_kernel<V, LANES, kGiven, kAnyKind>
             : g.dtype == MOE_DTYPE_BF16 ? balance_kernel<V, LANES, kBf16Keys, KIND>
                                         : balance_kernel<V, LANES, kF32Keys, KIND>;
    });
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return;
    kern<<<p.blocks, p.warps * 32, smem, s>>>(g, wide, partial);
    e = cudaGetLastError();
  });
  if (e != cudaSuccess || p.alone) return e;
  int width = 32;
  while (width < g.E) width *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, balance_finish_kernel, g, (const float*)partial, p.blocks, width);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_balance_loss_backward(const BalanceArgs& g, cudaStream_t s) {
  const bool wide = g.stride_e == 1 && whole_pieces(g.scores, g.dtype, g.stride_t, g.E);
  const bool wide_out = whole_pieces(g.dscores, g.dtype, g.E, g.E);
  by_experts<false>(g.E, g.T, [&](auto l) {
    const int64_t most = (int64_t)device_sm_count() * grad_each(l.V);
    const int64_t turn = 8 * (32 / l.LANES), b = (g.T + turn - 1) / turn;
    constexpr int V = decltype(l)::V, LANES = decltype(l)::LANES;
    auto kern = by_kind(g.kind, [&](auto kind) { return balance_grad_kernel<V, LANES, decltype(kind)::value>; });
    kern<<<(int)(b < most ? b : most), 256, 0, s>>>(g, wide, wide_out);
  });
  return cudaGetLastError();
}

}  // namespace moe
