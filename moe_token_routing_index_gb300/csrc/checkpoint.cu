// 8-bit activation checkpoints and the SiLU*mul passes that write and read them
// (include/moe_train.h).  Bound by memory: 32768 rows of 2 x 2048, SiLU*mul 83 us (6.4
// TB/s), its gradient 102 us (6.6 TB/s).  The passes that quantise are close to bound by
// instruction issue as well, so a block's largest value is found on pairs of bf16 as they
// were loaded.  Registers are held to four blocks a SM forward (three: 94 us, five: 100),
// five backward (two: 117 us).
//
// A thread holds 16 columns (32 bytes of bf16, 16 bytes of codes); the 8 threads of
// an aligned group hold one 128-column block and find its largest value by shuffles.
#include "common.cuh"
#include "launch.h"
#include "train_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -100, kMaxExp = 119;

// 16 bf16 as they lie in memory.
struct Raw16 {
  uint4 a, b;
  __device__ __forceinline__ void values(float* v) const {
    bf16x8_to_f32(a, v);
    bf16x8_to_f32(b, v + 8);
  }
};

__device__ __forceinline__ Raw16 load_raw(const __nv_bfloat16* p) {
  return {__ldg(reinterpret_cast<const uint4*>(p)), __ldg(reinterpret_cast<const uint4*>(p) + 1)};
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* v) {
  reinterpret_cast<uint4*>(p)[0] = f32_to_bf16x8(v);
  reinterpret_cast<uint4*>(p)[1] = f32_to_bf16x8(v + 8);
}

// Quantise this thread's 16 values v, loaded as r, with its block's exponent; all 8 threads
// of the group call it.  Returns the codes, *byte = exponent + 127.
__device__ __forceinline__ uint4 quantise16(const Raw16& r, const float* v, uint32_t* byte) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  uint32_t top = 0u;  // the largest |value| of either place of the pairs, as bits
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  uint32_t m = max(top >> 16, top & 0xffffu);
  float u[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = v[i];
  if (m >= 0x7f80u) {  // infinities are kept as NaN, and count for nothing
    m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = (__float_as_uint(v[i]) & 0x7fffffffu) >> 16;
      if (b < 0x7f80u) m = max(m, b);
      else u[i] = __uint_as_float(0x7fffffffu);
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  // m = 1.f * 2^(x - 127) and 448 = 1.75 * 2^8
  int e = (int)(m >> 7) - 127 - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0);
  e = min(max(e, kMinExp), kMaxExp);
  *byte = (uint32_t)(e + 127);
  const float s = __uint_as_float((uint32_t)(127 - e) << 23);
  const float2 s2 = make_float2(s, s);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = fmul2_rn(make_float2(u[4 * i], u[4 * i + 1]), s2);
    const float2 b = fmul2_rn(make_float2(u[4 * i + 2], u[4 * i + 3]), s2);
    q[i] = f32x2_to_e4m3x2(a.x, a.y) | (f32x2_to_e4m3x2(b.x, b.y) << 16);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

__device__ __forceinline__ void dequantise16(uint4 c, uint32_t byte, float* v) {
  const float s = __uint_as_float(byte << 23);
  const uint32_t q[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

// Valid rows: *valid clamped to a, or the clamped sum of the per-expert counts.
__device__ int row_count(const CheckpointArgs& g) {
  if (!g.sum_counts) return read_count(g.valid, g.a, g.err);
  __shared__ int s_rows;
  if (threadIdx.x < 32) {
    int v = 0;  // at most a, as is what is added: neither sum passes 31 bits
    for (int e = threadIdx.x; e < g.E; e += 32) v += min(max(__ldg(g.sum_counts + e), 0), g.a - v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += min(__shfl_xor_sync(0xffffffffu, v, o), g.a - v);
    if (threadIdx.x == 0) s_rows = v;
  }
  __syncthreads();
  return s_rows;
}

enum Op { kPack, kUnpack, kSilu, kSiluGrad };

template <int OP>
__global__ void __launch_bounds__(kThreads, OP == kSilu ? 4 : 5) checkpoint_kernel(const CheckpointArgs g) {
  const int nb = (g.W + MOE_CHECKPOINT_BLOCK - 1) / MOE_CHECKPOINT_BLOCK;
  const int64_t units = (int64_t)row_count(g) * nb * 8;  // a multiple of 8: groups of 8 threads are whole
  const int64_t rounded = (units + 31) / 32 * 32;        // and every warp's threads run the same passes
  for (int64_t u = blockIdx.x * (int64_t)kThreads + threadIdx.x; u < rounded; u += (int64_t)gridDim.x * kThreads) {
    const int64_t row = (u >> 3) / nb;
    const int blk = (int)((u >> 3) - row * nb);
    const int col = blk * MOE_CHECKPOINT_BLOCK + (int)(u & 7) * 16;
    const bool in = u < units, ok = in && col < g.W;
    const int64_t W = g.W;
    if (OP == kPack) {
      Raw16 r{};
      if (ok) r = load_raw(static_cast<const __nv_bfloat16*>(g.x0) + row * g.ld + col);
      float v[16];
      r.values(v);
      uint32_t b;
      const uint4 q = quantise16(r, v, &b);
      if (ok) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.codes) + row * W + col) = q;
      if (in && (u & 7) == 0) g.exponents[row * nb + blk] = (uint8_t)b;
    } else if (OP == kUnpack) {
      if (!ok) continue;
      float v[16];
      dequantise16(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(g.codes) + row * W + col)),
                   __ldg(g.exponents + row * nb + blk), v);
      store16(static_cast<__nv_bfloat16*>(g.out) + row * W + col, v);
    } else if (OP == kSilu) {
      Raw16 r0{}, r1{};
      if (ok) {
        r0 = load_raw(static_cast<const __nv_bfloat16*>(g.x0) + row * g.ld + col);
        r1 = load_raw(static_cast<const __nv_bfloat16*>(g.x1) + row * g.ld + col);
      }
      float v0[16], v1[16], z[16];
      r0.values(v0);
      r1.values(v1);
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = silu_mul_f32(v0[i], v1[i]);
      if (ok) store16(static_cast<__nv_bfloat16*>(g.out) + row * W + col, z);
      uint32_t b0, b1;
      const uint4 q0 = quantise16(r0, v0, &b0), q1 = quantise16(r1, v1, &b1);
      uint8_t* c = static_cast<uint8_t*>(g.codes) + row * 2 * W + col;
      if (ok) {
        *reinterpret_cast<uint4*>(c) = q0;
        *reinterpret_cast<uint4*>(c + W) = q1;
      }
      if (in && (u & 7) == 0) {
        g.exponents[row * 2 * nb + blk] = (uint8_t)b0;
        g.exponents[row * 2 * nb + nb + blk] = (uint8_t)b1;
      }
    } else {
      if (!ok) continue;
      const uint8_t* c = static_cast<const uint8_t*>(g.codes) + row * 2 * W + col;
      float y0[16], y1[16], dz[16];
      dequantise16(__ldg(reinterpret_cast<const uint4*>(c)), __ldg(g.exponents + row * 2 * nb + blk), y0);
      dequantise16(__ldg(reinterpret_cast<const uint4*>(c + W)), __ldg(g.exponents + row * 2 * nb + nb + blk), y1);
      load_raw(static_cast<const __nv_bfloat16*>(g.dz) + row * W + col).values(dz);
      float z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-y0[i])), a = y0[i] * s;
        z[i] = a * y1[i];
        y1[i] = dz[i] * y1[i] * s * (1.0f + y0[i] * (1.0f - s));  // d y0
        y0[i] = dz[i] * a;                                        // d y1
      }
      __nv_bfloat16* dy = static_cast<__nv_bfloat16*>(g.out) + row * 2 * W + col;
      store16(dy, y1);
      store16(dy + W, y0);
      if (g.z) store16(static_cast<__nv_bfloat16*>(g.z) + row * W + col, z);
    }
  }
}

template <int OP>
cudaError_t launch(const CheckpointArgs& g, cudaStream_t s) {
  const int64_t nb = (g.W + MOE_CHECKPOINT_BLOCK - 1) / MOE_CHECKPOINT_BLOCK;
  // enough blocks to even out their ends (the gradient at 32768 x 2048: 120 us with 8 a SM, 102 with 64)
  constexpr int each = OP == kSilu || OP == kPack ? 16 : 64;
  const int64_t b = (g.a * nb * 8 + kThreads - 1) / kThreads, cap = (int64_t)device_sm_count() * each;
  checkpoint_kernel<OP><<<(int)(b < cap ? b : cap), kThreads, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CheckpointArgs& g, cudaStream_t s) { return launch<kPack>(g, s); }
cudaError_t launch_checkpoint_unpack(const CheckpointArgs& g, cudaStream_t s) { return launch<kUnpack>(g, s); }
cudaError_t launch_silu_mul_checkpoint(const CheckpointArgs& g, cudaStream_t s) { return launch<kSilu>(g, s); }
cudaError_t launch_silu_mul_backward(const CheckpointArgs& g, cudaStream_t s) { return launch<kSiluGrad>(g, s); }

}  // namespace moe
