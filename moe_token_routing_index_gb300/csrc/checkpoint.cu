// 8-bit activation checkpoints and the SiLU*mul passes that write and read them
// (include/moe_train.h).
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

__device__ __forceinline__ void load16(const __nv_bfloat16* p, float* v) {
  bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(p)), v);
  bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(p) + 1), v + 8);
}

__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* v) {
  reinterpret_cast<uint4*>(p)[0] = f32_to_bf16x8(v);
  reinterpret_cast<uint4*>(p)[1] = f32_to_bf16x8(v + 8);
}

// Quantise this thread's 16 values with its block's exponent; all 8 threads of the
// group call it.  Returns the codes, *byte = exponent + 127.
__device__ __forceinline__ uint4 quantise16(float* v, uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
    if (u < 0x7f800000u) m = max(m, u);
    else v[i] = __uint_as_float(0x7fffffffu);  // infinities are kept as NaN
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  // m = 1.f * 2^(x - 127) and 448 = 1.75 * 2^8
  int e = (int)(m >> 23) - 127 - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, kMinExp), kMaxExp);
  *byte = (uint32_t)(e + 127);
  const float s = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = f32x2_to_e4m3x2(v[4 * i] * s, v[4 * i + 1] * s) |
           (f32x2_to_e4m3x2(v[4 * i + 2] * s, v[4 * i + 3] * s) << 16);
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
    int v = 0;
    for (int e = threadIdx.x; e < g.E; e += 32) v = min(v + max(__ldg(g.sum_counts + e), 0), g.a);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = min(v + __shfl_xor_sync(0xffffffffu, v, o), g.a);
    if (threadIdx.x == 0) s_rows = v;
  }
  __syncthreads();
  return s_rows;
}

enum Op { kPack, kUnpack, kSilu, kSiluGrad };

template <int OP>
__global__ void __launch_bounds__(kThreads) checkpoint_kernel(const CheckpointArgs g) {
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
      float v[16] = {};
      if (ok) load16(static_cast<const __nv_bfloat16*>(g.x0) + row * g.ld + col, v);
      uint32_t b;
      const uint4 q = quantise16(v, &b);
      if (ok) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.codes) + row * W + col) = q;
      if (in && (u & 7) == 0) g.exponents[row * nb + blk] = (uint8_t)b;
    } else if (OP == kUnpack) {
      if (!ok) continue;
      float v[16];
      dequantise16(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(g.codes) + row * W + col)),
                   __ldg(g.exponents + row * nb + blk), v);
      store16(static_cast<__nv_bfloat16*>(g.out) + row * W + col, v);
    } else if (OP == kSilu) {
      float v0[16] = {}, v1[16] = {}, z[16];
      if (ok) {
        load16(static_cast<const __nv_bfloat16*>(g.x0) + row * g.ld + col, v0);
        load16(static_cast<const __nv_bfloat16*>(g.x1) + row * g.ld + col, v1);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = silu_mul_f32(v0[i], v1[i]);
        store16(static_cast<__nv_bfloat16*>(g.out) + row * W + col, z);
      }
      uint32_t b0, b1;
      const uint4 q0 = quantise16(v0, &b0), q1 = quantise16(v1, &b1);
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
      load16(static_cast<const __nv_bfloat16*>(g.dz) + row * W + col, dz);
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
  const int64_t b = (g.a * nb * 8 + kThreads - 1) / kThreads, cap = (int64_t)device_sm_count() * 8;
  checkpoint_kernel<OP><<<(int)(b < cap ? b : cap), kThreads, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_checkpoint_pack(const CheckpointArgs& g, cudaStream_t s) { return launch<kPack>(g, s); }
cudaError_t launch_checkpoint_unpack(const CheckpointArgs& g, cudaStream_t s) { return launch<kUnpack>(g, s); }
cudaError_t launch_silu_mul_checkpoint(const CheckpointArgs& g, cudaStream_t s) { return launch<kSilu>(g, s); }
cudaError_t launch_silu_mul_backward(const CheckpointArgs& g, cudaStream_t s) { return launch<kSiluGrad>(g, s); }

}  // namespace moe
