// Orthogonalisation of matrices whose shorter side m is at most 128 (include/moe_train.h), each on the chip
// from its gradient to its result: a cluster of 1 to 16 CTAs holds X [m, n] by columns, kMaxCols or fewer
// a CTA, and one launch does all of a call.
//
// A CTA keeps X in fp32 in its tensor memory (one lane per row) and its value in fp16, scaled by 2^10, in
// shared memory, 64 columns a block, 128B swizzle: read K-major it is both operands of the CTA's part of
// A = X X^T, read MN-major the B operand of P X.  X's columns in tensor memory hold a X, scaled, when
// P X is accumulated onto them, so a step of X is one chain of products and one pass over the result.
// The CTAs' parts of A go through shared memory: each CTA adds the columns that are its own over
// the cluster, in the order of ranks, and stores them, rounded, into every CTA.
//
// Bound by latency: a step of 128 x 7168 on 16 CTAs takes 24000 cycles, of which A's part takes 4300, the way
// of the parts over the cluster 12000 and P, the product with X and the pass over it 2500 each; one CTA with
// 128 x 448 takes 11700.
//
// Waits on products are bounded; a CTA that gives one up records MOE_DEVERR_TIMEOUT and goes on (its results
// are then worthless), so that no CTA of the cluster waits for it in vain.
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "train_launch.h"

#include <type_traits>

namespace moe {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr int kSide = 128;                     // rows of a CTA's tiles
constexpr int kMaxCols = 448;                  // of X in a CTA: with kPart columns, all of tensor memory
constexpr int kPart = 64;                      // columns of A at a time
constexpr int kTmemCols = kMaxCols + kPart;
constexpr int kBlockBytes = kSide * 128;       // 64 columns (or k) of 128 rows
constexpr int kChunk = 16;                     // columns of a pass's step
constexpr float kScale = 1024.0f, kUnscale = 1.0f / kScale;
constexpr float kDown = 0x1p-80f;              // of squares whose sum overflows

// Shared memory: A and P (2 blocks each), where the fp32 part of A lies before them, the norm's sums, the
// barrier, then X.
struct Smem {
  static constexpr int a = 0;
  static constexpr int p = 2 * kBlockBytes;
  static constexpr int sums = 4 * kBlockBytes;            // float2 of this CTA
  static constexpr int warps = sums + 16;                 // float2 of each warp
  static constexpr int bar = warps + 8 * kThreads / 32;
  static constexpr int misc = bar + 8;                    // tensor memory, abort
  static constexpr int x = 5 * kBlockBytes;               // (1024-aligned)
  static constexpr int end = x + kMaxCols / 64 * kBlockBytes;
};
static_assert(Smem::misc + 8 <= Smem::x, "the small things fit in a block");
// All of an SM's shared memory, whatever X takes: a second CTA of a kernel that holds tensor memory must not
// come onto the SM, because it would wait for this one's, and CTAs of its cluster for it.
constexpr int kSmemBytes = 227 * 1024;
static_assert(Smem::end + 1024 <= kSmemBytes, "X fits");

struct Args {
  const void* g;
  int64_t batch, row;
  int dtype;
  float* momentum;
  float mu;
  int nesterov;
  int N, K, m, n, cols;  // cols: of a CTA
  bool tall;             // X is G transposed
  int steps;
  float a, b, c, eps;
  void* out;
  int w_dtype;
  float scale, decay;
  const float* lr;
  unsigned int* err;
};

__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {  // 64-column blocks kBlockBytes apart
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kBlockBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, uint32_t lo, uint32_t hi) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(lo), "r"(hi) : "memory");
}

// Byte offset of the 16-byte piece of columns c .. c + 7 of row r of 64-column blocks.
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return (uint32_t)((c >> 6) * kBlockBytes + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t pack_half(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Row r, columns c .. c + 15, as fp16.
__device__ __forceinline__ void store_row(uint8_t* blocks, int r, int c, const float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint4*>(blocks + piece(r, c + 8 * i)) =
        make_uint4(pack_half(v[8 * i], v[8 * i + 1]), pack_half(v[8 * i + 2], v[8 * i + 3]),
                   pack_half(v[8 * i + 4], v[8 * i + 5]), pack_half(v[8 * i + 6], v[8 * i + 7]));
}

// 32 bytes of a lane.
__device__ __forceinline__ void load32(const void* p, uint32_t* r) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Where element (row, column) of X [m, n] lies in G [N, K].
__device__ __forceinline__ int64_t place(const Args& p, int64_t row_stride, int r, int c) {
  return p.tall ? c * row_stride + r : r * row_stride + c;
}

// A row's columns c .. c + 15 as they lie in memory: whole, where X lies as its tensor does, rows and base are
// aligned to 32 bytes and n is a multiple of 16 (VEC 16); two pieces of 8, with 16 bytes and 8 (VEC 8); or single
// elements (VEC 1).  Reads are made whatever the place, of the nearest element or piece that exists, so that
// they do not wait for one another.  (32 bytes of each of 32 rows take the L1 cache as long as 16 of them.)
template <class T, int VEC>
struct Raw {
  static constexpr int kWords = kChunk * (int)sizeof(T) / 4;
  uint32_t word[VEC > 1 ? kWords : 1];
  T one[VEC > 1 ? 1 : kChunk];

  __device__ __forceinline__ void load(const Args& p, const T* from, int64_t row_stride, int r, int c) {
    r = min(r, p.m - 1);
    if constexpr (VEC == 16) {
      const uint32_t* at = reinterpret_cast<const uint32_t*>(from + place(p, row_stride, r, min(c, p.n - 16)));
#pragma unroll
      for (int i = 0; i < kWords; i += 8) load32(at + i, word + i);
    } else if constexpr (VEC == 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4* at = reinterpret_cast<const uint4*>(from + place(p, row_stride, r, min(c + 8 * h, p.n - 8)));
#pragma unroll
        for (int i = 0; i < kWords / 8; ++i) reinterpret_cast<uint4*>(word)[h * kWords / 8 + i] = at[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) one[i] = from[place(p, row_stride, r, min(c + i, p.n - 1))];
    }
  }
  // in fp32; 0 outside of X
  __device__ __forceinline__ void values(const Args& p, int r, int c, float* v) const {
    if constexpr (VEC > 1 && sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const float2 x = bf16x2_bits_to_f32(word[i]);
        v[2 * i] = x.x;
        v[2 * i + 1] = x.y;
      }
    } else if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[i] = __uint_as_float(word[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        if constexpr (sizeof(T) == 2) v[i] = __bfloat162float(one[i]);
        else v[i] = one[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (r >= p.m || c + i >= p.n) v[i] = 0.0f;
  }
  static __device__ __forceinline__ void store(const Args& p, T* to, int64_t row_stride, int r, int c, const float* v) {
    if (r >= p.m) return;
    if constexpr (VEC > 1) {
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          w[i] = __float_as_uint(v[i]);
        }
      }
      if constexpr (VEC == 16) {
        uint32_t* at = reinterpret_cast<uint32_t*>(to + place(p, row_stride, r, c));
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
          if (c < p.n) store32(at + i, w + i);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c + 8 * h < p.n) {
            uint4* at = reinterpret_cast<uint4*>(to + place(p, row_stride, r, c + 8 * h));
#pragma unroll
            for (int i = 0; i < kWords / 8; ++i) at[i] = reinterpret_cast<const uint4*>(w)[h * kWords / 8 + i];
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (c + i < p.n) {
          T* at = to + place(p, row_stride, r, c + i);
          if constexpr (sizeof(T) == 2) *at = __float2bfloat16_rn(v[i]);
          else *at = v[i];
        }
    }
  }
};

// The result of this thread's row from tensor memory, to bf16 or onto weights.
template <class T, int VEC, bool UPDATE>
__device__ __forceinline__ void finish(const Args& p, T* out, float keep, float scale, int row, int col0, int width,
                                       int group, uint32_t lanes) {
  constexpr int kAtOnce = UPDATE ? 3 : 1;
  for (int c0 = group * kChunk; c0 < width; c0 += 2 * kChunk * kAtOnce) {
    Raw<T, VEC> w[kAtOnce];
    if constexpr (UPDATE) {
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) w[j].load(p, out, p.K, row, col0 + c0 + 2 * kChunk * j);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int c = c0 + 2 * kChunk * j;
      if (c >= width) break;
      float v[kChunk];
      tmem_ld16(lanes + c, v);
      float old[kChunk];
      if constexpr (UPDATE) w[j].values(p, row, col0 + c, old);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[i] = UPDATE ? keep * old[i] - scale * v[i] : scale * v[i];
      Raw<T, VEC>::store(p, out, p.K, row, col0 + c, v);
    }
  }
}

template <class T, int VEC, bool UPDATE>
__global__ void __launch_bounds__(kThreads, 1) small_kernel(const Args p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t size;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  const int ctas = (int)size, rank = (int)cluster_ctarank(), b = blockIdx.x / ctas;
  const int col0 = rank * p.cols, cols = max(0, min(p.cols, p.n - col0));  // this CTA's
  const int width = (cols + 15) / 16 * 16;
  const int parts = (p.m + kPart - 1) / kPart, steps_m = (p.m + 15) / 16;
  const uint32_t bar = sbase + Smem::bar;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Smem::misc + 4);
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + Smem::misc),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(smem + Smem::misc);
  // warps w and w + 4 take the lanes of quarter w, every second chunk of columns each
  const int group = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  uint8_t* x = smem + Smem::x;

  // ------------------------------------------------------------ u and its norm
  float2 q = make_float2(0.0f, 0.0f);
  constexpr int kAtOnce = UPDATE || sizeof(T) == 4 ? 2 : 4;  // chunks under way together
  const T* g = static_cast<const T*>(p.g) + b * p.batch;
  float* momentum = UPDATE ? p.momentum + (int64_t)b * p.N * p.K : nullptr;
  for (int c0 = group * kChunk; c0 < width; c0 += 2 * kChunk * kAtOnce) {
    Raw<T, VEC> raw_u[kAtOnce];
    Raw<float, VEC> raw_m[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      raw_u[j].load(p, g, p.row, row, col0 + c0 + 2 * kChunk * j);
      if constexpr (UPDATE) raw_m[j].load(p, momentum, p.K, row, col0 + c0 + 2 * kChunk * j);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int c = c0 + 2 * kChunk * j;
      if (c >= width) break;
      float u[kChunk], m[kChunk];
      raw_u[j].values(p, row, col0 + c, u);
      if constexpr (UPDATE) {
        raw_m[j].values(p, row, col0 + c, m);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          m[i] = fmaf(p.mu, m[i], u[i]);
          u[i] = p.nesterov ? fmaf(p.mu, m[i], u[i]) : m[i];
        }
        Raw<float, VEC>::store(p, momentum, p.K, row, col0 + c, m);
      }
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        q.x = fmaf(u[i], u[i], q.x);
        const float d = u[i] * kDown;
        q.y = fmaf(d, d, q.y);
      }
      tmem_st16(lanes + c, u);
    }
  }
  tmem_st_wait();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    q.x += __shfl_xor_sync(0xffffffffu, q.x, o);
    q.y += __shfl_xor_sync(0xffffffffu, q.y, o);
  }
  if (lane == 0) reinterpret_cast<float2*>(smem + Smem::warps)[warp] = q;
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 t = make_float2(0.0f, 0.0f);
    for (int w = 0; w < kThreads / 32; ++w) {
      const float2 v = reinterpret_cast<const float2*>(smem + Smem::warps)[w];
      t.x += v.x;
      t.y += v.y;
    }
    *reinterpret_cast<float2*>(smem + Smem::sums) = t;
  }
  __syncthreads();
  if (ctas > 1) cluster_sync_all();
  // every CTA's sums, one a lane, added in the order of ranks
  const uint32_t theirs = map_to_rank(sbase + Smem::sums, min(lane, ctas - 1));
  const float2 mine = make_float2(ld_cluster(theirs), ld_cluster(theirs + 4));
  float2 t = make_float2(0.0f, 0.0f);
  for (int k = 0; k < ctas; ++k) {
    t.x += __shfl_sync(0xffffffffu, mine.x, k);
    t.y += __shfl_sync(0xffffffffu, mine.y, k);
  }
  const bool big = isinf(t.x);
  const float pre = big ? kDown : 1.0f;
  const float f = kScale / (sqrtf(big ? t.y : t.x) + p.eps * pre);

  // this thread's row, chunk by chunk: X from tensor memory by take(v), which leaves X's scaled value in v;
  // its fp16 goes to shared memory and kScale * a * X back
  auto settle = [&](auto take) {
    for (int c = group * kChunk; c < width; c += 2 * kChunk) {
      float v[kChunk];
      tmem_ld16(lanes + c, v);
      take(v);
      store_row(x, row, c, v);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[i] *= p.a * kScale;
      tmem_st16(lanes + c, v);
    }
    tmem_st_wait();
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  settle([&](float* v) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = v[i] * pre * f;
  });

  uint32_t parity = 0;
  const uint32_t base = (1u << 4) | ((uint32_t)(kSide >> 4) << 24);  // fp32 accumulation of fp16
  // one lane issues, with the values of a whole warp; all wait until the products are done
  auto multiply = [&](auto issue) {
    if (warp == 0) {
      if (elect_one()) {
        issue();
        mma_commit(bar);
      }
      __syncwarp();
    }
    if (!mbar_wait(bar, parity, abort)) {
      flag_error(p.err, MOE_DEVERR_TIMEOUT);
      *abort = 1;
    }
    parity ^= 1u;
    tc_fence_after();
  };
  // a part of a square product: D[:, 64 h ..] = sum over k16 steps of rows of `of`, K-major
  auto square = [&](uint32_t of, int k_steps, int h) {
    const uint32_t idesc = base | ((uint32_t)(kPart >> 3) << 17);
    for (int k = 0; k < k_steps; ++k) {
      const uint32_t at = of + (k >> 2) * kBlockBytes + (k & 3) * 32;
      mma_issue<false>(tmem + kMaxCols, smem_desc_sw128(at), smem_desc_sw128(at + h * kPart * 128), idesc, k > 0);
    }
  };
  // this thread's row of that part: columns group * 32 .. + 31 of it
  auto read_part = [&](float* v) {
    tmem_ld16(lanes + kMaxCols + group * 32, v);
    tmem_ld16(lanes + kMaxCols + group * 32 + 16, v + 16);
    tc_fence_before();  // (the next part's product writes there)
  };

  for (int step = 0; step < p.steps; ++step) {
    // ------------------------------------------------------------------ A
    float* part = reinterpret_cast<float*>(smem + Smem::a);  // [column][row]
    for (int h = 0; h < parts; ++h) {
      float v[32] = {};
      if (width > 0) {
        multiply([&] { square(sbase + Smem::x, width / 16, h); });
        read_part(v);
      }
      const int c = h * kPart + group * 32;
      if (ctas == 1) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= kUnscale;
        store_row(smem + Smem::a, row, c, v);
        store_row(smem + Smem::a, row, c + 16, v + 16);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) part[(c + i) * kSide + row] = v[i];
      }
      __syncthreads();
      tc_fence_after();
    }
    if (ctas > 1) {
      cluster_sync_all();
      // the columns that are this CTA's, 4 rows of one a thread and turn: 1 to 8 turns
      const int own = parts * kPart / ctas, turns = (own * kSide + 4 * kThreads - 1) / (4 * kThreads);
      float4 sum[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int first = 4 * threadIdx.x;
      const uint32_t at = sbase + Smem::a + (uint32_t)(rank * own * kSide + first) * 4;
      auto add = [&](float4& s, const float4 v) { s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w); };
      // 8 reads on the way at once: of 8 / TURNS CTAs
      auto gather = [&](auto turns_of) {
        constexpr int TURNS = decltype(turns_of)::value;
        for (int k = 0; k < ctas && first < own * kSide; k += 8 / TURNS) {
          float4 v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = ld_cluster4(map_to_rank(at, min(k + j / TURNS, ctas - 1)) + j % TURNS * kThreads * 16);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (k + j / TURNS < ctas) add(sum[j % TURNS], v[j]);
        }
      };
      if (turns == 1) gather(std::integral_constant<int, 1>());
      else if (turns == 2) gather(std::integral_constant<int, 2>());
      else if (turns == 4) gather(std::integral_constant<int, 4>());
      else gather(std::integral_constant<int, 8>());
      cluster_sync_all();  // every CTA has read the parts: A may lie over them
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // elements (column, r .. r + 3) of the symmetric A, as its row `column`
        const int e = first + 4 * i * kThreads, column = rank * own + e / kSide, r = e % kSide;
        if (i < turns && e < own * kSide) {
          const uint32_t lo = pack_half(sum[i].x * kUnscale, sum[i].y * kUnscale);
          const uint32_t hi = pack_half(sum[i].z * kUnscale, sum[i].w * kUnscale);
          const uint32_t to = sbase + Smem::a + piece(column, r & ~7) + (r & 7) * 2;
          for (int k = 0; k < ctas; ++k) st_cluster2(map_to_rank(to, k), lo, hi);
        }
      }
      asm volatile("fence.proxy.async;" ::: "memory");
      cluster_sync_all();
    }
    fence_proxy_async_shared();
    __syncthreads();
    // ------------------------------------------------------- P = b A + c A A
    for (int h = 0; h < parts; ++h) {
      multiply([&] { square(sbase + Smem::a, steps_m, h); });
      float v[32];
      read_part(v);
      const int c = h * kPart + group * 32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(smem + Smem::a + piece(row, c + 8 * i));
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&words[j]));
          float* o = v + 8 * i + 2 * j;
          o[0] = fmaf(p.b, a.x, o[0] * p.c * kUnscale);
          o[1] = fmaf(p.b, a.y, o[1] * p.c * kUnscale);
        }
      }
      store_row(smem + Smem::p, row, c, v);
      store_row(smem + Smem::p, row, c + 16, v + 16);
      if (h + 1 == parts) fence_proxy_async_shared();
      __syncthreads();
      tc_fence_after();
    }
    // -------------------------------------------------------- X = a X + P X
    if (width > 0)
      multiply([&] {
        for (int c = 0; c < width; c += 256) {
          const uint32_t idesc = base | (1u << 16) | ((uint32_t)(min(256, width - c) >> 3) << 17);
          for (int k = 0; k < steps_m; ++k)
            mma_issue<false>(tmem + c, smem_desc_sw128(sbase + Smem::p + (k >> 2) * kBlockBytes + (k & 3) * 32),
                             desc_mn(sbase + Smem::x + (c >> 6) * kBlockBytes + k * 2048), idesc, 1);
        }
      });
    if (step + 1 < p.steps)
      settle([&](float* v) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] *= kUnscale;
      });
  }

  // ------------------------------------------------------------------ result
  float lr = 1.0f;
  if (UPDATE && p.lr) lr = __ldg(p.lr);
  const float keep = 1.0f - lr * p.decay, scale = lr * p.scale * kUnscale * kUnscale;
  const int64_t at = (int64_t)b * p.N * p.K;
  if (UPDATE && p.w_dtype == MOE_DTYPE_F32)
    finish<float, VEC, UPDATE>(p, static_cast<float*>(p.out) + at, keep, scale, row, col0, width, group, lanes);
  else
    finish<__nv_bfloat16, VEC, UPDATE>(p, static_cast<__nv_bfloat16*>(p.out) + at, keep, scale, row, col0, width, group,
                                       lanes);
  tc_fence_before();
  __syncthreads();
  if (ctas > 1) cluster_sync_all();  // no CTA's shared memory goes while another may use it
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

template <class T>
auto pick(int vec, bool update) {
  if (vec == 16) return update ? small_kernel<T, 16, true> : small_kernel<T, 16, false>;
  if (vec == 8) return update ? small_kernel<T, 8, true> : small_kernel<T, 8, false>;
  return update ? small_kernel<T, 1, true> : small_kernel<T, 1, false>;
}

// CTAs of a cluster: a power of two, as few as hold n columns; 0: none.
int cluster_of(int n) {
  for (int c = 1; c <= 16; c *= 2)
    if (n <= c * kMaxCols) return c;
  return 0;
}

}  // namespace

// Sides that fit take this way, however many matrices: 60 of 128 x 7168, 9 rounds of 7 clusters, 673 us against
// 996 by the general way, one 74 against 127; 1000 of 100 x 400, 287 against 1211.
bool orthogonalize_small_fits(int N, int K) {
  const int m = N < K ? N : K, n = N < K ? K : N;
  return m <= kSide && cluster_of(n) > 0;
}

cudaError_t launch_orthogonalize_small(const OrthoArgs& g, cudaStream_t s) {
  Args p{};
  p.g = g.g;
  p.batch = g.batch_stride;
  p.row = g.row_stride;
  p.dtype = g.dtype;
  p.momentum = g.momentum;
  p.mu = g.mu;
  p.nesterov = g.nesterov;
  p.N = g.N;
  p.K = g.K;
  p.tall = g.N > g.K;
  p.m = p.tall ? g.K : g.N;
  p.n = p.tall ? g.N : g.K;
  const int ctas = cluster_of(p.n);
  p.cols = ((p.n + ctas - 1) / ctas + 15) / 16 * 16;
  const auto lies = [&](unsigned bytes, int columns) {  // rows in pieces of so many columns, aligned to so many bytes
    const int64_t step = bytes / (g.dtype == MOE_DTYPE_F32 ? 4 : 2);
    const auto on = [&](const void* q) { return reinterpret_cast<uintptr_t>(q) % bytes == 0; };
    return !p.tall && g.K % columns == 0 && g.row_stride % step == 0 && g.batch_stride % step == 0 && on(g.g) &&
           on(g.momentum) && on(g.out);
  };
  const int vec = lies(32, 16) ? 16 : lies(16, 8) ? 8 : 1;
  p.steps = g.steps;
  p.a = g.coef[0];
  p.b = g.coef[1];
  p.c = g.coef[2];
  p.eps = g.eps;
  p.out = g.out;
  p.w_dtype = g.w_dtype;
  p.scale = g.scale;
  p.decay = g.decay;
  p.lr = g.lr;
  p.err = g.err;
  const auto kern = g.dtype == MOE_DTYPE_F32 ? pick<float>(vec, g.update) : pick<__nv_bfloat16>(vec, g.update);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(g.B * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, (const Args)p);
}

}  // namespace moe
