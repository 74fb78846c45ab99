// Orthogonalisation of a batch of matrices by Newton-Schulz products, and the momentum update
// of weights that applies it (include/moe_train.h), on the pair GEMM.
//
// X = G / (|G| + eps), then for each step, with m the shorter side and X seen as [m, n]:
//   A = X X^T      P = b A + c A A      X = a X + P X
// A and P are symmetric: only the tiles on and below the diagonal are computed, and each is
// stored a second time across it.
//
// Operands are fp16 scaled by 2^10.  Singular values stay below 4 (checked on the host for the
// coefficients), so the entries of X, A and P stay below 2^15 after the scaling, and what a
// matrix of 10^4 columns holds on average (10^-4 and less) stays above fp16's least normal
// number.  fp16 rounds eight times finer than bf16 at the same rate: against 64 bits the result
// of five steps on Gaussian matrices is off by 1.7e-3 of its norm, with bf16 by 1.1e-2.  X itself
// is kept in two fp16 (its value and what the first leaves): a X is added from both, because
// the iteration multiplies what lies in small singular values by a at each step, and the
// rounding of the large ones with it (few strong directions over a weak rest: 1.4e-2 off with
// one fp16).
//
// Bound by the products, and the power they take, where the sides are thousands: 8 matrices of 2048 x 7168,
// 2680 us in all; 2 of 5120 x 8192 with the update, 5290 (in a loop of calls, at the power limit, 2900 to 3040 and
// 5390 to 5620).  Products cannot be timed inside the one launch; as
// launches of their own, an earlier form, A, P and X took 171 to 180, 92 and 339 to 342 us, and 2 of
// 5120 x 8192 300 to 319, 213 to 229 and 566 to 588.  X's epilogue reads and writes its two halves.  By latency
// where they are hundreds: 3 of 517 x 1003, 146 us for 15 turns.
#include "common.cuh"
#include "launch.h"
#include "pair_gemm.cuh"
#include "train_launch.h"

namespace moe {
namespace {

using namespace pg;

constexpr float kScale = 1024.0f, kUnscale = 1.0f / kScale;
constexpr int kNormThreads = 256;

// ------------------------------------------------- momentum, norm, first iterate

struct Input {             // u: g itself, or g and the momentum
  const void* g;
  int64_t batch, row;      // strides of g, elements
  float* momentum;         // nullable; contiguous
  float mu;
  int nesterov;
  int N, K;
};

// Squares whose sum would overflow are summed a second time as multiples of 2^160.
constexpr float kDown = 0x1p-80f;

struct Squares {
  float plain = 0.0f, small = 0.0f;
  __device__ __forceinline__ void add(float u) {
    plain = fmaf(u, u, plain);
    const float d = u * kDown;
    small = fmaf(d, d, small);
  }
};

__device__ __forceinline__ float2 block_sum(float2 v) {
  __shared__ float2 s[kNormThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float2 t = s[0];
  for (int i = 1; i < kNormThreads / 32; ++i) {
    t.x += s[i].x;
    t.y += s[i].y;
  }
  return t;
}

// V neighbouring elements of a row: 8 where rows and bases allow 16-byte accesses, else 1.
template <int V>
__device__ __forceinline__ void load_values(const float* p, float* v) {
  if constexpr (V == 8) {
    *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
    *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(p + 4);
  } else {
    *v = *p;
  }
}
template <int V>
__device__ __forceinline__ void load_values(const __nv_bfloat16* p, float* v) {
  if constexpr (V == 8) bf16x8_to_f32(*reinterpret_cast<const uint4*>(p), v);
  else *v = __bfloat162float(*p);
}

// Every V elements of matrix b that are this thread's: of kAtOnce places at once the inputs are loaded
// first, so that their ways overlap.  take(row, column, g's values, the momentum's, its address)
template <class T, int V, bool MOMENTUM, class Take>
__device__ __forceinline__ void each_value(const Input& p, int b, Take take) {
  constexpr int kAtOnce = MOMENTUM ? 2 : 4;
  const uint32_t per_row = (uint32_t)p.K / V;
  const int64_t total = (int64_t)per_row * p.N, stride = gridDim.x * kNormThreads;  // total is below 2^32
  const T* g = static_cast<const T*>(p.g) + b * p.batch;
  float* momentum = MOMENTUM ? p.momentum + (int64_t)b * p.N * p.K : nullptr;
  for (int64_t i = blockIdx.x * kNormThreads + threadIdx.x; i < total; i += kAtOnce * stride) {
    float u[kAtOnce][V], m[kAtOnce][V];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t at = i + j * stride;
      if (at < total) {
        const uint32_t r = (uint32_t)at / per_row, c = (uint32_t)at - r * per_row;
        load_values<V>(g + r * p.row + c * V, u[j]);
        if (MOMENTUM) load_values<V>(momentum + at * V, m[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t at = i + j * stride;
      if (at < total) {
        const uint32_t r = (uint32_t)at / per_row, c = (uint32_t)at - r * per_row;
        take(r, c * V, u[j], m[j], momentum + at * V);
      }
    }
  }
}

// Matrix blockIdx.y: the momentum is updated, and the squares of u are summed into part.
template <class T, int V, bool MOMENTUM>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const Input p, float2* part, unsigned int* arrived) {
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *arrived = 0u;  // of the products' barriers
  Squares q;
  each_value<T, V, MOMENTUM>(p, blockIdx.y, [&](uint32_t, uint32_t, const float* u, const float* m, float* to) {
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      v[k] = MOMENTUM ? fmaf(p.mu, m[k], u[k]) : u[k];
      q.add(MOMENTUM && p.nesterov ? fmaf(p.mu, v[k], u[k]) : v[k]);
    }
    if constexpr (MOMENTUM && V == 8) {
      reinterpret_cast<float4*>(to)[0] = *reinterpret_cast<const float4*>(v);
      reinterpret_cast<float4*>(to)[1] = *reinterpret_cast<const float4*>(v + 4);
    } else if constexpr (MOMENTUM) {
      *to = *v;
    }
  });
  const float2 t = block_sum(make_float2(q.plain, q.small));
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = t;
}

// X = u / (|u| + eps), scaled, in two fp16 with rows ld elements apart.
template <class T, int V, bool MOMENTUM>
__global__ void __launch_bounds__(kNormThreads) first_kernel(const Input p, const float2* part, int parts, float eps,
                                                             __half* hi, __half* lo, int ld) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y;
  float2 t = make_float2(0.0f, 0.0f);
  for (int i = threadIdx.x; i < parts; i += kNormThreads) {
    const float2 v = part[(int64_t)b * parts + i];
    t.x += v.x;
    t.y += v.y;
  }
  t = block_sum(t);
  const bool big = isinf(t.x);
  const float pre = big ? kDown : 1.0f;
  const float f = kScale / (sqrtf(big ? t.y : t.x) + eps * pre);
  each_value<T, V, MOMENTUM>(p, b, [&](uint32_t r, uint32_t c, const float* u, const float* m, float*) {
    __half h[V], l[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float x = (MOMENTUM ? (p.nesterov ? fmaf(p.mu, m[k], u[k]) : m[k]) : u[k]) * pre * f;
      h[k] = __float2half_rn(x);
      l[k] = __float2half_rn(x - __half2float(h[k]));
    }
    const int64_t o = ((int64_t)b * p.N + r) * ld + c;
    if constexpr (V == 8) {
      *reinterpret_cast<uint4*>(hi + o) = *reinterpret_cast<const uint4*>(h);
      *reinterpret_cast<uint4*>(lo + o) = *reinterpret_cast<const uint4*>(l);
    } else {
      hi[o] = *h;
      lo[o] = *l;
    }
  });
}

// ------------------------------------------------------------------ products

// A tile of 256 rows (lanes) x n columns of a [rows, cols] result of one matrix.
struct MatTile {
  int n, k;
  int at, row, col;    // the matrix, first row and first column
  int k0, split;       // where its part of the reduction begins, and which part that is
  bool mirror;         // symmetric results: stored across the diagonal too
};

// How a product ends: A, a part of A, alpha * src + beta * product (symmetric), the same with two sources
// (src and lo), X's next iterate, and what the call asked for.
enum Product { kGram, kPartial, kOneSource, kTwoSources, kNext, kOut, kWeights };

struct Dims {
  int count, rows, cols;  // of the result
  int ct;                 // tiles along its columns
  int per;                // tiles of a matrix
  int k;                  // the reduction's length
  int splits, part_k;     // kPartial: parts of the reduction, and the length of one
};

// 32 bytes of a lane.  (Next iterates through boxes in shared memory and TMA instead, which a third of the
// L1 cache's passes would go without: 3% on 8 matrices of 7168 x 2048, 1% on 16 of 2048 x 7168, and 1% more
// time on 2 of 5120 x 8192, whose long reductions miss the stage that made room.)
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

struct Result {
  __half* sym;          // symmetric results, rows ldm elements apart
  const __half* src;    // X: its first half
  __half* next;         // X's next first half
  __half* lo;           // X's second half, in place; the second source
  float* partial;       // A's parts: [splits][count][rows] of ld
  void* out;            // bf16 result, or weights
  int ld;               // of sym and src's matrices; X: of src, next and lo
  float alpha, beta;    // result = alpha * src + beta * product
  float scale, keep;    // out = scale * result, or keep * w - scale * result
  const float* lr;      // nullable: multiplies scale, and what keep takes from 1
  int w_dtype;
  bool whole;           // out's chunks are whole and 32-byte aligned
};

constexpr bool symmetric(Product k) { return k == kGram || k == kOneSource || k == kTwoSources; }
constexpr bool moves_x(Product k) { return k == kNext || k == kOut || k == kWeights; }
constexpr bool has_source(Product k) { return moves_x(k) || k == kOneSource || k == kTwoSources; }
constexpr bool has_second(Product k) { return moves_x(k) || k == kTwoSources; }
constexpr int kWords = kChunk / 2;

template <bool AMN, bool BMN, Product KIND>
struct Ns {
  static constexpr bool kAMN = AMN, kBMN = BMN, kF16 = true;
  struct Params {
    const CUtensorMap *a, *b;  // b: by box height where it is K-major
    Dims d;
    Result r;
  };
  using Tile = MatTile;
  // Symmetric results: the tiles of row block >= column block.
  static __device__ __forceinline__ Tile tile(const Params& p, const int*, int i) {
    const Dims& d = p.d;
    Tile t;
    t.at = i / d.per;
    int l = i - t.at * d.per, r, c;
    t.k0 = t.split = 0;
    t.k = d.k;
    t.mirror = false;
    if (KIND == kPartial) {
      t.split = l % d.splits;
      l /= d.splits;
      t.k0 = t.split * d.part_k;
      t.k = min(d.part_k, d.k - t.k0);
    }
    if (symmetric(KIND)) {  // row block r has the column blocks 0 .. r
      r = (int)((sqrtf(8.0f * (float)l + 1.0f) - 1.0f) * 0.5f);
      while (r * (r + 1) / 2 > l) --r;
      while ((r + 1) * (r + 2) / 2 <= l) ++r;
      c = l - r * (r + 1) / 2;
      t.mirror = c != r;
    } else {
      r = l / d.ct;
      c = l - r * d.ct;
    }
    t.row = r * kTileM;
    t.col = c * kMaxN;
    t.n = min(kMaxN, (d.cols - t.col + 31) / 32 * 32);
    return t;
  }
  static __device__ __forceinline__ void narrow(Tile* t, int part, int parts) {
    const int n = ((t->n + parts - 1) / parts + 31) / 32 * 32, from = part * n;
    t->col += from;
    t->n = max(0, min(n, t->n - from));
  }
  static __device__ __forceinline__ uint32_t stage_bytes(const Params&, const Tile& t) {
    return 2u * (uint32_t)(kOperandBytes + (BMN ? kOperandBytes : t.n / 2 * 128 * (kBK / 64)));
  }
  static __device__ __forceinline__ void load(const Params& p, const Tile& t, int rank, int block, uint32_t a, uint32_t b,
                                              uint32_t bar) {
    const int k = t.k0 + block * kBK;
    load_half<AMN>(a, p.a, bar, k, t.row + rank * kHalfM, t.at);
    load_half<BMN>(b, p.b + (BMN ? 0 : t.n / 32 - 1), bar, k, t.col + rank * (t.n / 2), t.at);
  }
  struct Source {  // a chunk of a row of the sources, and of the weights
    uint32_t hi[has_source(KIND) ? kWords : 1], lo[has_second(KIND) ? kWords : 1];
    uint32_t w[KIND == kWeights ? kChunk : 1];
  };
  static __device__ __forceinline__ float2 halves(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack_half(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  template <class Wait, class Release>
  static __device__ void epilogue(const Params& p, const Tile& t, int rank, int sub, int group, int lane, uint32_t tbase,
                                  Wait wait, Release release) {
    const Result& g = p.r;
    const int row = t.row + rank * kHalfM + sub * 32 + lane;
    const bool keep = row < p.d.rows;
    const int cols = min(t.n, p.d.cols - t.col);
    // rows of the workspace are multiples of kChunk apart: whole chunks are read and written, what lies past
    // the columns is not read as an operand
    const int64_t matrix = (int64_t)t.at * p.d.rows * g.ld;
    const int64_t at = matrix + (int64_t)(keep ? row : 0) * g.ld + t.col;
    const int64_t out_at = ((int64_t)t.at * p.d.rows + (keep ? row : 0)) * p.d.cols + t.col;
    float lr = 1.0f;
    if (KIND == kWeights && g.lr) lr = __ldg(g.lr);
    const float w_keep = 1.0f - lr * g.keep, w_scale = lr * g.scale;
    const bool f32 = KIND == kWeights && g.w_dtype == MOE_DTYPE_F32;
    auto load = [&](int c, Source& s) {
      if constexpr (has_source(KIND)) load32(g.src + at + c, s.hi);
      if constexpr (has_second(KIND)) load32(g.lo + at + c, s.lo);
      if constexpr (KIND == kWeights) {
        if (g.whole) {
          if (f32) {
            load32(static_cast<const float*>(g.out) + out_at + c, s.w);
            load32(static_cast<const float*>(g.out) + out_at + c + 8, s.w + 8);
          } else {
            load32(static_cast<const __nv_bfloat16*>(g.out) + out_at + c, s.w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            const int64_t o = out_at + min(c + i, cols - 1);
            s.w[i] = f32 ? static_cast<const uint32_t*>(g.out)[o] : static_cast<const uint16_t*>(g.out)[o];
          }
        }
      }
    };
    auto part = [&](int c, const Source&, const float* v) {
      float* o = g.partial + (int64_t)t.split * p.d.count * p.d.rows * g.ld + at + c;
      if (keep) {
        store32(o, reinterpret_cast<const uint32_t*>(v));
        store32(o + 8, reinterpret_cast<const uint32_t*>(v) + 8);
      }
    };
    auto use = [&](int c, const Source& s, float* v) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float2 x = make_float2(v[2 * i] * g.beta, v[2 * i + 1] * g.beta);
        if constexpr (has_source(KIND)) {
          const float2 h = halves(s.hi[i]);
          x = make_float2(fmaf(g.alpha, h.x, x.x), fmaf(g.alpha, h.y, x.y));
        }
        if constexpr (has_second(KIND)) {
          const float2 l = halves(s.lo[i]);
          x = make_float2(fmaf(g.alpha, l.x, x.x), fmaf(g.alpha, l.y, x.y));
        }
        v[2 * i] = x.x;
        v[2 * i + 1] = x.y;
      }
      if constexpr (symmetric(KIND) || KIND == kNext) {
        uint32_t hi[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) hi[i] = pack_half(v[2 * i], v[2 * i + 1]);
        if (keep) store32((symmetric(KIND) ? g.sym : g.next) + at + c, hi);
        if constexpr (KIND == kNext) {
          uint32_t lo[kWords];
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const float2 h = halves(hi[i]);
            lo[i] = pack_half(v[2 * i] - h.x, v[2 * i + 1] - h.y);
          }
          if (keep) store32(g.lo + at + c, lo);
        } else if (t.mirror) {  // the same across the diagonal, by columns
          const bool odd = lane & 1;
          __half* m = g.sym + matrix + (int64_t)(t.col + c + odd) * g.ld + (row & ~1);
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            const float2 w = deal(v, j, odd);
            // (an odd last row's pair writes one element into the padding)
            if ((row & ~1) < p.d.rows && c + 2 * j + odd < cols)
              *reinterpret_cast<uint32_t*>(m + (int64_t)(2 * j) * g.ld) = pack_half(w.x, w.y);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          if (KIND == kOut) {
            v[i] *= g.scale;
          } else {
            const uint32_t w = f32 ? s.w[i] : g.whole ? (i & 1 ? s.w[i / 2] & 0xffff0000u : s.w[i / 2] << 16) : s.w[i] << 16;
            v[i] = w_keep * __uint_as_float(w) - w_scale * v[i];
          }
        }
        if (!keep) return;
        if (f32) {
          float* o = static_cast<float*>(g.out) + out_at + c;
          if (g.whole) {
            store32(o, reinterpret_cast<const uint32_t*>(v));
            store32(o + 8, reinterpret_cast<const uint32_t*>(v) + 8);
          } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
              if (c + i < cols) o[i] = v[i];
          }
        } else {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(g.out) + out_at + c;
          if (g.whole) {
            uint32_t w[kWords];
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
              w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            store32(o, w);
          } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
              if (c + i < cols) o[i] = __float2bfloat16_rn(v[i]);
          }
        }
      }
    };
    if constexpr (KIND == kPartial) by_chunks<Source>(cols, group, tbase, load, part, wait, release);
    else by_chunks<Source>(cols, group, tbase, load, use, wait, release);
  }
};

// ------------------------------------------------------------------ iteration

// All products of a call in one launch, with a barrier over the grid between them: of small matrices a
// product's launch, prologue and first loads took 8 us each.  The epilogue's warps arrive when a CTA's
// results are stored; they and the producer wait.
//
// The first two steps may be made one (twice): with M = aI + P, the next A is M A M, so it follows from
// products of m x m matrices, and X takes both steps at once:
//   T = a A + A P,  A' = a T + P T,  P' = b A' + c A' A',  W = a P + a P' + P' P,  X = a^2 X + W X
// which saves a pass over X for A and one product of 2 m m n for three of m m m (symmetric: half each).
// The roundings cost what they cost in two steps, because A is far from I there; made one later, or
// four made two, they do not (Gaussian 512 x 2048: 1.7e-3 of the norm as it is and with the first two,
// 4.1e-3 with the last two, 2.6e-3 with the first four).
enum Op { oGram, oPartial, oReduce, oPoly, oTimes, oNextGram, oNextPoly, oBoth, oX };

struct Plan {
  CUtensorMap x_rows[2], x_cols[2];        // X as A: boxes of 128 rows, or of kBK rows x 64 columns
  CUtensorMap x_low[2][kHeights];          // X as a K-major B
  CUtensorMap q[3], q_low[3][kHeights];    // the square matrices as A and as B
  Dims sym, sym_square, square;            // A, the products of square matrices, X
  __half *x[2], *lo, *m[3];                // m: A (then A', W), P, and T (then P')
  float* partial;
  int steps, twice, side, ldx, ldm;
  float coef[3];
  Result last;                             // out and what goes with it
  unsigned int* arrived;
  unsigned int* err;
};

constexpr int kStages = 6;
constexpr int kEpiThreads = 32 * kEpiWarps;
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

// Until `target` CTAs have arrived (bounded).
__device__ __forceinline__ bool wait_grid(const Block<kStages>& b, const unsigned int* arrived, unsigned int target) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(arrived) : "memory");
    if (v >= target) return true;
    if (i == 0) t0 = global_timer_ns();
    if ((i & 63) == 63 && (*b.abort || global_timer_ns() - t0 > kWaitTimeoutNs)) return false;
  }
}

// A from its parts, added in order: 8 elements a thread.
__device__ __forceinline__ void reduce_parts(const Plan& p, int thread) {
  const int64_t size = (int64_t)p.sym.count * p.side * p.ldm;
  for (int64_t i = ((int64_t)blockIdx.x * kEpiThreads + thread) * 8; i < size; i += (int64_t)gridDim.x * kEpiThreads * 8) {
    float v[8] = {};
#pragma unroll 4
    for (int s = 0; s < p.sym.splits; ++s) {
      uint32_t w[8];
      load32(p.partial + s * size + i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(w[j]);
    }
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 x = __floats2half2_rn(v[2 * j] * kUnscale, v[2 * j + 1] * kUnscale);
      h[j] = *reinterpret_cast<const uint32_t*>(&x);
    }
    *reinterpret_cast<uint4*>(p.m[0] + i) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// One of the call's products: what it is, which iterate of X it reads, and whether X takes two steps or ends.
struct Turn {
  Op op;
  int cur;
  bool both, last;
};

// Calls role(policy, its parameters) for a turn.
template <bool TALL, Product LAST, class Role>
__device__ __forceinline__ bool product(const Plan& p, const Turn& turn, Role role) {
  const int cur = turn.cur;
  const float a0 = p.coef[0];
  Result r = p.last;
  if (turn.op == oGram || turn.op == oPartial) {
    r.sym = p.m[0];
    r.partial = p.partial;
    r.ld = p.ldm;
    r.beta = kUnscale;
    const CUtensorMap* a = TALL ? &p.x_cols[cur] : &p.x_rows[cur];
    const CUtensorMap* b = TALL ? &p.x_cols[cur] : p.x_low[cur];
    using G = Ns<TALL, TALL, kGram>;
    using S = Ns<TALL, TALL, kPartial>;
    if (turn.op == oGram) return role(G(), typename G::Params{a, b, p.sym, r});
    return role(S(), typename S::Params{a, b, p.sym, r});
  }
  if (turn.op == oBoth) {
    using W = Ns<false, false, kTwoSources>;
    r.sym = p.m[0];
    r.src = p.m[1];
    r.lo = p.m[2];
    r.ld = p.ldm;
    r.alpha = a0;
    r.beta = kUnscale;
    return role(W(), typename W::Params{&p.q[2], p.q_low[1], p.sym_square, r});
  }
  if (turn.op != oX) {
    using P = Ns<false, false, kOneSource>;
    const bool poly = turn.op == oPoly || turn.op == oNextPoly;
    const int to = turn.op == oPoly ? 1 : turn.op == oNextGram ? 0 : 2;
    const int src = turn.op == oNextGram ? 2 : 0, a = turn.op == oNextGram ? 1 : 0;
    const int b = turn.op == oTimes ? 1 : turn.op == oNextGram ? 2 : 0;
    r.sym = p.m[to];
    r.src = p.m[src];
    r.ld = p.ldm;
    r.alpha = poly ? p.coef[1] : a0;
    r.beta = poly ? p.coef[2] * kUnscale : kUnscale;
    return role(P(), typename P::Params{&p.q[a], p.q_low[b], p.sym_square, r});
  }
  // X [N, K]: P X (wide: P's rows, X's columns) or X P (tall: X's rows, P's rows, as P is symmetric)
  r.src = p.x[cur];
  r.next = p.x[cur ^ 1];
  r.lo = p.lo;
  r.ld = p.ldx;
  r.alpha = turn.both ? a0 * a0 : a0;
  r.beta = kUnscale;
  const int by = turn.both ? 0 : 1;
  const CUtensorMap* a = TALL ? &p.x_rows[cur] : &p.q[by];
  const CUtensorMap* b = TALL ? p.q_low[by] : &p.x_cols[cur];
  using N = Ns<false, !TALL, kNext>;
  using L = Ns<false, !TALL, LAST>;
  if (!turn.last) return role(N(), typename N::Params{a, b, p.square, r});
  return role(L(), typename L::Params{a, b, p.square, r});
}

template <bool TALL, Product LAST>
__global__ void __launch_bounds__(kThreads, 1) iterate_kernel(const __grid_constant__ Plan p) {
  extern __shared__ uint8_t smem_raw[];
  Block<kStages> b;
  b.begin(smem_raw, p.err);
  b.meet();
  // the products in order, with how many barriers lie before each
  auto all = [&](auto run) {
    unsigned int before = 0;
    bool ok = true;
    for (int step = 0, cur = 0; step < p.steps && ok; cur ^= 1) {
      const bool both = step == 0 && p.twice;
      step += both ? 2 : 1;
      auto turn = [&](Op op) {
        if (ok) ok = run(Turn{op, cur, both, op == oX && step >= p.steps}, before++);
      };
      if (p.sym.splits > 1) {
        turn(oPartial);
        turn(oReduce);
      } else {
        turn(oGram);
      }
      turn(oPoly);
      if (both) {
        turn(oTimes);
        turn(oNextGram);
        turn(oNextPoly);
        turn(oBoth);
      }
      turn(oX);
    }
    return ok;
  };
  auto walk = [&](const auto& params, auto policy) {
    using P = decltype(policy);
    return Walk<P>(params, nullptr, params.d.count * params.d.per, b.pair, b.pairs);
  };
  if (b.warp == 0) {
    if (b.lane == 0) {
      Producer<kStages> r(b);
      r.finish(all([&](const Turn& turn, unsigned int before) {
        if (turn.op == oReduce) return true;
        if (!wait_grid(b, p.arrived, before * gridDim.x)) return false;
        asm volatile("fence.proxy.async.global;" ::: "memory");  // the loads see what other CTAs stored
        return product<TALL, LAST>(p, turn, [&](auto policy, const auto& params) {
          return r.template run<decltype(policy)>(params, walk(params, policy));
        });
      }));
    }
  } else if (b.warp == 1) {
    if (b.rank == 0) {
      Issuer<kStages> r(b);
      r.finish(all([&](const Turn& turn, unsigned int) {
        if (turn.op == oReduce) return true;
        return product<TALL, LAST>(p, turn, [&](auto policy, const auto& params) {
          return r.template run<decltype(policy)>(walk(params, policy));
        });
      }));
    }
  } else {
    Epilogue<kStages> r(b);
    const int thread = threadIdx.x - 64;
    int* s_ok = b.tables();
    all([&](const Turn& turn, unsigned int before) {
      if (turn.op == oReduce) {
        reduce_parts(p, thread);
      } else {  // (a warp that gives up raises the abort flag, and stays for the barriers)
        product<TALL, LAST>(p, turn, [&](auto policy, const auto& params) {
          return r.template run<decltype(policy)>(params, walk(params, policy));
        });
      }
      if (turn.last) return true;
      // this CTA's results are stored; then those of all
      epilogue_sync();
      if (thread == 0) {  // (the release covers what the other warps stored before the barrier)
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.arrived) : "memory");
        const bool all_here = wait_grid(b, p.arrived, (before + 1) * gridDim.x);
        if (!all_here) b.fail();
        *s_ok = all_here && !*b.abort;
      }
      epilogue_sync();
      return *s_ok != 0;
    });
  }
  b.end();
}

// ------------------------------------------------------------------- host

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Blocks of a matrix in the passes over G, 32 elements a thread or more.  They go by the matrix alone, so
// that its norm is the same in any batch.
int norm_blocks(const OrthoArgs& g) {
  const int64_t want = ((int64_t)g.N * g.K + 32 * kNormThreads - 1) / (32 * kNormThreads);
  return (int)(want < 1024 ? want : 1024);
}

constexpr int kPairsGB300 = kNumSmsGB300 / 2;
// A's reduction is split where its tiles are few and each would take long: what it saves, in blocks of
// kBK, has to be worth a barrier and a pass over the parts (about 4 us).
constexpr int kWorthSplitting = 24;

// The first two steps are made one where that saves 3 B m m (n - m) operations or more: the turn that it adds
// takes about 5 us, 7e9 operations.
constexpr double kWorthTwice = 5e9;

struct Layout {
  int m, ldx, ldm, splits;
  bool twice;
  size_t arrived, part, x0, x1, lo, m0, m1, m2, partial, total;  // offsets
};

Layout layout(const OrthoArgs& g) {
  Layout l;
  l.m = g.N < g.K ? g.N : g.K;
  l.ldx = (int)up(g.K, kChunk);
  l.ldm = (int)up(l.m, kChunk);
  const int64_t side = (l.m + kTileM - 1) / kTileM, blocks = ((g.N < g.K ? g.K : g.N) + kBK - 1) / kBK;
  int64_t splits = kPairsGB300 / (g.B * side * side);
  if (splits > blocks / 4) splits = blocks / 4;
  l.splits = splits > 1 && blocks - blocks / splits >= kWorthSplitting ? (int)splits : 1;
  const size_t x = up((int64_t)g.B * g.N * l.ldx * 2, 256), sym = up((int64_t)g.B * l.m * l.ldm * 2, 256);
  l.arrived = 0;
  l.part = 256;
  l.x0 = l.part + up((int64_t)g.B * norm_blocks(g) * (int64_t)sizeof(float2), 256);
  l.x1 = l.x0 + x;
  l.lo = l.x1 + x;
  // (the same for any number of steps and coefficients: it goes into the workspace's size)
  l.twice = l.splits == 1 && (double)g.B * l.m * l.m * ((double)(g.N < g.K ? g.K : g.N) - l.m) >= kWorthTwice;
  l.m0 = l.lo + x;
  l.m1 = l.m0 + sym;
  l.m2 = l.m1 + sym;
  l.partial = l.m2 + (l.twice ? sym : 0);
  l.total = l.partial + (l.splits > 1 ? 2 * sym * l.splits : 0);
  return l;
}

// For coefficients that fit: whether the polynomial of the first two steps, but for its linear term, stays in that
// range as well.  It is of degree 12 in s^2: between these points it exceeds its largest value at them by less than
// 2%, and the kernels' range ends at twice the limit.
bool two_steps_fit(const float* c) {
  for (int i = 0; i <= 1024; ++i) {
    double s = i / 1024.0, m = 1.0;
    for (int k = 0; k < 2; ++k) {
      const double p = (c[1] + c[2] * s * s) * s * s;
      m *= c[0] + p;
      s = fabs((c[0] + p) * s);
    }
    if (!(fabs(m - c[0] * c[0]) < 32.0)) return false;
  }
  return true;
}

// The tiles of a result [rows, cols] of each matrix; reduction over k.
bool make_dims(Dims* d, int B, int rows, int cols, int k, bool sym, int splits) {
  const int rt = (rows + kTileM - 1) / kTileM;
  d->count = B;
  d->rows = rows;
  d->cols = cols;
  d->ct = (cols + kMaxN - 1) / kMaxN;
  d->k = k;
  d->splits = splits;
  const int blocks = (k + kBK - 1) / kBK;
  d->part_k = (blocks + splits - 1) / splits * kBK;
  d->splits = (k + d->part_k - 1) / d->part_k;  // parts that are not empty
  const int64_t per = sym && splits == 1 ? (int64_t)rt * (rt + 1) / 2 : (int64_t)rt * d->ct * d->splits;
  if (per * B > INT32_MAX / 16) return false;
  d->per = (int)per;
  return true;
}

template <bool TALL, Product LAST>
cudaError_t iterate(const OrthoArgs& g, const Layout& l, char* ws, cudaStream_t s) {
  Plan p{};
  const int n = TALL ? g.N : g.K;
  if (!make_dims(&p.sym, g.B, l.m, l.m, n, true, l.splits) || !make_dims(&p.sym_square, g.B, l.m, l.m, l.m, true, 1) ||
      !make_dims(&p.square, g.B, g.N, g.K, l.m, false, 1))
    return cudaErrorNotSupported;
  p.x[0] = reinterpret_cast<__half*>(ws + l.x0);
  p.x[1] = reinterpret_cast<__half*>(ws + l.x1);
  p.lo = reinterpret_cast<__half*>(ws + l.lo);
  p.m[0] = reinterpret_cast<__half*>(ws + l.m0);
  p.m[1] = reinterpret_cast<__half*>(ws + l.m1);
  p.m[2] = reinterpret_cast<__half*>(ws + l.m2);
  p.partial = reinterpret_cast<float*>(ws + l.partial);
  p.twice = l.twice && g.steps >= 2 && two_steps_fit(g.coef);
  auto map = [&](CUtensorMap* to, const void* x, bool of_x, int box) {
    return of_x ? make_map_3d(to, x, true, g.B, g.N, g.K, l.ldx, box) : make_map_3d(to, x, true, g.B, l.m, l.m, l.ldm, box);
  };
  bool ok = true;
  for (int i = 0; i < 2 && ok; ++i) ok = map(&p.x_rows[i], p.x[i], true, kHalfM) && map(&p.x_cols[i], p.x[i], true, kBK);
  for (int i = 0; i < (p.twice ? 3 : 2) && ok; ++i) ok = map(&p.q[i], p.m[i], false, kHalfM);
  for (int h = 0; h < kHeights && ok; ++h) {
    for (int i = 0; i < (p.twice ? 3 : 2) && ok; ++i) ok = map(&p.q_low[i][h], p.m[i], false, box_rows(h));
    for (int i = 0; i < 2 && ok && !TALL; ++i) ok = map(&p.x_low[i][h], p.x[i], true, box_rows(h));
  }
  if (!ok) return cudaErrorInvalidValue;
  p.steps = g.steps;
  p.side = l.m;
  p.ldx = l.ldx;
  p.ldm = l.ldm;
  for (int i = 0; i < 3; ++i) p.coef[i] = g.coef[i];
  p.last.out = g.out;
  p.last.scale = kUnscale * g.scale;
  p.last.keep = g.decay;
  p.last.lr = g.lr;
  p.last.w_dtype = g.w_dtype;
  p.last.whole = g.K % kChunk == 0 && (reinterpret_cast<uintptr_t>(g.out) & 31) == 0;
  p.arrived = reinterpret_cast<unsigned int*>(ws + l.arrived);
  p.err = g.err;
  // no more pairs than the product with the most tiles, cut as they may be, has work for
  int64_t most = p.sym.per > p.square.per ? p.sym.per : p.square.per;
  most *= (int64_t)g.B * (kMaxN / 32);
  Launch launch;
  const auto kern = iterate_kernel<TALL, LAST>;
  cudaError_t e = launch.prepare(kern, Smem<kStages>::bytes(16), most, s);
  if (e != cudaSuccess) return e;
  launch.attr[1].id = cudaLaunchAttributeCooperative;  // the CTAs wait for one another: all are resident
  launch.attr[1].val.cooperative = 1;
  launch.cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&launch.cfg, kern, p);
}

// The norms and the first iterate.
template <class T, int V, bool MOMENTUM>
cudaError_t begin(const OrthoArgs& g, const Layout& l, char* ws, cudaStream_t s) {
  Input in{};
  in.g = g.g;
  in.batch = g.batch_stride;
  in.row = g.row_stride;
  in.momentum = g.momentum;
  in.mu = g.mu;
  in.nesterov = g.nesterov;
  in.N = g.N;
  in.K = g.K;
  float2* part = reinterpret_cast<float2*>(ws + l.part);
  const int parts = norm_blocks(g);
  const dim3 grid(parts, g.B);
  norm_kernel<T, V, MOMENTUM><<<grid, kNormThreads, 0, s>>>(in, part, reinterpret_cast<unsigned int*>(ws + l.arrived));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kNormThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, first_kernel<T, V, MOMENTUM>, (const Input)in, (const float2*)part, parts, g.eps,
                            reinterpret_cast<__half*>(ws + l.x0), reinterpret_cast<__half*>(ws + l.lo), l.ldx);
}

}  // namespace

size_t orthogonalize_workspace_bytes(int B, int N, int K) {
  if (orthogonalize_small_fits(N, K)) return 0;
  OrthoArgs g{};
  g.B = B;
  g.N = N;
  g.K = K;
  return layout(g).total;
}

cudaError_t launch_orthogonalize(const OrthoArgs& g, cudaStream_t s) {
  if (orthogonalize_small_fits(g.N, g.K)) return launch_orthogonalize_small(g, s);
  const Layout l = layout(g);
  char* ws = static_cast<char*>(g.ws);
  const auto whole = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vector = g.K % 8 == 0 && g.row_stride % 8 == 0 && g.batch_stride % 8 == 0 && whole(g.g) && whole(g.momentum);
  const bool f32 = g.dtype == MOE_DTYPE_F32;
  cudaError_t e;
  if (g.momentum) {
    if (vector) e = f32 ? begin<float, 8, true>(g, l, ws, s) : begin<__nv_bfloat16, 8, true>(g, l, ws, s);
    else e = f32 ? begin<float, 1, true>(g, l, ws, s) : begin<__nv_bfloat16, 1, true>(g, l, ws, s);
  } else {
    if (vector) e = f32 ? begin<float, 8, false>(g, l, ws, s) : begin<__nv_bfloat16, 8, false>(g, l, ws, s);
    else e = f32 ? begin<float, 1, false>(g, l, ws, s) : begin<__nv_bfloat16, 1, false>(g, l, ws, s);
  }
  if (e != cudaSuccess) return e;
  if (g.update) return g.N > g.K ? iterate<true, kWeights>(g, l, ws, s) : iterate<false, kWeights>(g, l, ws, s);
  return g.N > g.K ? iterate<true, kOut>(g, l, ws, s) : iterate<false, kOut>(g, l, ws, s);
}

}  // namespace moe
