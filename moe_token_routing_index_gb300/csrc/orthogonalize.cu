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
  const uint32_t per_row = (uint32_t)p.K / V, total = per_row * (uint32_t)p.N;
  const uint32_t stride = gridDim.x * kNormThreads;
  const T* g = static_cast<const T*>(p.g) + b * p.batch;
  float* momentum = MOMENTUM ? p.momentum + (int64_t)b * p.N * p.K : nullptr;
  for (uint32_t i = blockIdx.x * kNormThreads + threadIdx.x; i < total; i += kAtOnce * stride) {
    float u[kAtOnce][V], m[kAtOnce][V];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const uint32_t at = i + j * stride;
      if (at >= i && at < total) {  // (the sum may pass 32 bits)
        const uint32_t r = at / per_row, c = at - r * per_row;
        load_values<V>(g + r * p.row + c * V, u[j]);
        if (MOMENTUM) load_values<V>(momentum + (int64_t)at * V, m[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const uint32_t at = i + j * stride;
      if (at >= i && at < total) take(at / per_row, at % per_row * V, u[j], m[j], momentum + (int64_t)at * V);
    }
  }
}

// Matrix blockIdx.y: the momentum is updated, and the squares of u are summed into part.
template <class T, int V, bool MOMENTUM>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const Input p, float2* part) {
  pdl_launch_dependents();
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
  // (a sum that overflowed means entries above 2^60: eps is far below the norm)
  const bool big = isinf(t.x);
  const float pre = big ? kDown : 1.0f;
  const float f = kScale / (big ? sqrtf(t.y) : sqrtf(t.x) + eps);
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
  bool mirror;         // symmetric results: stored across the diagonal too
};

struct Mats {
  CUtensorMap a, b[kHeights];
  int count, rows, cols;  // of the result
  int ct, rt;             // tiles along its columns and rows
  int per;                // tiles of a matrix
  int k;                  // the reduction's length
};

// SYM: the tiles of row block >= column block (cols == rows).
template <bool SYM>
__device__ __forceinline__ MatTile locate_mat(const Mats& p, int i) {
  MatTile t;
  t.at = i / p.per;
  const int l = i - t.at * p.per;
  int r, c;
  if (SYM) {  // row block r has the column blocks 0 .. r
    r = (int)((sqrtf(8.0f * (float)l + 1.0f) - 1.0f) * 0.5f);
    while (r * (r + 1) / 2 > l) --r;
    while ((r + 1) * (r + 2) / 2 <= l) ++r;
    c = l - r * (r + 1) / 2;
    t.mirror = c != r;
  } else {
    r = l / p.ct;
    c = l - r * p.ct;
    t.mirror = false;
  }
  t.row = r * kTileM;
  t.col = c * kMaxN;
  t.n = min(kMaxN, (p.cols - t.col + 31) / 32 * 32);
  t.k = p.k;
  return t;
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

enum Product { kGram, kPolynomial, kNext, kOut, kWeights };

struct Result {
  __half* sym;          // A or P, rows ldm elements apart
  const __half* src;    // P: A.  X: its first half
  __half* next;         // X's next first half
  __half* lo;           // X's second half, in place
  void* out;            // bf16 result, or weights
  int ld;               // of sym and src's matrices; X: of src, next and lo
  float alpha, beta;    // result = alpha * src + beta * product
  float scale, keep;    // out = scale * result, or keep * w - scale * result
  const float* lr;      // nullable: multiplies scale, and what keep takes from 1
  int w_dtype;
  bool whole;           // out's chunks are whole and 32-byte aligned
};

template <bool AMN, bool BMN, Product KIND>
struct Ns {
  static constexpr bool kAMN = AMN, kBMN = BMN, kF16 = true;
  static constexpr bool kSym = KIND == kGram || KIND == kPolynomial;
  struct Params {
    Mats m;
    Result r;
    unsigned int* err;
  };
  using Tile = MatTile;
  static __device__ int setup(const Params& p, int*) { return p.m.count * p.m.per; }
  static __device__ void narrow(Tile* t, int part, int parts) {
    const int n = ((t->n + parts - 1) / parts + 31) / 32 * 32, from = part * n;
    t->col += from;
    t->n = max(0, min(n, t->n - from));
  }
  static __device__ Tile tile(const Params& p, const int*, int i) { return locate_mat<kSym>(p.m, i); }
  static __device__ uint32_t stage_bytes(const Params&, const Tile& t) {
    return 2u * (uint32_t)(kOperandBytes + (BMN ? kOperandBytes : t.n / 2 * 128 * (kBK / 64)));
  }
  static __device__ void load(const Params& p, const Tile& t, int rank, int block, uint32_t a, uint32_t b,
                              uint32_t bar) {
    load_half<AMN>(a, &p.m.a, bar, block * kBK, t.row + rank * kHalfM, t.at);
    const int col = t.col + rank * (t.n / 2);
    load_half<BMN>(b, &p.m.b[BMN ? 0 : t.n / 32 - 1], bar, block * kBK, col, t.at);
  }
  static constexpr int kWords = kChunk / 2;
  struct Source {  // a chunk of a row: of X's halves, or of A; of the weights
    uint32_t hi[KIND == kGram ? 1 : kWords], lo[kSym ? 1 : kWords];
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
    const bool keep = row < p.m.rows;
    const int cols = min(t.n, p.m.cols - t.col);
    // rows of the workspace are multiples of kChunk apart: whole chunks are read and written, what lies past
    // the columns is not read as an operand
    const int64_t matrix = (int64_t)t.at * p.m.rows * g.ld;
    const int64_t at = matrix + (int64_t)(keep ? row : 0) * g.ld + t.col;
    const int64_t out_at = ((int64_t)t.at * p.m.rows + (keep ? row : 0)) * p.m.cols + t.col;
    float lr = 1.0f;
    if (KIND == kWeights && g.lr) lr = __ldg(g.lr);
    const float w_keep = 1.0f - lr * g.keep, w_scale = lr * g.scale;
    const bool f32 = KIND == kWeights && g.w_dtype == MOE_DTYPE_F32;
    auto load = [&](int c, Source& s) {
      if constexpr (KIND != kGram) load32(g.src + at + c, s.hi);
      if constexpr (!kSym) load32(g.lo + at + c, s.lo);
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
    auto use = [&](int c, const Source& s, float* v) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float2 x = make_float2(v[2 * i] * g.beta, v[2 * i + 1] * g.beta);
        if constexpr (KIND != kGram) {
          const float2 h = halves(s.hi[i]);
          x = make_float2(fmaf(g.alpha, h.x, x.x), fmaf(g.alpha, h.y, x.y));
        }
        if constexpr (!kSym) {
          const float2 l = halves(s.lo[i]);
          x = make_float2(fmaf(g.alpha, l.x, x.x), fmaf(g.alpha, l.y, x.y));
        }
        v[2 * i] = x.x;
        v[2 * i + 1] = x.y;
      }
      if constexpr (kSym || KIND == kNext) {
        uint32_t hi[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) hi[i] = pack_half(v[2 * i], v[2 * i + 1]);
        if (keep) store32((kSym ? g.sym : g.next) + at + c, hi);
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
            if ((row & ~1) < p.m.rows && c + 2 * j + odd < cols)
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
    by_chunks<Source>(cols, group, tbase, load, use, wait, release);
  }
};

// ------------------------------------------------------------------- host

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Blocks of a matrix in the passes over G: no more than 8 on an SM in all, 8 elements a thread or more.
int norm_blocks(const OrthoArgs& g) {
  const int64_t most = (8 * (int64_t)kNumSmsGB300 + g.B - 1) / g.B;
  const int64_t want = ((int64_t)g.N * g.K + 8 * kNormThreads - 1) / (8 * kNormThreads);
  return (int)(want < most ? want : most);
}

struct Layout {
  int m, ldx, ldm;
  size_t part, x0, x1, lo, gram, poly, total;  // offsets
};

Layout layout(const OrthoArgs& g) {
  Layout l;
  l.m = g.N < g.K ? g.N : g.K;
  l.ldx = (int)up(g.K, kChunk);
  l.ldm = (int)up(l.m, kChunk);
  const size_t x = up((int64_t)g.B * g.N * l.ldx * 2, 256), sym = up((int64_t)g.B * l.m * l.ldm * 2, 256);
  l.part = 0;
  l.x0 = up((int64_t)g.B * norm_blocks(g) * (int64_t)sizeof(float2), 256);
  l.x1 = l.x0 + x;
  l.lo = l.x1 + x;
  l.gram = l.lo + x;
  l.poly = l.gram + sym;
  l.total = l.poly + sym;
  return l;
}

// The result [rows, cols] of count matrices; reduction over k.
bool make_mats(Mats* m, const OrthoArgs& g, int rows, int cols, int k, bool sym) {
  m->count = g.B;
  m->rows = rows;
  m->cols = cols;
  m->ct = (cols + kMaxN - 1) / kMaxN;
  m->rt = (rows + kTileM - 1) / kTileM;
  m->k = k;
  m->per = sym ? m->rt * (m->rt + 1) / 2 : m->rt * m->ct;
  return (int64_t)m->per * g.B <= INT32_MAX / 2;
}

// The operand maps: matrices [rows, cols] with rows ld elements apart.
bool map_a(Mats* m, bool mn, const void* x, int count, int rows, int cols, int ld) {
  return make_map_3d(&m->a, x, true, count, rows, cols, ld, mn ? kBK : kHalfM);
}
bool map_b(Mats* m, bool mn, const void* x, int count, int rows, int cols, int ld) {
  for (int h = 0; h < kHeights; ++h)
    if (!make_map_3d(&m->b[h], x, true, count, rows, cols, ld, mn ? kBK : box_rows(h))) return false;
  return true;
}

template <class P>
cudaError_t launch(const typename P::Params& p, cudaStream_t s) {
  return launch_pairs<P>(p, (int64_t)p.m.count * p.m.per, 0, true, s);
}

template <bool TALL, Product KIND>
cudaError_t multiply(const OrthoArgs& g, const Layout& l, const Result& r, const __half* poly, cudaStream_t s) {
  // X [N, K]: P X (wide: P's rows, X's columns) or X P (tall: X's rows, P's rows, as P is symmetric)
  using P = Ns<false, !TALL, KIND>;
  typename P::Params p{};
  if (!make_mats(&p.m, g, g.N, g.K, l.m, false)) return cudaErrorNotSupported;
  if (TALL ? !(map_a(&p.m, false, r.src, g.B, g.N, g.K, l.ldx) && map_b(&p.m, false, poly, g.B, l.m, l.m, l.ldm))
           : !(map_a(&p.m, false, poly, g.B, l.m, l.m, l.ldm) && map_b(&p.m, true, r.src, g.B, g.N, g.K, l.ldx)))
    return cudaErrorInvalidValue;
  p.r = r;
  p.err = g.err;
  return launch<P>(p, s);
}

template <bool TALL>
cudaError_t iterate(const OrthoArgs& g, const Layout& l, char* ws, cudaStream_t s) {
  __half* x[2] = {reinterpret_cast<__half*>(ws + l.x0), reinterpret_cast<__half*>(ws + l.x1)};
  __half* gram = reinterpret_cast<__half*>(ws + l.gram);
  __half* poly = reinterpret_cast<__half*>(ws + l.poly);
  using Gram = Ns<TALL, TALL, kGram>;
  using Poly = Ns<false, false, kPolynomial>;
  for (int step = 0; step < g.steps; ++step) {
    const __half* cur = x[step & 1];
    typename Gram::Params a{};
    if (!make_mats(&a.m, g, l.m, l.m, TALL ? g.N : g.K, true)) return cudaErrorNotSupported;
    if (!map_a(&a.m, TALL, cur, g.B, g.N, g.K, l.ldx) || !map_b(&a.m, TALL, cur, g.B, g.N, g.K, l.ldx))
      return cudaErrorInvalidValue;
    a.r.sym = gram;
    a.r.ld = l.ldm;
    a.r.beta = kUnscale;
    a.err = g.err;
    cudaError_t e = launch<Gram>(a, s);
    if (e != cudaSuccess) return e;

    typename Poly::Params q{};
    if (!make_mats(&q.m, g, l.m, l.m, l.m, true)) return cudaErrorNotSupported;
    if (!map_a(&q.m, false, gram, g.B, l.m, l.m, l.ldm) || !map_b(&q.m, false, gram, g.B, l.m, l.m, l.ldm))
      return cudaErrorInvalidValue;
    q.r.sym = poly;
    q.r.src = gram;
    q.r.ld = l.ldm;
    q.r.alpha = g.coef[1];
    q.r.beta = g.coef[2] * kUnscale;
    q.err = g.err;
    e = launch<Poly>(q, s);
    if (e != cudaSuccess) return e;

    Result r{};
    r.src = cur;
    r.next = x[(step + 1) & 1];
    r.lo = reinterpret_cast<__half*>(ws + l.lo);
    r.ld = l.ldx;
    r.alpha = g.coef[0];
    r.beta = kUnscale;
    r.out = g.out;
    r.scale = kUnscale * g.scale;
    r.keep = g.decay;
    r.lr = g.lr;
    r.w_dtype = g.w_dtype;
    r.whole = g.K % kChunk == 0 && (reinterpret_cast<uintptr_t>(g.out) & 31) == 0;
    if (step + 1 < g.steps) e = multiply<TALL, kNext>(g, l, r, poly, s);
    else if (g.update) e = multiply<TALL, kWeights>(g, l, r, poly, s);
    else e = multiply<TALL, kOut>(g, l, r, poly, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
  norm_kernel<T, V, MOMENTUM><<<grid, kNormThreads, 0, s>>>(in, part);
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
  OrthoArgs g{};
  g.B = B;
  g.N = N;
  g.K = K;
  return layout(g).total;
}

cudaError_t launch_orthogonalize(const OrthoArgs& g, cudaStream_t s) {
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
  return g.N > g.K ? iterate<true>(g, l, ws, s) : iterate<false>(g, l, ws, s);
}

}  // namespace moe
