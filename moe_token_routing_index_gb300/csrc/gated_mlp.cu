// The experts' gated feed-forward block in training (include/moe_train.h) on the pair GEMM.
//
//   forward   y = x w13_e^T with z = act(y0) * y1 in the epilogue, then out = z w2_e^T
//   backward  dz = dout w2_e with the gradient of act * mul in the epilogue (dy, z), then dx = dy w13_e
//
// The weights are the A operand (256 of a product's output columns a tile) and the routed rows
// the B operand (n rows, a multiple of 32): an expert of c rows is cut into ceil(c / 256) equal
// parts, so that a product costs what its rows, rounded up to 32, cost.  The backward reads the
// weights as they lie, as MN-major operands, and needs no transposed copies.
//
// Forward, each lane of tensor memory is a column of y.  The TMA box takes 16 rows of w1, the 16
// rows of w3 that belong to them, the next 16 of w1 and so on (w13 seen as [E][H/16][2][16][D]),
// so lanes j and j + 16 of a warp hold y0 and y1 of one column, and one shuffle for two
// accumulators brings the pairs together.
//
// Bound by reading the weights below about 280 rows an expert, by the products above.  8192 rows of 16
// experts, D = 5120, H = 8192: 755 us gate and up (1820 TFLOP/s), 410 us down (1680), 416 us the gradient
// of dz (1650), 773 us dx (1780).  32768 rows of 128 experts, D = 7168, H = 2048: 1231 to 1241, 685 to 699, 713
// to 720 and 1259 to 1272 us.  128 rows of 16 experts, D = 5120, H = 8192, forward: 603 us, 6.7 TB/s.  These are
// short runs; in a loop of calls the GPU is at its power limit, and that gradient takes 1547 to 1638 us in all (1260
// to 1330 TFLOP/s), the uneven forward 2600 to 2670 (2360 to 2440 in short runs).  The gradient's epilogue has y two chunks ahead in registers, from clamped addresses: loaded at their place
// behind a condition, its values came one after another (the first form, 1273 us for that gradient; 481
// with addresses clamped and wider accesses, and 416 with all later steps).
#include "common.cuh"
#include "launch.h"
#include "pair_gemm.cuh"
#include "train_launch.h"

namespace moe {
namespace {

using namespace pg;

struct Rows {           // the routed rows and how the tiles walk them
  CUtensorMap w;
  CUtensorMap x[kHeights];
  const int32_t* counts;
  int E, a_max;
  int mt;               // tiles along a product's output columns
  int band;             // row tiles of a band of the tile order
  int k;                // the reduction's length
};

struct RowTile {
  int n, k;
  int m, expert, row0, rows;  // tile along the columns; rows: those of the tile that are the expert's
};

// tables: the experts' first row tiles [E + 1] and rows [E + 1].  Counts as in the grouped GEMMs: negative
// ones are empty, a sum past a_max is cut, both flagged.
__device__ __forceinline__ int setup_rows(const Rows& p, int* tables, unsigned int* err) {
  int* tile_start = tables;
  int* row_off = tables + p.E + 1;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    int64_t run = 0;
    int tiles = 0;
    bool bad = false;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      int c = e < p.E ? p.counts[e] : 0;
      if (c < 0) {
        c = 0;
        bad = true;
      }
      int64_t incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int r0 = (int)min(run + incl - c, (int64_t)p.a_max), r1 = (int)min(run + incl, (int64_t)p.a_max);
      const int mine = (r1 - r0 + kMaxN - 1) / kMaxN;
      int n = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += v;
      }
      if (e < p.E) {
        tile_start[e] = tiles + n - mine;
        row_off[e] = r0;
      }
      tiles += __shfl_sync(0xffffffffu, n, 31);
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (run > p.a_max) bad = true;
    if (lane == 0) {
      tile_start[p.E] = tiles;
      row_off[p.E] = (int)min(run, (int64_t)p.a_max);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) flag_error(err, MOE_DEVERR_BAD_COUNT);
  }
  __syncthreads();
  return tile_start[p.E] * p.mt;
}

// Tile i: the experts in order; within one, bands of row tiles, in a band the row tiles innermost, so that
// pairs running together share the weights' tile and the band's rows.  (Experts by their rows, and each
// pair, or half of the pairs, taking tiles from either end of that order, so that tiles bound by the weights
// run beside those bound by the products: one run each, 32768 rows of 128 experts by Zipf's law, forward, 2415
// and 2428 us in this order, 2430 to 2550 in those; 128 experts of 344 rows, gradient, 1232 and 1287 in this
// order, 1236 and 1248 by rows alone, 1300 to 1630 from either end.)
__device__ __forceinline__ RowTile locate_rows(const Rows& p, const int* tables, int i) {
  const int* tile_start = tables;
  const int* row_off = tables + p.E + 1;
  const int g = i / p.mt;
  int lo = 0, hi = p.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= g) lo = mid;
    else hi = mid - 1;
  }
  RowTile t;
  t.expert = lo;
  const int nt = tile_start[lo + 1] - tile_start[lo], c = row_off[lo + 1] - row_off[lo];
  const int local = i - tile_start[lo] * p.mt;
  const int b = local / (p.band * p.mt);
  const int in_band = min(p.band, nt - b * p.band), lb = local - b * p.band * p.mt;
  t.m = lb / in_band;
  const int rt = b * p.band + lb - t.m * in_band;
  if (b & 1) t.m = p.mt - 1 - t.m;  // the band before ended on these weights
  // equal parts of a multiple of 32 rows; c > 256 (nt - 1), so the last one has rows too
  const int part = ((c + nt - 1) / nt + 31) / 32 * 32;
  t.row0 = row_off[lo] + rt * part;
  t.rows = min(part, c - rt * part);
  t.n = (t.rows + 31) / 32 * 32;
  t.k = p.k;
  return t;
}

__device__ __forceinline__ void narrow_rows(RowTile* t, int part, int parts) {
  const int n = ((t->n + parts - 1) / parts + 31) / 32 * 32, from = part * n;
  t->row0 += from;
  t->rows = min(n, t->rows - from);
  t->n = max(0, min(n, t->n - from));
}

__device__ __forceinline__ uint32_t row_stage_bytes(const RowTile& t) {
  return 2u * (uint32_t)(kOperandBytes + t.n / 2 * 128 * (kBK / 64));
}

__device__ __forceinline__ void load_rows(const Rows& p, const RowTile& t, int rank, int block, uint32_t dst,
                                          uint32_t bar) {
  const int row = t.row0 + rank * (t.n / 2), k = block * kBK;
  const CUtensorMap* map = &p.x[t.n / 32 - 1];
#pragma unroll
  for (int h = 0; h < kBK / 64; ++h) load_2d(dst + h * 128 * 128, map, bar, k + 64 * h, row);
}

// ------------------------------------------------------------- activations

// act(v) = v * sigmoid(u(v)): u = v (SiLU), or sqrt(8 / pi) (v + 0.044715 v^3) (GELU, tanh form).
__device__ __forceinline__ float rcp(float v) {  // to 1 ulp; 0 for infinity
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

template <int ACT>
__device__ __forceinline__ float gate_of(float v) {
  const float u = ACT == MOE_ACT_SILU ? v : 1.5957691216f * v * fmaf(0.044715f * v, v, 1.0f);
  return rcp(1.0f + __expf(-u));
}

template <int ACT>
__device__ __forceinline__ float act(float v) {
  return v * gate_of<ACT>(v);
}

// act and its derivative p + v p (1 - p) u'(v).
template <int ACT>
__device__ __forceinline__ void act_slope(float v, float* f, float* slope) {
  const float p = gate_of<ACT>(v);
  *f = v * p;
  const float q = *f * (1.0f - p);
  if (ACT == MOE_ACT_SILU) {
    *slope = p + q;
  } else {
    const float du = fmaf(0.2140644488f * v, v, 1.5957691216f);
    *slope = q == 0.0f ? p : fmaf(q, du, p);  // (du may be infinite where q has vanished)
  }
}

// ------------------------------------------------------- the four products

// z = act(y0) y1 and y, from w13.
template <int ACT>
struct GatedForward {
  static constexpr bool kAMN = false, kBMN = false, kF16 = false;
  struct Params {
    Rows rows;
    __nv_bfloat16* y;  // nullable
    __nv_bfloat16* z;
    int H;
    unsigned int* err;
  };
  using Tile = RowTile;
  static __device__ int setup(const Params& p, int* tables) { return setup_rows(p.rows, tables, p.err); }
  static __device__ void narrow(Tile* t, int part, int parts) { narrow_rows(t, part, parts); }
  static __device__ Tile tile(const Params& p, const int* tables, int i) { return locate_rows(p.rows, tables, i); }
  static __device__ uint32_t stage_bytes(const Params&, const Tile& t) { return row_stage_bytes(t); }
  static __device__ void load(const Params& p, const Tile& t, int rank, int block, uint32_t a, uint32_t b,
                              uint32_t bar) {
#pragma unroll
    for (int h = 0; h < kBK / 64; ++h)
      load_5d(a + h * 128 * 128, &p.rows.w, bar, block * kBK + 64 * h, 0, 0, t.m * 8 + rank * 4, t.expert);
    load_rows(p.rows, t, rank, block, b, bar);
  }
  template <class Wait, class Release>
  static __device__ void epilogue(const Params& p, const Tile& t, int rank, int sub, int group, int lane, uint32_t tbase,
                                  Wait wait, Release release) {
    const int f = t.m * 128 + rank * 64 + sub * 16 + (lane & 15);
    const bool first = lane < 16, keep = f < p.H;  // (H is a multiple of 16: all of a half-warp)
    const int64_t H = p.H;
    __nv_bfloat16* z = p.z + (int64_t)t.row0 * H + f;
    __nv_bfloat16* y = p.y + (int64_t)t.row0 * 2 * H + f;
    auto use = [&](int c, const NoSource&, const float* v) {
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        // the first half-warp takes row 2j, the second row 2j + 1
        const float other = __shfl_xor_sync(0xffffffffu, first ? v[2 * j + 1] : v[2 * j], 16);
        const float y0 = first ? v[2 * j] : other, y1 = first ? other : v[2 * j + 1];
        const int r = c + 2 * j + (first ? 0 : 1);
        const float zr = act<ACT>(y0) * y1;
        if (keep && r < t.rows) {
          z[r * H] = __float2bfloat16_rn(zr);
          if (p.y) {
            y[r * 2 * H] = __float2bfloat16_rn(y0);
            y[r * 2 * H + H] = __float2bfloat16_rn(y1);
          }
        }
      }
    };
    by_chunks<NoSource>(t.rows, group, tbase, [](int, NoSource&) {}, use, wait, release);
  }
};

struct Kept {  // y0 and y1 of a lane's share of a chunk: two bf16, or two codes and their exponent byte
  uint32_t y0[kChunk / 2], y1[kChunk / 2];
};

// dy and z from dz = dout w2 and the kept y (bf16, or a checkpoint's codes and exponents).
template <int ACT, bool CODES>
struct GatedGrad {
  static constexpr bool kAMN = true, kBMN = false, kF16 = false;
  struct Params {
    Rows rows;
    const void* y;
    const uint8_t* exponents;
    __nv_bfloat16* dy;
    __nv_bfloat16* z;  // nullable
    int H;
    unsigned int* err;
  };
  using Tile = RowTile;
  static __device__ int setup(const Params& p, int* tables) { return setup_rows(p.rows, tables, p.err); }
  static __device__ void narrow(Tile* t, int part, int parts) { narrow_rows(t, part, parts); }
  static __device__ Tile tile(const Params& p, const int* tables, int i) { return locate_rows(p.rows, tables, i); }
  static __device__ uint32_t stage_bytes(const Params&, const Tile& t) { return row_stage_bytes(t); }
  static __device__ void load(const Params& p, const Tile& t, int rank, int block, uint32_t a, uint32_t b,
                              uint32_t bar) {
    load_half<true>(a, &p.rows.w, bar, block * kBK, t.m * kTileM + rank * kHalfM, t.expert);
    load_rows(p.rows, t, rank, block, b, bar);
  }
  template <class Wait, class Release>
  static __device__ void epilogue(const Params& p, const Tile& t, int rank, int sub, int group, int lane, uint32_t tbase,
                                  Wait wait, Release release) {
    // two neighbouring columns of y, of every second row (H is a multiple of 16: both or none)
    const int f = t.m * kTileM + rank * kHalfM + sub * 32 + (lane & 30);
    const bool odd = lane & 1, keep = f < p.H;
    const int fc = keep ? f : 0;  // lanes without columns read what others read
    const int64_t H = p.H;
    const int nb = (p.H + 127) / 128;
    auto load = [&](int c, Kept& s) {
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        const int64_t r = t.row0 + min(c + 2 * j + odd, t.rows - 1);
        if (CODES) {
          const uint8_t* e = p.exponents + r * 2 * nb + fc / 128;
          const uint8_t* q = static_cast<const uint8_t*>(p.y) + r * 2 * H + fc;
          s.y0[j] = *reinterpret_cast<const uint16_t*>(q) | (uint32_t)__ldg(e) << 16;
          s.y1[j] = *reinterpret_cast<const uint16_t*>(q + H) | (uint32_t)__ldg(e + nb) << 16;
        } else {
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.y) + r * 2 * H + fc;
          s.y0[j] = __ldg(reinterpret_cast<const uint32_t*>(q));
          s.y1[j] = __ldg(reinterpret_cast<const uint32_t*>(q + H));
        }
      }
    };
    auto values = [](uint32_t v) {
      if (!CODES) return bf16x2_bits_to_f32(v);
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xffffu), __NV_E4M3);
      const float2 q = __half22float2(__half2(h));
      const float s = __uint_as_float((v >> 16) << 23);
      return make_float2(q.x * s, q.y * s);
    };
    auto pack = [](float x, float y) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      return *reinterpret_cast<const uint32_t*>(&h);
    };
    auto use = [&](int c, const Kept& s, const float* v) {
      const int64_t r = t.row0 + c + odd;
      __nv_bfloat16* dy = p.dy + r * 2 * H + f;
      __nv_bfloat16* z = p.z + r * H + f;
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        const float2 dz = deal(v, j, odd), y0 = values(s.y0[j]), y1 = values(s.y1[j]);
        float2 g, slope;
        act_slope<ACT>(y0.x, &g.x, &slope.x);
        act_slope<ACT>(y0.y, &g.y, &slope.y);
        if (keep && c + 2 * j + odd < t.rows) {
          *reinterpret_cast<uint32_t*>(dy) = pack(dz.x * y1.x * slope.x, dz.y * y1.y * slope.y);
          *reinterpret_cast<uint32_t*>(dy + H) = pack(dz.x * g.x, dz.y * g.y);
          if (p.z) *reinterpret_cast<uint32_t*>(z) = pack(g.x * y1.x, g.y * y1.y);
        }
        dy += 4 * H;
        z += 2 * H;
      }
    };
    by_chunks<Kept>(t.rows, group, tbase, load, use, wait, release);
  }
};

// out[r, f] = sum_k x[r, k] w_e[f, k], or w_e[k, f] (WMN).
template <bool WMN>
struct Plain {
  static constexpr bool kAMN = WMN, kBMN = false, kF16 = false;
  struct Params {
    Rows rows;
    __nv_bfloat16* out;
    int F;
    unsigned int* err;
  };
  using Tile = RowTile;
  static __device__ int setup(const Params& p, int* tables) { return setup_rows(p.rows, tables, p.err); }
  static __device__ void narrow(Tile* t, int part, int parts) { narrow_rows(t, part, parts); }
  static __device__ Tile tile(const Params& p, const int* tables, int i) { return locate_rows(p.rows, tables, i); }
  static __device__ uint32_t stage_bytes(const Params&, const Tile& t) { return row_stage_bytes(t); }
  static __device__ void load(const Params& p, const Tile& t, int rank, int block, uint32_t a, uint32_t b,
                              uint32_t bar) {
    load_half<WMN>(a, &p.rows.w, bar, block * kBK, t.m * kTileM + rank * kHalfM, t.expert);
    load_rows(p.rows, t, rank, block, b, bar);
  }
  template <class Wait, class Release>
  static __device__ void epilogue(const Params& p, const Tile& t, int rank, int sub, int group, int lane, uint32_t tbase,
                                  Wait wait, Release release) {
    const int f = t.m * kTileM + rank * kHalfM + sub * 32 + (lane & 30);
    const bool odd = lane & 1, keep = f < p.F;  // (F is a multiple of 16)
    auto use = [&](int c, const NoSource&, const float* v) {
      __nv_bfloat16* out = p.out + (int64_t)(t.row0 + c + odd) * p.F + f;
#pragma unroll
      for (int j = 0; j < kChunk / 2; ++j) {
        const float2 w = deal(v, j, odd);
        if (keep && c + 2 * j + odd < t.rows)
          *reinterpret_cast<__nv_bfloat162*>(out + (int64_t)(2 * j) * p.F) = __floats2bfloat162_rn(w.x, w.y);
      }
    };
    by_chunks<NoSource>(t.rows, group, tbase, [](int, NoSource&) {}, use, wait, release);
  }
};

// ------------------------------------------------------------------- host

// Bytes of routed rows that a band of the tile order may span.
constexpr int64_t kBandBytes = 30ll << 20;

// The routed rows x [a_max, K] and `cols` output columns, tiles of tile_cols.
bool make_rows(Rows* r, const GatedArgs& g, const void* x, int K, int cols, int tile_cols) {
  r->counts = g.counts;
  r->E = g.E;
  r->a_max = g.a_max;
  r->mt = (cols + tile_cols - 1) / tile_cols;
  r->k = K;
  const int64_t b = kBandBytes / ((int64_t)kMaxN * K * 2);
  r->band = (int)(b < 1 ? 1 : b > 1024 ? 1024 : b);
  for (int h = 0; h < kHeights; ++h) {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)g.a_max};
    const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows(h)};
    if (!make_map(&r->x[h], x, false, 2, dims, strides, box)) return false;
  }
  return true;
}

template <class P>
cudaError_t launch(const typename P::Params& p, bool pdl, cudaStream_t s) {
  const Rows& r = p.rows;
  const int64_t tiles = ((int64_t)r.a_max / kMaxN + r.E) * r.mt;  // at most
  if (tiles > INT32_MAX / 2) return cudaErrorNotSupported;
  return launch_pairs<P>(p, tiles, r.k, 2 * (r.E + 1) * (int)sizeof(int), pdl, s);
}

template <bool WMN>
cudaError_t launch_plain(const GatedArgs& g, const void* x, int K, const void* w, int F, void* out, cudaStream_t s) {
  typename Plain<WMN>::Params p{};
  if (!make_rows(&p.rows, g, x, K, F, kTileM)) return cudaErrorInvalidValue;
  if (!(WMN ? make_map_3d(&p.rows.w, w, false, g.E, K, F, F, kBK) : make_map_3d(&p.rows.w, w, false, g.E, F, K, K, kHalfM)))
    return cudaErrorInvalidValue;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.F = F;
  p.err = g.err;
  return launch<Plain<WMN>>(p, true, s);
}

template <int ACT>
cudaError_t forward(const GatedArgs& g, cudaStream_t s) {
  typename GatedForward<ACT>::Params p{};
  if (!make_rows(&p.rows, g, g.x, g.D, g.H, 128)) return cudaErrorInvalidValue;
  const cuuint64_t row = (cuuint64_t)g.D * 2;
  const cuuint64_t dims[5] = {(cuuint64_t)g.D, 16, 2, (cuuint64_t)g.H / 16, (cuuint64_t)g.E};
  const cuuint64_t strides[4] = {row, row * g.H, row * 16, row * 2 * g.H};
  const cuuint32_t box[5] = {64, 16, 2, 4, 1};
  if (!make_map(&p.rows.w, g.w13, false, 5, dims, strides, box)) return cudaErrorInvalidValue;
  p.y = static_cast<__nv_bfloat16*>(g.y);
  p.z = static_cast<__nv_bfloat16*>(g.z);
  p.H = g.H;
  p.err = g.err;
  return launch<GatedForward<ACT>>(p, false, s);
}

template <int ACT, bool CODES>
cudaError_t gradient(const GatedArgs& g, cudaStream_t s) {
  typename GatedGrad<ACT, CODES>::Params p{};
  if (!make_rows(&p.rows, g, g.x, g.D, g.H, kTileM) || !make_map_3d(&p.rows.w, g.w2, false, g.E, g.D, g.H, g.H, kBK))
    return cudaErrorInvalidValue;
  p.y = g.y;
  p.exponents = g.exponents;
  p.dy = static_cast<__nv_bfloat16*>(g.dy);
  p.z = static_cast<__nv_bfloat16*>(g.z);
  p.H = g.H;
  p.err = g.err;
  return launch<GatedGrad<ACT, CODES>>(p, false, s);
}

}  // namespace

cudaError_t launch_gated_mlp(const GatedArgs& g, cudaStream_t s) {
  cudaError_t e = g.activation == MOE_ACT_SILU ? forward<MOE_ACT_SILU>(g, s) : forward<MOE_ACT_GELU>(g, s);
  if (e != cudaSuccess) return e;
  return launch_plain<false>(g, g.z, g.H, g.w2, g.D, g.out, s);
}

cudaError_t launch_gated_mlp_backward(const GatedArgs& g, cudaStream_t s) {
  cudaError_t e;
  if (g.activation == MOE_ACT_SILU)
    e = g.exponents ? gradient<MOE_ACT_SILU, true>(g, s) : gradient<MOE_ACT_SILU, false>(g, s);
  else
    e = g.exponents ? gradient<MOE_ACT_GELU, true>(g, s) : gradient<MOE_ACT_GELU, false>(g, s);
  if (e != cudaSuccess) return e;
  return launch_plain<true>(g, g.dy, 2 * g.H, g.w13, g.D, g.out, s);
}

}  // namespace moe
