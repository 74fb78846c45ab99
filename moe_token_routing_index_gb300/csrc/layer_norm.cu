// Layer norm of the token rows and its gradient (include/moe_train.h).  Both are bound
// by memory: a row is read from it once and kept on chip between its reductions.
//
// A group of R threads (whole warps) owns a row, N values a thread, in pieces of VEC
// consecutive columns: 8 where columns, strides and addresses allow 16-byte accesses,
// else 1.  Groups of a block are independent (named barriers), so narrow rows fill a block
// too, and the grids are persistent, a block for each SM.
//
// Forward: the mean, then the variance from the centred values, two group reductions.
// Backward: one reduction of two sums a row; each thread keeps its columns' sums of dgamma
// and dbeta over the rows of its group.  The block's groups are added in order through
// shared memory, and a second kernel adds the blocks' partial sums in order.
//
// Rows wider than a warp's go through a ring of rows in shared memory for each group,
// filled by bulk copies several rows ahead (Ring), with the weights in fp32 beside it;
// narrower rows, few rows, very wide fp32 rows and rows whose tensors are aligned apart are
// loaded straight into registers.  Where that is 16 or 32 columns a thread by single accesses, or
// backward 32 fp32 columns, the registers spill (0.2 to 1.3 KB a thread): 5000 rows of 5120 in
// bf16 that start 2 bytes past 16 take 121 us and 146 backward, 2000 of 16384 in fp32 75 and 171.
//
// Loaded one row ahead into registers, 11000 rows of 4096 took 49 us and the gradient of 8192 rows of 5120 took 106 us (bf16): the values held
// ahead left too few warps to hide the reductions; through the ring 35 and 54 us, 5.2 and
// 4.7 TB/s.  Arithmetic is in pairs (fma.rn.f32x2), and 32 values a thread spread a row's
// fixed cost over enough elements.
//
// Dense rows of a width that is no multiple of 16 bytes start at varying offsets inside 16
// bytes (SHIFT).  They repeat every 8 rows at most, and a group's rows are a multiple of 8
// apart, so each group has its own offset throughout, and cuts its rows into the 8-column
// pieces that are aligned in memory: only a row's first and last piece are not whole.
// 5000 rows of 4097 in bf16 take 42 us and 74 backward; by single columns, 112 and 129.
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "train_launch.h"

namespace moe {
namespace {

constexpr int kMaxGroups = 15;  // named barriers 1 .. 15

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32(float v) {
  return v;
}
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// VEC consecutive values as they lie in memory.
template <typename T, int VEC>
struct Piece;
template <typename T>
struct Piece<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = __ldg(p); }
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
  __device__ __forceinline__ static void store(T* p, const float* f) { put(p, f[0]); }
};
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float* f) {
    *reinterpret_cast<uint4*>(p) = f32_to_bf16x8(f);
  }
};
template <>
struct Piece<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ float get(int i) const {
    const float4& h = i < 4 ? a : b;
    const int j = i & 3;
    return j == 0 ? h.x : j == 1 ? h.y : j == 2 ? h.z : h.w;
  }
  __device__ __forceinline__ static void store(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Two fp32 values in a register pair.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 both(float v) { return pack(v, v); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f2 v) {
  const float2 u = unpack(v);
  return u.x + u.y;
}

// A thread's N values of a row of D columns, as they lie in memory: value i is column
// ((i / VEC) * R + its number in the group) * VEC + i % VEC.  Columns past D are zeros.
template <typename T, int VEC, int N>
struct Row {
  static constexpr int C = N / VEC;
  Piece<T, VEC> p[C];
  __device__ __forceinline__ void load(const T* row, int R, int gt, int D) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int d = (c * R + gt) * VEC;
      if (d < D) p[c].load(row + d);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < C; ++c) p[c] = Piece<T, VEC>{};
  }
  __device__ __forceinline__ f2 pair(int j) const {
    return pack(p[2 * j / VEC].get(2 * j % VEC), p[(2 * j + 1) / VEC].get((2 * j + 1) % VEC));
  }
  // Stores a result a(j) for each pair j, piece by piece.
  template <typename F>
  __device__ __forceinline__ static void store(T* row, int R, int gt, int D, F a) {
    constexpr int P = VEC == 1 ? 2 : VEC;  // values computed together
#pragma unroll
    for (int c = 0; c < N / P; ++c) {
      float o[P];
#pragma unroll
      for (int j = 0; j < P / 2; ++j) {
        const float2 v = unpack(a(c * (P / 2) + j));
        o[2 * j] = v.x;
        o[2 * j + 1] = v.y;
      }
#pragma unroll
      for (int k = 0; k < P / VEC; ++k) {
        const int d = ((c * (P / VEC) + k) * R + gt) * VEC;
        if (d < D) Piece<T, VEC>::store(row + d, o + k * VEC);
      }
    }
  }
};

// A group's ring of rows in shared memory: `mats` rows (of x, and of dy) a stage, filled by
// the group's first thread and awaited by all of it.  bars: one mbarrier a stage.
struct Ring {
  uint32_t base, bars;
  int slot, mats, stages;    // slot: bytes of a row's place
  int stage = 0, next = 0;   // being read; to be filled
  uint32_t parity = 0;       // of the stage being read

  __device__ __forceinline__ uint32_t at(int st, int mat) const {
    return base + (uint32_t)((st * mats + mat) * slot);
  }
  // n bytes of each row, from 16-byte boundaries.
  __device__ __forceinline__ void fill(const void* x, const void* dy, int n) {
    const uint32_t bar = bars + 8 * next;
    tc::mbar_arrive_expect_tx(bar, (uint32_t)(n * mats));
    copy(at(next, 0), x, n, bar);
    if (mats == 2) copy(at(next, 1), dy, n, bar);
    if (++next == stages) next = 0;
  }
  __device__ __forceinline__ void copy(uint32_t dst, const void* src, int n, uint32_t bar) const {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
        "r"(n), "r"(bar)
        : "memory");
  }
  __device__ __forceinline__ bool wait() const { return tc::mbar_wait(bars + 8 * stage, parity, nullptr); }
  __device__ __forceinline__ void advance() {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

// How a group's rows lie: sh elements past a 16-byte boundary.  A copy starts at that boundary
// (before a row's start only where other rows precede it: row 0 has no offset) and ends at
// the one after the row, but for the last row of the tensors at the one before.
template <typename T, bool SHIFT>
struct Placing {
  int D, last, sh;
  __device__ __forceinline__ Placing(int D_, int T_, int64_t t0)
      : D(D_), last(T_ - 1), sh(SHIFT ? (int)(t0 * D_ * (int)sizeof(T) & 15) / (int)sizeof(T) : 0) {}
  __device__ __forceinline__ int bytes(int64_t t) const {
    const int n = (D + sh) * (int)sizeof(T);
    return !SHIFT || t == last ? n & ~15 : (n + 15) & ~15;
  }
  // First column of piece `piece` (may be negative), whether it has any column of the row, all 8.
  __device__ __forceinline__ int column(int piece) const { return piece * 8 - sh; }
  __device__ __forceinline__ bool any(int d) const { return d < D; }  // (sh < 8)
  __device__ __forceinline__ bool whole(int d) const { return !SHIFT || (d >= 0 && d + 8 <= D); }
};
template <typename T>
__host__ __device__ __forceinline__ int slot_bytes(int D, bool shift) {
  return (shift ? (D + 14) / 8 * 8 : D) * (int)sizeof(T);  // whole pieces
}

constexpr int kMaxStages = 6;

// A piece of a row in shared memory.
template <typename T>
__device__ __forceinline__ Piece<T, 8> shared_piece(uint32_t row, int d);
template <>
__device__ __forceinline__ Piece<__nv_bfloat16, 8> shared_piece(uint32_t row, int d) {
  Piece<__nv_bfloat16, 8> p;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(p.v.x), "=r"(p.v.y), "=r"(p.v.z), "=r"(p.v.w)
               : "r"(row + 2 * d));
  return p;
}
template <>
__device__ __forceinline__ Piece<float, 8> shared_piece(uint32_t row, int d) {
  Piece<float, 8> p;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(p.a.x), "=f"(p.a.y), "=f"(p.a.z), "=f"(p.a.w)
               : "r"(row + 4 * d));
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(p.b.x), "=f"(p.b.y), "=f"(p.b.z), "=f"(p.b.w)
               : "r"(row + 4 * d + 16));
  return p;
}

// A group's barrier at which it agrees on `ok`.
__device__ __forceinline__ bool group_agrees(bool ok, int group, int R) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "r"(group + 1), "r"(R)
      : "memory");
  return all != 0;
}

// The weights of a row in shared memory as fp32.  Whole pieces: the first four of each 8
// columns, then the last four (16-byte accesses of neighbouring threads are then contiguous).
// SHIFT: one by one with 8 zeros on either side and a gap every 32 (neighbouring threads'
// pieces, 8 apart, then lie in different banks).
template <bool SHIFT>
__host__ __device__ __forceinline__ int weight_floats(int D) {
  return SHIFT ? ((D + 16) + (D + 16) / 32 + 4) / 4 * 4 : D;
}
template <bool SHIFT>
__device__ __forceinline__ void stage_weights(float* s, const void* w, int dtype, int D) {
  if constexpr (SHIFT) {
    for (int i = threadIdx.x; i < D + 16; i += blockDim.x) {
      const int d = i - 8;
      float v = 0.0f;
      if (w && d >= 0 && d < D)
        v = dtype == MOE_DTYPE_F32 ? __ldg(static_cast<const float*>(w) + d)
                                   : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + d));
      s[i + (i >> 5)] = v;
    }
  } else {
    for (int c = threadIdx.x; c < D / 8; c += blockDim.x) {
      float v[8] = {};
      if (w) {
        if (dtype == MOE_DTYPE_F32) {
          Piece<float, 8> p;
          p.load(static_cast<const float*>(w) + 8 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = p.get(i);
        } else {
          Piece<__nv_bfloat16, 8> p;
          p.load(static_cast<const __nv_bfloat16*>(w) + 8 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = p.get(i);
        }
      }
      reinterpret_cast<float4*>(s)[c] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(s + D / 2)[c] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}
// Pairs 0 .. 3 of the 8 weights from column d (SHIFT: -7 .. D - 1; 0 outside the row).
template <bool SHIFT>
__device__ __forceinline__ void shared_weights(const float* s, int d, int D, f2* w) {
  if constexpr (SHIFT) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = d + 8 + 2 * j;
      w[j] = pack(s[i + (i >> 5)], s[i + 1 + ((i + 1) >> 5)]);
    }
  } else {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s + (d >> 1));
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(s + D / 2 + (d >> 1));
    w[0] = a.x;
    w[1] = a.y;
    w[2] = b.x;
    w[3] = b.y;
  }
}

template <typename T>
__device__ __forceinline__ f2 piece_pair(const Piece<T, 8>& p, int j) {
  return pack(p.get(2 * j), p.get(2 * j + 1));
}
// Stores 8 values held as pairs.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const f2* v) {
  float o[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 u = unpack(v[j]);
    o[2 * j] = u.x;
    o[2 * j + 1] = u.y;
  }
  Piece<T, 8>::store(p, o);
}

// Of a piece that is not whole: zeros outside the row; its values where the copy of the
// tensors' last row left them out; its stores.
__device__ __forceinline__ f2 masked_pair(f2 v, int d, int D) {
  const float2 u = unpack(v);
  return pack(d >= 0 && d < D ? u.x : 0.0f, d + 1 >= 0 && d + 1 < D ? u.y : 0.0f);
}
template <typename T>
__device__ __forceinline__ f2 direct_pair(const T* row, int d, int D) {
  return pack(d >= 0 && d < D ? to_f32(__ldg(row + d)) : 0.0f,
              d + 1 >= 0 && d + 1 < D ? to_f32(__ldg(row + d + 1)) : 0.0f);
}
template <typename T>
__device__ __forceinline__ void store_part(T* row, int d, int D, const f2* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 u = unpack(v[j]);
    const int k = d + 2 * j;
    if (k >= 0 && k < D) put(row + k, u.x);
    if (k + 1 >= 0 && k + 1 < D) put(row + k + 1, u.y);
  }
}
// The pairs of a row's piece in shared memory from column d, `piece` 8 values in.
template <typename T, bool SHIFT>
__device__ __forceinline__ void row_piece(const Placing<T, SHIFT>& at, uint32_t slot, int piece, int d, const T* row,
                                          bool last, f2* v) {
  const Piece<T, 8> p = shared_piece<T>(slot, piece * 8);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = piece_pair(p, j);
  if (!at.whole(d)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = last ? direct_pair(row, d + 2 * j, at.D) : masked_pair(v[j], d + 2 * j, at.D);
  }
}

// The barriers of all rings of the block, and this group's ring.
__device__ __forceinline__ Ring make_ring(uint8_t* rows, uint64_t* bars, int mats, int stages, int slot, int groups,
                                          int group) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < groups; ++i)
      for (int st = 0; st < stages; ++st) tc::mbar_init(tc::smem_u32(bars + i * kMaxStages + st), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tc::fence_proxy_async_shared();
  }
  Ring r;
  r.slot = slot;
  r.mats = mats;
  r.stages = stages;
  r.base = tc::smem_u32(rows) + (uint32_t)(group * stages * mats * slot);
  r.bars = tc::smem_u32(bars + group * kMaxStages);
  return r;
}

// After a copy that did not land: those under way do so before the block ends.
__device__ __forceinline__ void drain_ring(unsigned int* err) {
  flag_error(err, MOE_DEVERR_TIMEOUT);
  const uint64_t since = tc::global_timer_ns();
  while (tc::global_timer_ns() - since < tc::kDrainTimeoutNs) {
  }
}

constexpr int kRingValues = 32;  // a thread's values in the ring kernels, 4 pieces of 8

// The sums of a group's warps; ok: whether every thread of it says so.
__device__ __forceinline__ float2 ring_sum(float2 v, float2* s, int group, int R, bool* ok) {
  v = make_float2(warp_sum(v.x), warp_sum(v.y));
  if (R == 32) {
    *ok = __all_sync(0xffffffffu, *ok);
    return v;
  }
  const int gt = threadIdx.x - group * R, first = group * (R / 32);
  if ((gt & 31) == 0) s[first + (gt >> 5)] = v;
  *ok = group_agrees(*ok, group, R);
  v = make_float2(0.0f, 0.0f);
  for (int i = 0; i < R / 32; ++i) {
    v.x += s[first + i].x;
    v.y += s[first + i].y;
  }
  return v;
}

template <typename T, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_ring_kernel(const NormArgs g, int R, float inv_d, int stages) {
  extern __shared__ __align__(128) uint8_t s_mem[];  // gamma, beta, the rings
  __shared__ float2 s_sum[2][2][THREADS / 32];       // by turns, two sums of each warp
  __shared__ uint64_t s_bars[kMaxGroups * kMaxStages];
  const int groups = blockDim.x / R, group = threadIdx.x / R, gt = threadIdx.x - group * R;
  const int n = read_count(g.valid, g.T, g.err), D = g.D;
  const int64_t stride = (int64_t)gridDim.x * groups;
  int64_t t = (int64_t)blockIdx.x * groups + group, ahead = t;  // the next row to fill a stage with
  const T* x0 = static_cast<const T*>(g.x);
  const Placing<T, SHIFT> at(D, g.T, t);
  float* gamma = reinterpret_cast<float*>(s_mem);
  float* beta = gamma + weight_floats<SHIFT>(D);
  Ring ring = make_ring(reinterpret_cast<uint8_t*>(beta + weight_floats<SHIFT>(D)), s_bars, 1, stages,
                        slot_bytes<T>(D, SHIFT), groups, group);
  auto fill = [&] { ring.fill(x0 + ahead * g.ldx - at.sh, nullptr, at.bytes(ahead)); };
  __syncthreads();
  if (gt == 0)
    for (int st = 0; st < stages - 1 && ahead < n; ++st, ahead += stride) fill();
  stage_weights<SHIFT>(gamma, g.gamma, g.weight_dtype, D);
  stage_weights<SHIFT>(beta, g.beta, g.weight_dtype, D);
  __syncthreads();
  bool ok = true;
  for (int turn = 0; t < n; t += stride, turn ^= 1) {
    ok = ring.wait();
    const T* row = x0 + t * g.ldx;
    f2 v[kRingValues / 2], s = both(0.0f);
#pragma unroll
    for (int c = 0; c < kRingValues / 8; ++c) {
      const int d = at.column(c * R + gt);
      if (at.any(d)) {
        row_piece(at, ring.at(ring.stage, 0), c * R + gt, d, row, t == at.last, v + 4 * c);
#pragma unroll
        for (int j = 4 * c; j < 4 * c + 4; ++j) s = add2(s, v[j]);
      }
    }
    const float mean = ring_sum(make_float2(sum2(s), 0.0f), s_sum[turn][0], group, R, &ok).x * inv_d;
    if (!ok) break;
    // the group has read this row and those before: refill the stage of the last
    if (gt == 0 && ahead < n) {
      tc::fence_proxy_async_shared();
      fill();
    }
    ahead += stride;
    ring.advance();
    s = both(0.0f);
#pragma unroll
    for (int c = 0; c < kRingValues / 8; ++c) {
      const int d = at.column(c * R + gt);
      if (at.any(d)) {
#pragma unroll
        for (int j = 4 * c; j < 4 * c + 4; ++j) v[j] = add2(v[j], both(-mean));
        if (!at.whole(d)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * c + j] = masked_pair(v[4 * c + j], d + 2 * j, D);
        }
#pragma unroll
        for (int j = 4 * c; j < 4 * c + 4; ++j) s = fma2(v[j], v[j], s);
      }
    }
    const float rstd =
        rsqrtf(ring_sum(make_float2(sum2(s), 0.0f), s_sum[turn][1], group, R, &ok).x * inv_d + g.eps);
    T* y = static_cast<T*>(g.y) + t * D;
#pragma unroll
    for (int c = 0; c < kRingValues / 8; ++c) {
      const int d = at.column(c * R + gt);
      if (at.any(d)) {
        f2 w[4], b[4];
        shared_weights<SHIFT>(gamma, d, D, w);
        shared_weights<SHIFT>(beta, d, D, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = fma2(mul2(v[4 * c + j], both(rstd)), w[j], b[j]);
        if (at.whole(d)) store_piece(y + d, w);
        else store_part(y, d, D, w);
      }
    }
    if (gt == 0) {
      if (g.mean) g.mean[t] = mean;
      if (g.rstd) g.rstd[t] = rstd;
    }
  }
  if (t < n && gt == 0) drain_ring(g.err);
}

// This block's row of partial [blocks][2][D]: each group's sums into s [groups][2][D], whose
// columns are then added over the groups in order.  A thread's piece c of VEC values begins
// at column col(c); WHOLE: no piece reaches past the row.
template <int VEC, int C, bool WHOLE, typename F>
__device__ __forceinline__ void store_partial(float* partial, float* s, const f2* dg, const f2* db, int group,
                                              int groups, int D, F col) {
  __syncthreads();  // s is free
  float* mine = s + (int64_t)group * 2 * D;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int d = col(c);
    if (d >= D) continue;
    if constexpr (VEC == 8 && !WHOLE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = unpack(dg[4 * c + j]), b = unpack(db[4 * c + j]);
        const int k = d + 2 * j;
        if (k >= 0 && k < D) {
          mine[k] = a.x;
          mine[D + k] = b.x;
        }
        if (k + 1 >= 0 && k + 1 < D) {
          mine[k + 1] = a.y;
          mine[D + k + 1] = b.y;
        }
      }
    } else if constexpr (VEC == 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<ulonglong2*>(mine + d + 4 * h) = make_ulonglong2(dg[4 * c + 2 * h], dg[4 * c + 2 * h + 1]);
        *reinterpret_cast<ulonglong2*>(mine + D + d + 4 * h) =
            make_ulonglong2(db[4 * c + 2 * h], db[4 * c + 2 * h + 1]);
      }
    } else {
      const float2 a = unpack(dg[c / 2]), b = unpack(db[c / 2]);
      mine[d] = c & 1 ? a.y : a.x;
      mine[D + d] = c & 1 ? b.y : b.x;
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < 2 * D; d += blockDim.x) {
    float v = s[d];
    for (int k = 1; k < groups; ++k) v += s[(int64_t)k * 2 * D + d];
    partial[(int64_t)blockIdx.x * 2 * D + d] = v;
  }
}

template <typename T, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    norm_grad_ring_kernel(const NormArgs g, int R, float inv_d, int stages, float* partial) {
  extern __shared__ __align__(128) uint8_t s_mem[];  // gamma, the rings; then the groups' sums
  __shared__ float2 s_sum[2][THREADS / 32];          // by turns, two sums of each warp
  __shared__ uint64_t s_bars[kMaxGroups * kMaxStages];
  pdl_launch_dependents();                           // the reduction's blocks wait for this grid's end
  const int groups = blockDim.x / R, group = threadIdx.x / R, gt = threadIdx.x - group * R;
  const int n = read_count(g.valid, g.T, g.err), D = g.D;
  const int64_t stride = (int64_t)gridDim.x * groups;
  int64_t t = (int64_t)blockIdx.x * groups + group, ahead = t;
  const T* x0 = static_cast<const T*>(g.x);
  const T* dy0 = static_cast<const T*>(g.dy);
  const Placing<T, SHIFT> at(D, g.T, t);
  float* gamma = reinterpret_cast<float*>(s_mem);
  Ring ring = make_ring(reinterpret_cast<uint8_t*>(gamma + weight_floats<SHIFT>(D)), s_bars, 2, stages,
                        slot_bytes<T>(D, SHIFT), groups, group);
  auto fill = [&] { ring.fill(x0 + ahead * g.ldx - at.sh, dy0 + ahead * D - at.sh, at.bytes(ahead)); };
  __syncthreads();
  if (gt == 0)
    for (int st = 0; st < stages - 1 && ahead < n; ++st, ahead += stride) fill();
  stage_weights<SHIFT>(gamma, g.gamma, g.weight_dtype, D);
  __syncthreads();
  f2 dg[kRingValues / 2], db[kRingValues / 2];
#pragma unroll
  for (int j = 0; j < kRingValues / 2; ++j) dg[j] = db[j] = both(0.0f);
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (t < n) {
    next_mean = __ldg(g.mean + t);
    next_rstd = __ldg(g.rstd + t);
  }
  bool ok = true;
  for (int turn = 0; t < n; t += stride, turn ^= 1) {
    const float rstd = next_rstd;
    const f2 r2 = both(rstd), m2 = both(-next_mean);
    if (t + stride < n) {
      next_mean = __ldg(g.mean + t + stride);
      next_rstd = __ldg(g.rstd + t + stride);
    }
    ok = ring.wait();
    const uint32_t xr = ring.at(ring.stage, 0), dyr = ring.at(ring.stage, 1);
    const T* x = x0 + t * g.ldx;
    const T* dy = dy0 + t * D;
    f2 s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
    for (int c = 0; c < kRingValues / 8; ++c) {
      const int d = at.column(c * R + gt);
      if (at.any(d)) {
        f2 px[4], py[4], w[4];
        row_piece(at, xr, c * R + gt, d, x, t == at.last, px);
        row_piece(at, dyr, c * R + gt, d, dy, t == at.last, py);
        shared_weights<SHIFT>(gamma, d, D, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f2 xc = add2(px[j], m2), gd = mul2(py[j], w[j]);
          dg[4 * c + j] = fma2(mul2(py[j], r2), xc, dg[4 * c + j]);
          db[4 * c + j] = add2(db[4 * c + j], py[j]);
          s0 = add2(s0, gd);
          s1 = fma2(gd, xc, s1);
        }
      }
    }
    const float2 s = ring_sum(make_float2(sum2(s0), sum2(s1)), s_sum[turn], group, R, &ok);
    if (!ok) break;
    // the group is past the row before this one: refill its stage
    if (gt == 0 && ahead < n) {
      tc::fence_proxy_async_shared();
      fill();
    }
    ahead += stride;
    // dx = r gd - r m0 - (x - mean) r^2 m1 with m0 = (1/D) sum gd, m1 = (1/D) sum gd r (x - mean)
    const f2 k0 = both(-rstd * s.x * inv_d), k1 = both(-(rstd * s.y * inv_d) * rstd * rstd);
    T* dx = static_cast<T*>(g.y) + t * D;
    const T* res = g.residual ? static_cast<const T*>(g.residual) + t * D : nullptr;
#pragma unroll
    for (int c = 0; c < kRingValues / 8; ++c) {
      const int d = at.column(c * R + gt);
      if (at.any(d)) {
        f2 px[4], py[4], w[4];
        row_piece(at, xr, c * R + gt, d, x, t == at.last, px);
        row_piece(at, dyr, c * R + gt, d, dy, t == at.last, py);
        shared_weights<SHIFT>(gamma, d, D, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = fma2(mul2(py[j], w[j]), r2, fma2(add2(px[j], m2), k1, k0));
        if (at.whole(d)) {
          if (res) {
            Piece<T, 8> pr;
            pr.load(res + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = add2(w[j], piece_pair(pr, j));
          }
          store_piece(dx + d, w);
        } else {
          if (res) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = add2(w[j], direct_pair(res, d + 2 * j, D));
          }
          store_part(dx, d, D, w);
        }
      }
    }
    ring.advance();
  }
  if (t < n && gt == 0) drain_ring(g.err);
  store_partial<8, kRingValues / 8, !SHIFT>(partial, reinterpret_cast<float*>(s_mem), dg, db, group, groups, D,
                                            [&](int c) { return at.column(c * R + gt); });
}

// Rows straight into registers.
// Blocks of a direct kernel that share an SM's registers: with single columns one row in
// flight does not hide its loads.
constexpr int direct_blocks(int vec, int threads) { return vec == 1 ? (threads <= 320 ? 3 : 2) : 1; }

template <typename T, typename W, int VEC, int N, int THREADS>
__global__ void __launch_bounds__(THREADS, direct_blocks(VEC, THREADS))
    norm_kernel(const NormArgs g, int R, float inv_d) {
  __shared__ float2 s_sum[2][2][THREADS / 32];  // by turns, two sums of each warp
  const int groups = blockDim.x / R, group = threadIdx.x / R, gt = threadIdx.x - group * R;
  const int n = read_count(g.valid, g.T, g.err), D = g.D;
  const int64_t stride = (int64_t)gridDim.x * groups;
  bool ok = true;
  int turn = 0;
  for (int64_t t = (int64_t)blockIdx.x * groups + group; t < n; t += stride, turn ^= 1) {
    Row<T, VEC, N> x;
    x.clear();
    x.load(static_cast<const T*>(g.x) + t * g.ldx, R, gt, D);
    f2 v[N / 2], s = both(0.0f);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      v[j] = x.pair(j);
      s = add2(s, v[j]);
    }
    const float mean = ring_sum(make_float2(sum2(s), 0.0f), s_sum[turn][0], group, R, &ok).x * inv_d;
    s = both(0.0f);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      v[j] = add2(v[j], both(-mean));
      const bool in0 = ((2 * j / VEC) * R + gt) * VEC < D, in1 = (((2 * j + 1) / VEC) * R + gt) * VEC < D;
      const float2 u = unpack(v[j]);
      v[j] = pack(in0 ? u.x : 0.0f, in1 ? u.y : 0.0f);
      s = fma2(v[j], v[j], s);
    }
    Row<W, VEC, N> gamma, beta;
    beta.clear();
    gamma.load(static_cast<const W*>(g.gamma), R, gt, D);
    if (g.beta) beta.load(static_cast<const W*>(g.beta), R, gt, D);
    const float rstd =
        rsqrtf(ring_sum(make_float2(sum2(s), 0.0f), s_sum[turn][1], group, R, &ok).x * inv_d + g.eps);
    Row<T, VEC, N>::store(static_cast<T*>(g.y) + t * D, R, gt, D, [&](int j) {
      return fma2(mul2(v[j], both(rstd)), gamma.pair(j), beta.pair(j));
    });
    if (gt == 0) {
      if (g.mean) g.mean[t] = mean;
      if (g.rstd) g.rstd[t] = rstd;
    }
  }
}

template <typename T, typename W, int VEC, int N, int THREADS>
__global__ void __launch_bounds__(THREADS, VEC == 1 && THREADS <= 512 ? 2 : 1)
    norm_grad_kernel(const NormArgs g, int R, float inv_d, float* partial) {
  extern __shared__ __align__(128) uint8_t s_mem[];  // the groups' sums
  __shared__ float2 s_sum[2][THREADS / 32];
  pdl_launch_dependents();
  const int groups = blockDim.x / R, group = threadIdx.x / R, gt = threadIdx.x - group * R;
  const int n = read_count(g.valid, g.T, g.err), D = g.D;
  const int64_t stride = (int64_t)gridDim.x * groups;
  f2 dg[N / 2], db[N / 2];
#pragma unroll
  for (int j = 0; j < N / 2; ++j) dg[j] = db[j] = both(0.0f);
  bool ok = true;
  int turn = 0;
  for (int64_t t = (int64_t)blockIdx.x * groups + group; t < n; t += stride, turn ^= 1) {
    Row<T, VEC, N> x, dy;
    Row<W, VEC, N> gamma;
    x.clear();
    dy.clear();
    gamma.clear();
    x.load(static_cast<const T*>(g.x) + t * g.ldx, R, gt, D);
    dy.load(static_cast<const T*>(g.dy) + t * D, R, gt, D);
    gamma.load(static_cast<const W*>(g.gamma), R, gt, D);
    const float rstd = __ldg(g.rstd + t);
    const f2 r2 = both(rstd), m2 = both(-__ldg(g.mean + t));
    f2 s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const f2 y = dy.pair(j), xc = add2(x.pair(j), m2), gd = mul2(y, gamma.pair(j));
      dg[j] = fma2(mul2(y, r2), xc, dg[j]);
      db[j] = add2(db[j], y);
      s0 = add2(s0, gd);
      s1 = fma2(gd, xc, s1);
    }
    const float2 s = ring_sum(make_float2(sum2(s0), sum2(s1)), s_sum[turn], group, R, &ok);
    const f2 k0 = both(-rstd * s.x * inv_d), k1 = both(-(rstd * s.y * inv_d) * rstd * rstd);
    auto grad = [&](int j) {
      return fma2(mul2(dy.pair(j), gamma.pair(j)), r2, fma2(add2(x.pair(j), m2), k1, k0));
    };
    T* dx = static_cast<T*>(g.y) + t * D;
    if (g.residual) {
      Row<T, VEC, N> res;
      res.clear();
      res.load(static_cast<const T*>(g.residual) + t * D, R, gt, D);
      Row<T, VEC, N>::store(dx, R, gt, D, [&](int j) { return add2(grad(j), res.pair(j)); });
    } else {
      Row<T, VEC, N>::store(dx, R, gt, D, grad);
    }
  }
  store_partial<VEC, N / VEC, true>(partial, reinterpret_cast<float*>(s_mem), dg, db, group, groups, D,
                                    [&](int c) { return (c * R + gt) * VEC; });
}

// dgamma and dbeta: a block of 32 columns of the 2 D and 32 lanes of rows, each adding every
// 32nd block's partial sum; the lanes are then added in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ partial, int blocks, int D,
                                                           float* dgamma, float* dbeta) {
  __shared__ float s[32][33];
  pdl_wait();
  const int c = threadIdx.x & 31, l = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;
  float v = 0.0f;
  if (col < 2 * (int64_t)D) {
    float a[5];  // 152 blocks in one round of loads
    for (int b = l; b < blocks; b += 5 * 32) {
#pragma unroll
      for (int i = 0; i < 5; ++i) a[i] = b + 32 * i < blocks ? partial[(int64_t)(b + 32 * i) * 2 * D + col] : 0.0f;
#pragma unroll
      for (int i = 0; i < 5; ++i) v += a[i];
    }
  }
  s[l][c] = v;
  __syncthreads();
  v = warp_sum(s[c][l]);  // column l, lane c
  const int64_t out = (int64_t)blockIdx.x * 32 + l;
  if (c == 0 && out < 2 * (int64_t)D) {
    if (out < D) dgamma[out] = v;
    else if (dbeta) dbeta[out - D] = v;
  }
}

template <int V>
struct Int {
  static constexpr int v = V;
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// How the rows lie: in whole 16-byte pieces (kWide); at offsets that are the same for all of a
// row's tensors (kShifted); or neither.
enum Layout { kWide, kShifted, kSingle };

Layout layout_of(const NormArgs& g) {
  const int es = g.dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!aligned16(g.x) || !aligned16(g.y) || !aligned16(g.dy) || !aligned16(g.residual)) return kSingle;
  if (g.D % 8 == 0 && g.ldx * es % 16 == 0 && aligned16(g.gamma) && aligned16(g.beta)) return kWide;
  return (g.ldx - g.D) * es % 16 == 0 ? kShifted : kSingle;
}

// f(x element, weight element, layout)
template <typename F>
cudaError_t by_types(const NormArgs& g, F f) {
  const bool xf = g.dtype == MOE_DTYPE_F32, wf = g.weight_dtype == MOE_DTYPE_F32;
  const Layout layout = layout_of(g);
  auto with_layout = [&](auto x, auto w) {
    return layout == kWide      ? f(x, w, Int<kWide>{})
           : layout == kShifted ? f(x, w, Int<kShifted>{})
                                : f(x, w, Int<kSingle>{});
  };
  if (xf) return wf ? with_layout(float{}, float{}) : with_layout(float{}, __nv_bfloat16{});
  return wf ? with_layout(__nv_bfloat16{}, float{}) : with_layout(__nv_bfloat16{}, __nv_bfloat16{});
}

// How a row of D columns is held: values a thread, threads of its group, groups of a block
// of up to `most` threads.
struct Shape {
  int n, R, groups;
};
Shape shape(int D, int n, int most) {
  const int R = ((D + n - 1) / n + 31) / 32 * 32, groups = most / R;
  return {n, R, groups < 1 ? 1 : groups > kMaxGroups ? kMaxGroups : groups};
}

// Rows up to this are a warp's (8 or 16 values a thread).  16384 rows of 512 in bf16 take 12.4 us, 17.8
// backward, and 15.1, 21.4 through the ring; rows of 640 24.4, 31.7 in two warps, 17.5, 24.8 through it.
constexpr int kWarpColumns = 512;
// Of a ring kernel's block, in whole groups; fewer where the pieces at a row's ends cost registers.
constexpr int forward_threads(bool shift) { return shift ? 640 : 768; }
constexpr int backward_threads(bool shift) { return shift ? 384 : 512; }
constexpr int kRingBytes = 216 * 1024;

// Rows without whole pieces up to here are held 8 columns a thread, and that is faster than
// their ring: forward, 2400 rows of 1001 in bf16 take 9 us and 13 through the ring, rows of
// 2051 28 and 17; backward, 2400 rows of 2051 take 23 and 25, rows of 4097 68 and 45.
constexpr int kSingleForward = 8 * 256, kSingleBackward = 8 * 320;

static_assert(kNumSmsGB300 % 8 == 0, "a group's rows are a multiple of 8 apart");
// The backward's grid: up to `each` blocks for each SM, fewer for few rows.
int grad_blocks(int T, const Shape& sh, int each) {
  const int64_t need = ((int64_t)T + sh.groups - 1) / sh.groups, most = (int64_t)kNumSmsGB300 * each;
  return (int)(need < most ? need : most);
}
constexpr int kMaxGradEach = 2;

// The ring kernels' shape: the most groups that leave two stages or more for each beside
// `fixed` bytes; stages 0: none do.
Shape ring_shape(int D, bool shift, int most, int64_t fixed, int64_t stage_bytes, int* stages) {
  Shape sh = shape(shift ? D + 7 : D, kRingValues, most);
  *stages = 0;
  if (sh.R > most) return sh;
  for (;; --sh.groups) {
    const int64_t n = (kRingBytes - fixed) / (sh.groups * stage_bytes);
    *stages = n < 2 ? 0 : n > kMaxStages ? kMaxStages : (int)n;
    if (*stages || sh.groups == 1) return sh;
  }
}

template <typename T, bool SHIFT>
cudaError_t forward_ring(const NormArgs& g, const Shape& sh, int stages, cudaStream_t s) {
  auto kern = norm_ring_kernel<T, SHIFT, forward_threads(SHIFT)>;
  const size_t smem = (size_t)8 * weight_floats<SHIFT>(g.D) + (size_t)sh.groups * stages * slot_bytes<T>(g.D, SHIFT);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t need = ((int64_t)g.T + sh.groups - 1) / sh.groups;
  const int64_t most = (device_sm_count() + 7) / 8 * 8;  // a group's rows are a multiple of 8 apart, or it has one
  kern<<<(int)(need < most ? need : most), sh.groups * sh.R, smem, s>>>(g, sh.R, 1.0f / g.D, stages);
  return cudaGetLastError();
}

template <typename T, typename W, int VEC, int N, int THREADS>
cudaError_t forward(const NormArgs& g, const Shape& sh, cudaStream_t s) {
  const int64_t need = ((int64_t)g.T + sh.groups - 1) / sh.groups;
  const int64_t most = (int64_t)device_sm_count() * (VEC == 1 ? direct_blocks(VEC, THREADS) : 2048 / THREADS);
  norm_kernel<T, W, VEC, N, THREADS>
      <<<(int)(need < most ? need : most), sh.groups * sh.R, 0, s>>>(g, sh.R, 1.0f / g.D);
  return cudaGetLastError();
}

template <typename T, bool SHIFT>
cudaError_t backward_ring(const NormArgs& g, const Shape& sh, int stages, int* blocks, cudaStream_t s) {
  auto kern = norm_grad_ring_kernel<T, SHIFT, backward_threads(SHIFT)>;
  size_t smem = (size_t)4 * weight_floats<SHIFT>(g.D) + (size_t)sh.groups * stages * 2 * slot_bytes<T>(g.D, SHIFT);
  if (smem < (size_t)sh.groups * 8 * g.D) smem = (size_t)sh.groups * 8 * g.D;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  *blocks = grad_blocks(g.T, sh, 1);
  kern<<<*blocks, sh.groups * sh.R, smem, s>>>(g, sh.R, 1.0f / g.D, stages, static_cast<float*>(g.ws));
  return cudaGetLastError();
}

template <typename T, typename W, int VEC, int N, int THREADS>
cudaError_t backward(const NormArgs& g, const Shape& sh, int* blocks, cudaStream_t s) {
  auto kern = norm_grad_kernel<T, W, VEC, N, THREADS>;
  const size_t smem = (size_t)sh.groups * 8 * g.D;  // at most 128 KB: one group of 16384 columns
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  *blocks = grad_blocks(g.T, sh, VEC == 1 ? kMaxGradEach : 1);
  kern<<<*blocks, sh.groups * sh.R, smem, s>>>(g, sh.R, 1.0f / g.D, static_cast<float*>(g.ws));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const NormArgs& g, cudaStream_t s) {
  return by_types(g, [&](auto x, auto w, auto layout) {
    using T = decltype(x);
    using W = decltype(w);
    constexpr int L = decltype(layout)::v, VEC = L == kWide ? 8 : 1;
    constexpr bool SHIFT = L == kShifted;
    const int D = g.D;
    // few rows: a block each, with nothing to fill a ring with (bf16: 304 rows of 5120 4.0 us, 5.8 through the
    // ring, 1216 11.2 and 9.5; of 1024 columns direct wins longer: 1216 rows 4.4 and 6.7, 16384 25.5 and 20.5)
    if (L != kSingle && D > (SHIFT ? kSingleForward : kWarpColumns) && g.T > 2 * device_sm_count()) {
      int stages;
      const Shape sh = ring_shape(D, SHIFT, forward_threads(SHIFT), (int64_t)8 * weight_floats<SHIFT>(D),
                                  slot_bytes<T>(D, SHIFT), &stages);
      if (stages) return forward_ring<T, SHIFT>(g, sh, stages, s);
    }
    if constexpr (VEC == 8) {
      if (D <= 8 * 32) return forward<T, W, VEC, 8, 256>(g, shape(D, 8, 256), s);
      if (D <= kWarpColumns) return forward<T, W, VEC, 16, 256>(g, shape(D, 16, 256), s);
      return forward<T, W, VEC, 32, 512>(g, shape(D, 32, 1), s);
    } else {
      if (D <= kSingleForward) return forward<T, W, VEC, 8, 256>(g, shape(D, 8, 256), s);
      if (D <= 16 * 512) return forward<T, W, VEC, 16, 512>(g, shape(D, 16, 512), s);
      return forward<T, W, VEC, 32, 512>(g, shape(D, 32, 512), s);
    }
  });
}

size_t layer_norm_backward_workspace_bytes(int T, int D) {
  if (D == 0) return 0;
  // of the kernel with the most blocks (which one runs goes by the rows' alignment too)
  const int64_t most = (int64_t)kNumSmsGB300 * kMaxGradEach;
  return (size_t)(T < most ? T : most) * 2 * D * sizeof(float);
}

cudaError_t launch_layer_norm_backward(const NormArgs& g, cudaStream_t s) {
  int blocks = 0;
  if (g.T > 0) {
    cudaError_t e = by_types(g, [&](auto x, auto w, auto layout) {
      using T = decltype(x);
      using W = decltype(w);
      constexpr int L = decltype(layout)::v, VEC = L == kWide ? 8 : 1;
      constexpr bool SHIFT = L == kShifted;
      const int D = g.D;
      if (L != kSingle && D > (SHIFT ? kSingleBackward : kWarpColumns)) {
        int stages;
        const Shape sh = ring_shape(D, SHIFT, backward_threads(SHIFT), (int64_t)4 * weight_floats<SHIFT>(D),
                                    2 * slot_bytes<T>(D, SHIFT), &stages);
        if (stages) return backward_ring<T, SHIFT>(g, sh, stages, &blocks, s);
      }
      if constexpr (VEC == 8) {
        if (D <= 8 * 32) return backward<T, W, VEC, 8, 320>(g, shape(D, 8, 320), &blocks, s);
        if (D <= kWarpColumns) return backward<T, W, VEC, 16, 320>(g, shape(D, 16, 320), &blocks, s);
        // fp32 rows of more than 11000 columns (every bf16 row fits the ring)
        if constexpr (sizeof(T) == 4) return backward<T, W, VEC, 32, 512>(g, shape(D, 32, 1), &blocks, s);
        return cudaErrorInvalidValue;
      } else {
        if (D <= kSingleBackward) return backward<T, W, VEC, 8, 320>(g, shape(D, 8, 320), &blocks, s);
        if (D <= 16 * 320) return backward<T, W, VEC, 16, 320>(g, shape(D, 16, 320), &blocks, s);
        return backward<T, W, VEC, 16, 1024>(g, shape(D, 16, 1), &blocks, s);
      }
    });
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((2 * (int64_t)g.D + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, norm_reduce_kernel, static_cast<const float*>(g.ws), blocks, g.D, g.dgamma,
                                     g.dbeta);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace moe
