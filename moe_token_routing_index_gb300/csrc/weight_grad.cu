// The experts' weight gradients dW[e] = dY_e^T X_e (include/moe_train.h) on the
// 5th-generation tensor cores.
//
// Both operands are row-major with the reduction (the expert's rows) as their outer
// dimension, so a TMA box of 64 rows x 128 bytes lands in shared memory as an
// MN-major, 128B-swizzled operand and nothing is transposed.
//
// Kernel structure (one CTA per SM, persistent, 6 warps), tiles of 128 columns of dY
// x 256 columns of X of one expert:
//   warp 0     TMA producer: 64 rows of the two operands per stage (16 + 32 KB) into a
//              4-stage ring guarded by mbarriers.
//   warp 1     MMA issuer: tcgen05.mma (M = 128, N = 256, 16 rows each) into one of two
//              256-column accumulators.  Where an expert's rows end inside a step of 16,
//              the warp first zeroes the rest of that step in shared memory: those rows
//              belong to the next expert, or to none, and may hold anything.
//   warps 2-5  epilogue: accumulator rows through a staging block to TMA stores (or fp32
//              reductions, for accumulate) that clip at the edges of dW[e].
// An expert without rows has its tiles written as zeros by the epilogue alone.
//
// Every mbarrier wait is bounded; on expiry the kernel records MOE_DEVERR_TIMEOUT,
// all roles stop, copies and MMAs in flight are drained, and tensor memory is freed.
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"
#include "train_launch.h"

namespace moe {
namespace {

using namespace tc;

constexpr int kBM = 128, kBN = 256;       // tile: columns of dY, columns of X
constexpr int kBR = 64;                   // rows per stage
constexpr int kBoxCols = 64, kBoxBytes = kBR * 128;
constexpr int kABoxes = kBM / kBoxCols, kBBoxes = kBN / kBoxCols;
constexpr int kStageBytes = (kABoxes + kBBoxes) * kBoxBytes;  // 48 KB
constexpr int kStages = 4, kAccBufs = 2;
constexpr int kTmemCols = kAccBufs * kBN;
constexpr int kThreads = 192;
constexpr int kEpiStageBytes = 32 * 128;  // per epilogue warp: 32 rows x 128 bytes

struct Smem {
  static constexpr int stage = 0;
  static constexpr int epi = stage + kStages * kStageBytes;
  static constexpr int bars = epi + 4 * kEpiStageBytes;  // full[S], empty[S], tfull[2], tempty[2], drain
  static constexpr int misc = bars + (2 * kStages + 2 * kAccBufs + 1) * 8;
  static constexpr int rows = misc + 16;  // row_off[E + 1]
  static constexpr int bytes_for(int E) { return rows + (E + 1) * 4; }
};

struct Shape {
  int E, a_max, N, K;
  int mt, kt;       // tiles of an expert along N and K
  int f32, accumulate;
};

// Shared-memory descriptor of an MN-major operand, 128B swizzle: 64-column blocks one
// box apart, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kBoxBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// mbar_wait by a whole warp, whose lanes agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}

struct Tile {
  int expert, n0, k0, row0, rows;
};

// Tile id -> expert and place: an expert's tiles in groups of 16 along N, N innermost,
// so the CTAs running together read few columns of either operand.
__device__ __forceinline__ Tile locate(const Shape& p, int64_t tile, const int* row_off) {
  const int per = p.mt * p.kt;
  Tile t;
  t.expert = (int)(tile / per);
  const int local = (int)(tile - (int64_t)t.expert * per);
  const int group = local / (16 * p.kt), in = local - group * 16 * p.kt;
  const int width = min(16, p.mt - group * 16);
  t.n0 = (group * 16 + in % width) * kBM;
  t.k0 = in / width * kBN;
  t.row0 = row_off[t.expert];
  t.rows = row_off[t.expert + 1] - t.row0;
  return t;
}

// One accumulator tile of one epilogue warp: rows n0 + 32 sub + lane, in chunks of 128
// bytes of a row.  zero: the tile of an expert without rows.
__device__ __forceinline__ void store_tile(const Shape& p, const Tile& t, int sub, int lane, uint32_t tbase, bool zero,
                                           uint8_t* stage, const CUtensorMap* map) {
  const int row = t.n0 + 32 * sub;
  if (row >= p.N) return;
  const int step = p.f32 ? 32 : 64;
  const int cols = min(kBN, p.K - t.k0);
#pragma unroll 1
  for (int c = 0; c < cols; c += step) {
    float v[64];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 64; ++i) v[i] = 0.0f;
    } else {
      tmem_ld32(tbase + c, v);
      if (!p.f32) tmem_ld32(tbase + c + 32, v + 32);
    }
    if (lane == 0) bulk_wait_group_read0();  // the previous store has read the staging block
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint4 o;
      if (p.f32)
        o = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                       __float_as_uint(v[4 * q + 3]));
      else
        o = f32_to_bf16x8(v + 8 * q);
      *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) = o;
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (p.accumulate) tma_add_3d(map, smem_u32(stage), t.k0 + c, row, t.expert);
      else tma_store_3d(map, smem_u32(stage), t.k0 + c, row, t.expert);
      bulk_commit_group();
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    weight_grad_kernel(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_x,
                       const __grid_constant__ CUtensorMap map_dw, const int32_t* __restrict__ counts, const Shape p,
                       unsigned int* err) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::bars);
  auto bar_full = [&](int s) { return smem_u32(&bars[s]); };
  auto bar_empty = [&](int s) { return smem_u32(&bars[kStages + s]); };
  auto bar_tfull = [&](int b) { return smem_u32(&bars[2 * kStages + b]); };
  auto bar_tempty = [&](int b) { return smem_u32(&bars[2 * kStages + kAccBufs + b]); };
  const uint32_t bar_drain = smem_u32(&bars[2 * kStages + 2 * kAccBufs]);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Smem::misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + Smem::misc + 4);
  int* row_off = reinterpret_cast<int*>(smem + Smem::rows);

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < kAccBufs; ++b) {
      mbar_init(bar_tfull(b), 1);
      mbar_init(bar_tempty(b), 4);
    }
    mbar_init(bar_drain, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tma_prefetch_desc(&map_dy);
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_dw);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 2) {
    // row offsets: a warp-wide scan of the counts, cut at a_max (64-bit: bad counts may add up past 31 bits)
    int64_t run = 0;
    bool bad = false;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      int c = e < p.E ? counts[e] : 0;
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
      if (e < p.E) row_off[e] = (int)min(run + incl - c, (int64_t)p.a_max);
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      row_off[p.E] = (int)min(run, (int64_t)p.a_max);
      if (run > p.a_max) bad = true;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) flag_error(err, MOE_DEVERR_BAD_COUNT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = *s_tmem;
  const int64_t total = (int64_t)p.E * p.mt * p.kt;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const Tile t = locate(p, tile, row_off);
        // boxes that lie past the columns are not loaded: what they leave stale reaches only
        // accumulator rows and columns that are not stored
        const int na = min(kABoxes, (p.N - t.n0 + kBoxCols - 1) / kBoxCols);
        const int nb = min(kBBoxes, (p.K - t.k0 + kBoxCols - 1) / kBoxCols);
        for (int r = 0; r < t.rows; r += kBR) {
          if (!mbar_wait(bar_empty(s), phase ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          const uint32_t dst = sbase + Smem::stage + s * kStageBytes;
          mbar_arrive_expect_tx(bar_full(s), (uint32_t)(na + nb) * kBoxBytes);
          for (int i = 0; i < na; ++i)
            tma_load_2d(dst + i * kBoxBytes, &map_dy, bar_full(s), t.n0 + i * kBoxCols, t.row0 + r);
          for (int i = 0; i < nb; ++i)
            tma_load_2d(dst + (kABoxes + i) * kBoxBytes, &map_x, bar_full(s), t.k0 + i * kBoxCols, t.row0 + r);
          issued_mask |= 1u << s;
          issued_parity = (issued_parity & ~(1u << s)) | (phase << s);
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        flag_error(err, MOE_DEVERR_TIMEOUT);
        *s_abort = 1;
        for (int i = 0; i < kStages; ++i)
          if ((issued_mask >> i) & 1u) mbar_wait(bar_full(i), (issued_parity >> i) & 1u, nullptr, kDrainTimeoutNs);
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA
    // fp32 accumulate, bf16 operands, both MN-major
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                           ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
    int s = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true, issued_any = false;
    for (int64_t tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const Tile t = locate(p, tile, row_off);
      if (t.rows == 0) continue;
      if (!warp_wait(bar_tempty(acc), acc_phase ^ 1u, s_abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc * kBN);
      for (int r = 0; r < t.rows; r += kBR) {
        if (!warp_wait(bar_full(s), phase, s_abort)) {
          ok = false;
          break;
        }
        const uint32_t a = sbase + Smem::stage + s * kStageBytes, b = a + kABoxes * kBoxBytes;
        const int left = min(t.rows - r, kBR), steps = (left + 15) / 16;
        if (left < steps * 16) {
          // zero rows left .. 16 * steps - 1 of every box (128-byte lines: the swizzle stays inside them)
          const int pieces = (steps * 16 - left) * 8;
          uint8_t* st = smem + Smem::stage + s * kStageBytes + left * 128;
          for (int box = 0; box < kABoxes + kBBoxes; ++box)
            for (int i = lane; i < pieces; i += 32)
              *reinterpret_cast<uint4*>(st + box * kBoxBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_shared();
        }
        __syncwarp();
        tc_fence_after();
        if (lane == 0) {
          for (int k = 0; k < steps; ++k)
            mma_issue<false>(d, desc_mn(a + k * 2048), desc_mn(b + k * 2048), idesc, (r | k) != 0);
          mma_commit(bar_empty(s));
        }
        issued_any = true;
        if (++s == kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) mma_commit(bar_tfull(acc));
      if (++acc == kAccBufs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      flag_error(err, MOE_DEVERR_TIMEOUT);
      *s_abort = 1;
      if (issued_any) {
        mma_commit(bar_drain);
        mbar_wait(bar_drain, 0, nullptr, kDrainTimeoutNs);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue
    const int sub = warp & 3;  // TMEM lane quarter this warp may access
    uint8_t* stage = smem + Smem::epi + (warp - 2) * kEpiStageBytes;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const Tile t = locate(p, tile, row_off);
      if (t.rows == 0) {
        if (!p.accumulate) store_tile(p, t, sub, lane, 0, true, stage, &map_dw);
        continue;
      }
      if (!warp_wait(bar_tfull(acc), acc_phase, s_abort)) {
        if (lane == 0) flag_error(err, MOE_DEVERR_TIMEOUT);
        *s_abort = 1;
        break;
      }
      tc_fence_after();
      store_tile(p, t, sub, lane, tmem_base + ((uint32_t)(sub * 32) << 16) + (uint32_t)(acc * kBN), false, stage,
                 &map_dw);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_tempty(acc));
      if (++acc == kAccBufs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_group0();  // this warp's stores are complete before the block exits
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------- host

// dW [E, N, K] as a 3-D map, boxes of 32 rows x 128 bytes in one expert: stores clip at its edges.
bool make_dw_map(CUtensorMap* map, void* base, int E, int N, int K, bool f32) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t es = f32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)E};
  cuuint64_t strides[2] = {(cuuint64_t)K * es, (cuuint64_t)N * K * es};
  cuuint32_t box[3] = {(cuuint32_t)(128 / es), 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t weight_grad_workspace_bytes(int, int a_max, int, int K, bool packed) {
  return packed ? ((size_t)a_max * K * 2 + 255) / 256 * 256 : 0;
}

cudaError_t launch_weight_grad(const WeightGradArgs& g, cudaStream_t s) {
  const void* x = g.x;
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
    x = g.ws;
  }
  const Shape p{g.E, g.a_max, g.N, g.K, (g.N + kBM - 1) / kBM, (g.K + kBN - 1) / kBN, g.dw_dtype == MOE_DTYPE_F32,
                g.accumulate};
  CUtensorMap dw, dy, mx;
  if (!make_dw_map(&dw, g.dw, g.E, g.N, g.K, p.f32)) return cudaErrorInvalidValue;
  dy = mx = dw;  // without rows nothing is loaded
  if (g.a_max > 0 && (!make_map_sw128(&dy, g.dy, g.a_max, g.N, false, kBR) ||
                      !make_map_sw128(&mx, x, g.a_max, g.K, false, kBR)))
    return cudaErrorInvalidValue;
  const int smem = Smem::bytes_for(g.E) + 1024;
  cudaError_t e = cudaFuncSetAttribute(weight_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)g.E * p.mt * p.kt;
  const int sms = device_sm_count();
  weight_grad_kernel<<<(int)(tiles < sms ? tiles : sms), kThreads, smem, s>>>(dy, mx, dw, g.counts, p, g.err);
  return cudaGetLastError();
}

}  // namespace moe
