// The experts' weight gradients dW[e] = dY_e^T X_e (include/moe_train.h) on the
// 5th-generation tensor cores.
//
// Both operands are row-major with the reduction (the expert's rows) as their outer
// dimension, so a TMA box of 96 rows x 128 bytes lands in shared memory as an
// MN-major, 128B-swizzled operand and nothing is transposed.
//
// A cluster of two CTAs (two SMs) computes one tile of 256 columns of dY x 256 columns of
// X of an expert with tcgen05.mma.cta_group::2: CTA r loads 128 columns of each operand,
// the MMAs of the leader (rank 0) read both CTAs' shared memory, and each CTA's tensor
// memory receives its 128 rows of the tile.  Persistent, 7 warps per CTA:
//   warp 0     TMA producer: 96 rows of this CTA's columns per stage (24 + 24 KB) into a
//              4-stage ring guarded by mbarriers.  What a box costs besides its bytes
//              binds: one expert of 8192 rows, N = K = 8192, takes 611 us (1800 TFLOP/s),
//              with 6 stages of 64 rows 688, with 12 of 32 1239; 16 of about 512 rows, N = 16384,
//              K = 5120, 957, 997 and 1656, and 1008 with 3 of 128.
//              Both CTAs' copies complete on the leader's barrier.  Where an expert's rows
//              end inside a step of 16, the rest of that step holds rows of the next expert,
//              or of none, which may be anything: those copies complete on the CTA's own
//              barrier, and then
//   warp 6     writes zeros over them by copies from beyond the operand's last row, which
//              complete on the leader's barrier in their turn.  (Zeroed by the threads, that
//              needs a release at cluster scope, whose fence waits for the epilogue's
//              stores: 16 experts of 509 rows, N = K = 4096, took 232 us that way.)
//   warp 1     (leader) MMA issuer: M = 256, N = 256, 16 rows each, into one of two
//              256-column accumulators.
//   warps 2-5  epilogue: accumulator rows through a staging block to TMA stores (or fp32
//              reductions, for accumulate) that clip at the edges of dW[e].
// An expert without rows has its tiles written as zeros by the epilogue alone.
//
// Where an expert's dW is too few tiles for the device, experts with many rows are cut into
// parts of equal length; a part's tiles go to the workspace in fp32, and a second kernel
// adds an expert's parts in order (one expert of 32768 rows, N = K = 256: 181 us uncut).
//
// A tile costs its store whatever its rows, and its products by its rows: the tiles of
// experts with many rows are bound by the tensor cores, the others by memory.  So that both
// are busy at any time, the experts are ordered by their rows, and each pair works through
// its tiles of that order from both ends at once, a long one in one accumulator and short
// ones in the other (Schedule).
//
// Times in this file are the GPU's, of calls in a graph, those of one comparison of one session.
// Between machines they differ by up to 5%.
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

constexpr int kTile = 256;                // columns of dY and of X of a pair's tile
constexpr int kHalf = kTile / 2;          // ... that one CTA loads, and rows of the tile it stores
constexpr int kBR = 96;                   // rows per stage
constexpr int kBoxCols = 64, kBoxBytes = kBR * 128;
constexpr int kBoxes = kHalf / kBoxCols;  // of each operand
constexpr int kStageBytes = 2 * kBoxes * kBoxBytes;  // 48 KB
constexpr int kStages = 4, kAccBufs = 2;
constexpr int kTmemCols = kAccBufs * kTile;
constexpr int kThreads = 224;
// Experts (or parts) up to which the rank sort is run, whose steps grow with their square.  16384
// rows, Zipf-like, N = 1024, K = 2304, sorted and not: 200 experts 206 and 211 us, 384 366 and 361,
// 500 470 and 454, 1000 932 and 872.
constexpr int kMaxSorted = 384;
constexpr int kPairsGB300 = kNumSmsGB300 / 2;
constexpr int kMinPart = 960;             // rows
constexpr int kWhole = 0xffff;            // the slot of an expert that is not cut
constexpr int kEpiBlockBytes = 32 * 128;  // staging block of an epilogue warp: 32 rows x 128 bytes
// Staging blocks of an epilogue warp: two, which short experts' tiles need to write at 6.3
// TB/s (6.1 with one); one where the tables of experts or parts want the room.
constexpr int kTwoBlocksMaxE = 256;
// Tiles with more rows than this use one block whatever there is: their stores then spread
// over the products of the next tile, whose loads a burst delays.  16 experts of 519
// rows, N = K = 4096: 198.6 us, 218.7 with both blocks.  64 of 100 rows: 349 us with
// both, 400 with one.
constexpr int kBurstRows = 256;

struct Smem {
  static constexpr int stage = 0;
  static constexpr int epi = stage + kStages * kStageBytes;
  // after 4 * blocks staging blocks:
  static constexpr int bars = 0;  // full[S], ready[S], empty[S], tfull[2], tempty[2], drain
  static constexpr int misc = bars + (3 * kStages + 2 * kAccBufs + 1) * 8;
  static constexpr int units = misc + 16;  // off[U + 1], then order, owner and slot [U] in 16 bits
  static constexpr int tail(int blocks) { return epi + 4 * blocks * kEpiBlockBytes; }
  static constexpr int bytes_for(int units_most, bool split, int blocks) {
    return tail(blocks) + units + (units_most + 1) * 4 + units_most * (split ? 6 : 2);
  }
};

// n / d for 0 <= n < 2^31 by one multiplication and a correction: a tile's place costs its
// roles tens of cycles, where 64-bit divisions held tiles of one stage to 0.8 us.
struct Divisor {
  uint32_t d, m;
};
inline Divisor divisor(int d) { return {(uint32_t)d, d == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / (uint32_t)d)}; }
__device__ __forceinline__ int quotient(int n, Divisor v) {
  const uint32_t q = __umulhi((uint32_t)n, v.m);  // n / d or one less
  return (int)(q + ((uint32_t)n - q * v.d >= v.d));
}

constexpr int kGroup = 8;  // tiles along N of a group in the tile order

struct Shape {
  int E, a_max, N, K;
  int units;         // most units: experts, or their parts
  int part;          // rows of a part; 0: experts are not cut
  int mt, kt;        // tiles of an expert along N and K
  Divisor per;       // tiles of an expert
  Divisor band;      // tiles of a group of kGroup along N
  Divisor last;      // tiles along N of an expert's last group
  int accumulate;
  int blocks;        // staging blocks of an epilogue warp
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

// The store is written once and not read here: it leaves L2 first, for the operands to stay
// (64 experts of 16 rows, N = K = 4096: 374 -> 313 us).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
  asm volatile(
      "{\n\t.reg .b64 pol;\n\tcreatepolicy.fractional.L2::evict_first.b64 pol, 1.0;\n\t"
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], pol;\n\t}" ::
          "l"(reinterpret_cast<uint64_t>(map)),
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

// mbar_wait for arrivals that come from the other CTA of the pair too: acquires at cluster scope.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (i == 0) t0 = global_timer_ns();
    if ((i & 63) == 63 && (*abort_flag || global_timer_ns() - t0 > kWaitTimeoutNs)) return false;
  }
}

__device__ __forceinline__ void mma_issue_pair(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Arrive on the barrier at this shared-memory offset in both CTAs of the pair once the
// leader's MMAs issued so far have completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)0x3)
      : "memory");
}

// TMA load into this CTA's shared memory, completing on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int c0,
                                                 int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}

// Boxes of one CTA's half of an operand with `cols` columns left.  Boxes past the columns are
// not loaded: what they leave stale reaches only accumulator rows and columns that are not stored.
__device__ __forceinline__ int boxes(int cols) { return max(0, min(kBoxes, (cols + kBoxCols - 1) / kBoxCols)); }

// Whether a unit's last block, of `left` rows, ends inside a step of 16, and the rows that
// are zeroed behind it: 16, in one copy, where they fit the box (a copy costs as much time
// as it takes to issue, whatever its rows), else to the end of the box.
__device__ __forceinline__ bool ragged(int left) { return (left & 15) != 0; }
__device__ __forceinline__ int zero_rows(int left) { return min(16, kBR - left); }
constexpr int kHeights = 5;  // copies of 1, 2, 4, 8 and 16 rows
// Of a block that few rows are left for, lower boxes are loaded (w13 of 16 experts from 8-bit
// rows: 972 us with whole ones, 957).
constexpr int kLoadHeights = 4;  // 16, 32, 64 and 96 rows
__host__ __device__ constexpr int load_rows(int h) { return h == 3 ? kBR : 16 << h; }
__device__ __forceinline__ int load_height(int left) { return left > 64 ? 3 : left > 32 ? 2 : left > 16 ? 1 : 0; }
struct Maps {
  CUtensorMap dy[kLoadHeights], x[kLoadHeights];
  CUtensorMap zero[kHeights];
  CUtensorMap dw, part;
};

// Arrival on the leader's barrier by a warp that has read its accumulator rows (tcgen05.wait::ld):
// nothing it wrote has to be seen, so no release at cluster scope, whose fence would wait.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The units of work: an expert's rows, or a part of them.  Unit u holds the rows from
// off[u] to off[u + 1] of expert owner[u]; slot[u]: where its part goes (kWhole: to dW).
struct Units {
  int* off;
  uint16_t* order;  // by descending rows
  uint16_t* owner;
  uint16_t* slot;
  int n, total;     // units; tiles of them all
};

struct Tile {
  int unit, n0, k0, row0, rows;
};

// Tile `tile` in the order of the units' ranks.  A unit's tiles come in groups of kGroup
// along N, N innermost, so that the pairs running together read few columns of either operand.
__device__ __forceinline__ Tile locate(const Shape& p, int tile, const Units& units) {
  Tile t;
  const int rank = quotient(tile, p.per);
  t.unit = units.order[rank];
  const int local = tile - rank * (int)p.per.d;
  const int group = quotient(local, p.band), in = local - group * (int)p.band.d;
  const bool whole = (group + 1) * kGroup <= p.mt;
  const int k = whole ? in / kGroup : quotient(in, p.last);
  const int n = in - k * (whole ? kGroup : (int)p.last.d);
  t.n0 = (group * kGroup + n) * kTile;
  t.k0 = k * kTile;
  t.row0 = units.off[t.unit];
  t.rows = units.off[t.unit + 1] - t.row0;
  return t;
}

// A pair's work in order, the same for all of its roles.  Its tiles are every pairs-th of
// the order of ranks, most rows first; accumulator 0 takes them from the front and
// accumulator 1 from the back until they meet.  A tile from the back is multiplied whole;
// of the one from the front kChunk blocks follow each time, the time that storing a tile
// takes, or all that is left when that is no more than twice as many.  Tiles of one length
// so alternate between the accumulators.  On 128 experts of Zipf-like load, N = 7168,
// K = 2048, taking whole tiles from the two ends in turn took 990 us, this 976.
constexpr int kChunk = 4;

struct Schedule {
  int pair, pairs, front, back;  // the next tile of this pair from either end
  int done;                      // blocks multiplied of the front's tile, 0: none is under way
  bool short_turn;
  Tile t;                        // the front's tile

  __device__ Schedule(const Units& units, int pair_, int pairs_)
      : pair(pair_), pairs(pairs_), front(0), back(units.total > pair_ ? (units.total - 1 - pair_) / pairs_ : -1),
        done(0), short_turn(true) {}
};

// Blocks first .. first + count - 1 of a tile of `blocks` blocks, in accumulator acc.
struct Chunk {
  Tile t;
  int acc, first, count, blocks;
};

__device__ __forceinline__ bool next_chunk(Schedule& w, const Shape& p, const Units& units, Chunk* c) {
  const bool take_back = w.short_turn && w.front <= w.back;
  w.short_turn = !take_back;
  if (take_back) {
    c->t = locate(p, w.pair + w.back * w.pairs, units);
    --w.back;
    c->acc = 1;
    c->first = 0;
    c->count = c->blocks = (c->t.rows + kBR - 1) / kBR;
    return true;
  }
  if (w.done == 0) {
    if (w.front > w.back) return false;
    w.t = locate(p, w.pair + w.front * w.pairs, units);
    ++w.front;
  }
  c->t = w.t;
  c->acc = 0;
  c->blocks = (w.t.rows + kBR - 1) / kBR;
  c->first = w.done;
  const int left = c->blocks - w.done;
  c->count = left <= 2 * kChunk || w.front > w.back ? left : kChunk;
  w.done += c->count;
  if (w.done == c->blocks) w.done = 0;
  return true;
}

// 64 consecutive fp32 accumulator columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t* r) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t* v = r + 32 * h;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr + 32 * h));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Stores a staging block's 32 rows x 128 bytes (o[q]: piece q of this lane's row) as columns
// from c on, rows from row on of matrix `at` of map; add: to what is there (fp32).
__device__ __forceinline__ void store_block(const Shape& p, const Tile& t, const uint4* o, int c, int row, int lane,
                                            uint8_t* stage, int* blk, const CUtensorMap* map, int at, bool add) {
  if (lane == 0) {  // the store that last used this block has read it
    if (p.blocks == 1 || t.rows > kBurstRows) bulk_wait_group_read0();
    else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
  }
  __syncwarp();
  uint8_t* b = stage + *blk * kEpiBlockBytes;
#pragma unroll
  for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(b + lane * 128 + ((q ^ (lane & 7)) << 4)) = o[q];
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    if (add) tma_add_3d(map, smem_u32(b), t.k0 + c, row, at);
    else tma_store_3d(map, smem_u32(b), t.k0 + c, row, at);
    bulk_commit_group();
  }
  if (++*blk == p.blocks) *blk = 0;
}

// One epilogue warp's rows of a tile: row (its first) + lane, to matrix `at` of map.  zero:
// the tile of an expert without rows.  release() gives the accumulator back: for bf16 once
// all of it is in registers as pairs, before the stores, which take most of the time (128
// experts of Zipf-like load, N = 7168, K = 2048: 987 us when it came after them).
template <bool F32, typename Release>
__device__ __forceinline__ void store_tile(const Shape& p, const Tile& t, int row, int lane, uint32_t tbase, bool zero,
                                           uint8_t* stage, int* blk, const CUtensorMap* map, int at, bool add,
                                           Release release) {
  if (row >= p.N) {
    release();
    return;
  }
  const int cols = min(kTile, p.K - t.k0);
  if constexpr (F32) {
#pragma unroll 1
    for (int c = 0; c < cols; c += 64) {
      uint32_t v[64] = {};
      if (!zero) tmem_ld64(tbase + c, v);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (c + 32 * h < cols)
          store_block(p, t, reinterpret_cast<const uint4*>(v + 32 * h), c + 32 * h, row, lane, stage, blk, map, at, add);
    }
    release();
  } else {
    uint4 w[kTile / 64][8] = {};
    if (!zero) {
#pragma unroll
      for (int j = 0; j < kTile / 64; ++j)
        if (64 * j < cols) {
          uint32_t v[64];
          tmem_ld64(tbase + 64 * j, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) w[j][q] = f32_to_bf16x8(reinterpret_cast<const float*>(v) + 8 * q);
        }
    }
    release();
#pragma unroll
    for (int j = 0; j < kTile / 64; ++j)
      if (64 * j < cols) store_block(p, t, w[j], 64 * j, row, lane, stage, blk, map, at, false);
  }
}

// cut (SPLIT): for the join, the number of experts that are cut, then of each its number,
// first slot and number of parts.
template <bool F32, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    weight_grad_kernel(const __grid_constant__ Maps maps, const int32_t* __restrict__ counts, const Shape p, int* cut,
                       unsigned int* err) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank() & 1u;
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  uint8_t* tail = smem + Smem::tail(p.blocks);
  uint64_t* bars = reinterpret_cast<uint64_t*>(tail + Smem::bars);
  auto bar_full = [&](int s) { return smem_u32(&bars[s]); };               // this CTA's copies of a ragged end
  auto bar_ready = [&](int s) { return smem_u32(&bars[kStages + s]); };    // leader's: both CTAs' stages are whole
  auto bar_empty = [&](int s) { return smem_u32(&bars[2 * kStages + s]); };
  auto bar_tfull = [&](int b) { return smem_u32(&bars[3 * kStages + b]); };
  auto bar_tempty = [&](int b) { return smem_u32(&bars[3 * kStages + kAccBufs + b]); };
  const uint32_t bar_drain = smem_u32(&bars[3 * kStages + 2 * kAccBufs]);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tail + Smem::misc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tail + Smem::misc + 4);
  int* s_units = reinterpret_cast<int*>(tail + Smem::misc + 8);
  Units units;
  units.off = reinterpret_cast<int*>(tail + Smem::units);
  units.order = reinterpret_cast<uint16_t*>(units.off + p.units + 1);
  units.owner = units.order + p.units;
  units.slot = units.owner + p.units;

  if (SPLIT) pdl_launch_dependents();  // the join waits for this grid's end
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_ready(s), 2);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < kAccBufs; ++b) {
      mbar_init(bar_tfull(b), 1);
      mbar_init(bar_tempty(b), 8);  // 4 epilogue warps in each CTA of the pair
    }
    mbar_init(bar_drain, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tma_prefetch_desc(&maps.dy[kLoadHeights - 1]);
    tma_prefetch_desc(&maps.x[kLoadHeights - 1]);
    tma_prefetch_desc(&maps.dw);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 2) {
    // the units' row offsets: a warp-wide scan of the counts, cut at a_max (64-bit: bad counts may add up
    // past 31 bits)
    int64_t run = 0;
    int first = 0, slot = 0, ncut = 0;  // the next unit and slot; experts cut
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
      const int row0 = (int)min(run + incl - c, (int64_t)p.a_max), row1 = (int)min(run + incl, (int64_t)p.a_max);
      if constexpr (SPLIT) {
        const int parts = max(1, (row1 - row0 + p.part - 1) / p.part);
        const int slots = parts > 1 ? parts : 0;
        int nu = e < p.E ? parts : 0, ns = e < p.E ? slots : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, nu, o), v = __shfl_up_sync(0xffffffffu, ns, o);
          if (lane >= o) {
            nu += u;
            ns += v;
          }
        }
        if (e < p.E) {
          const int u0 = first + nu - parts, s0 = slot + ns - slots;
          for (int k = 0; k < parts; ++k) {
            units.off[u0 + k] = row0 + k * p.part;
            units.owner[u0 + k] = (uint16_t)e;
            units.slot[u0 + k] = (uint16_t)(slots ? s0 + k : kWhole);
          }
        }
        const uint32_t more = __ballot_sync(0xffffffffu, e < p.E && slots > 0);
        if (blockIdx.x == 0 && e < p.E && slots > 0) {
          int* entry = cut + 1 + 3 * (ncut + __popc(more & ((1u << lane) - 1u)));
          entry[0] = e;
          entry[1] = slot + ns - slots;
          entry[2] = slots;
        }
        ncut += __popc(more);
        first += __shfl_sync(0xffffffffu, nu, 31);
        slot += __shfl_sync(0xffffffffu, ns, 31);
      } else {
        if (e < p.E) units.off[e] = row0;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      const int n = SPLIT ? first : p.E;
      if (SPLIT && blockIdx.x == 0) cut[0] = ncut;
      units.off[n] = (int)min(run, (int64_t)p.a_max);
      *s_units = n;
      if (run > p.a_max) bad = true;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) flag_error(err, MOE_DEVERR_BAD_COUNT);
  }
  __syncthreads();
  units.n = *s_units;
  units.total = units.n * (int)p.per.d;
  // the units by descending rows (equal ones by number): each one's rank by counting
  for (int u = threadIdx.x; u < units.n; u += kThreads) {
    int at = u;
    if (units.n <= kMaxSorted) {
      const int mine = units.off[u + 1] - units.off[u];
      at = 0;
      for (int i = 0; i < units.n; ++i) {
        const int other = units.off[i + 1] - units.off[i];
        at += other > mine || (other == mine && i < u);
      }
    }
    units.order[at] = (uint16_t)u;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any arrival from the other
  tc_fence_after();

  const uint32_t tmem_base = *s_tmem;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      const uint32_t ready0 = map_to_rank(bar_ready(0), 0);
      int s = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0, issued_parity = 0;
      bool ok = true;
      Schedule work(units, pair, pairs);
      Chunk c;
      while (ok && next_chunk(work, p, units, &c)) {
        const Tile& t = c.t;
        const int n0 = t.n0 + (int)rank * kHalf, k0 = t.k0 + (int)rank * kHalf;
        const int na = boxes(p.N - n0), nb = boxes(p.K - k0);
        const int both = boxes(p.N - t.n0) + boxes(p.N - t.n0 - kHalf) + boxes(p.K - t.k0) + boxes(p.K - t.k0 - kHalf);
        for (int r = c.first * kBR; r < min((c.first + c.count) * kBR, t.rows); r += kBR) {
          if (!mbar_wait(bar_empty(s), phase ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          const uint32_t dst = sbase + Smem::stage + s * kStageBytes;
          const int left = t.rows - r;
          const uint32_t bytes = 128u * (uint32_t)load_rows(load_height(left));  // of a box
          const bool end = left < kBR && ragged(left);
          uint32_t bar = ready0 + (uint32_t)(s * 8);
          if (end) {
            if (leader) {  // the zeros of both CTAs
              mbar_arrive_expect_tx(bar_ready(s), (uint32_t)(both * zero_rows(left)) * 128);
              mbar_arrive(bar_ready(s));
            }
            if (na + nb > 0) mbar_arrive_expect_tx(bar_full(s), (uint32_t)(na + nb) * bytes);
            bar = map_to_rank(bar_full(s), rank);  // this CTA's own
          } else if (leader) {
            mbar_arrive_expect_tx(bar_ready(s), (uint32_t)both * bytes);
            mbar_arrive(bar_ready(s));
          }
          // (each height's loads by themselves: a map chosen by an index slows all of them)
          auto load = [&](const CUtensorMap* dy, const CUtensorMap* x) {
            for (int b = 0; b < na; ++b)
              tma_load_2d_pair(dst + b * kBoxBytes, dy, bar, n0 + b * kBoxCols, t.row0 + r);
            for (int b = 0; b < nb; ++b)
              tma_load_2d_pair(dst + (kBoxes + b) * kBoxBytes, x, bar, k0 + b * kBoxCols, t.row0 + r);
          };
          if (left > 64) load(&maps.dy[3], &maps.x[3]);
          else if (left > 32) load(&maps.dy[2], &maps.x[2]);
          else if (left > 16) load(&maps.dy[1], &maps.x[1]);
          else load(&maps.dy[0], &maps.x[0]);
          issued_mask |= 1u << s;
          issued_parity = (issued_parity & ~(1u << s)) | (phase << s);
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (ok) {
        // every stage this CTA filled has been read by the pair's MMAs before it exits
        for (int b = 0; b < kStages; ++b)
          if ((issued_mask >> b) & 1u && !mbar_wait(bar_empty(b), (issued_parity >> b) & 1u, s_abort)) ok = false;
      }
      if (!ok) {
        flag_error(err, MOE_DEVERR_TIMEOUT);
        *s_abort = 1;
        const uint64_t t0 = global_timer_ns();  // copies in flight complete on either barrier: give them time to land
        while (global_timer_ns() - t0 < kDrainTimeoutNs) {
        }
      }
    }
  } else if (warp == 6) {
    // ------------------------------------------------------- ragged ends
    const uint32_t ready0 = map_to_rank(bar_ready(0), 0);
    if (lane == 0) {
      uint32_t parity = 0;   // of each stage's next use of its full barrier
      int s = 0;             // the stage of this chunk's first block
      bool ok = true;
      Schedule work(units, pair, pairs);
      Chunk c;
      while (ok && next_chunk(work, p, units, &c)) {
        const Tile& t = c.t;
        if (c.count == 0) continue;
        const int mine = (s + c.count - 1) % kStages, left = t.rows - (c.blocks - 1) * kBR;
        s = mine + 1 == kStages ? 0 : mine + 1;
        if (c.first + c.count < c.blocks || !ragged(left)) continue;
        const int na = boxes(p.N - t.n0 - (int)rank * kHalf), nb = boxes(p.K - t.k0 - (int)rank * kHalf);
        if (na + nb == 0) continue;  // (else the stage is not used again before its zeros)
        ok = mbar_wait(bar_full(mine), (parity >> mine) & 1u, s_abort);
        if (!ok) break;
        parity ^= 1u << mine;
        const uint32_t st = sbase + Smem::stage + mine * kStageBytes, ready = ready0 + (uint32_t)(mine * 8);
        for (int b = 0; b < 2 * kBoxes; ++b) {
          if (b < kBoxes ? b >= na : b - kBoxes >= nb) continue;
          // 128-byte lines: the operand's swizzle stays inside them
          uint32_t at = st + b * kBoxBytes + left * 128;
          for (int n = zero_rows(left); n > 0; n &= n - 1) {
            const int h = __ffs(n) - 1;
            tma_load_2d_pair(at, &maps.zero[h], ready, 0, p.a_max);
            at += 128 << h;
          }
        }
      }
      if (!ok) {
        flag_error(err, MOE_DEVERR_TIMEOUT);
        *s_abort = 1;
        const uint64_t t0 = global_timer_ns();  // copies in flight complete on the leader's barrier: let them land
        while (global_timer_ns() - t0 < kDrainTimeoutNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA (leader)
    if (lane == 0 && leader) {
      // fp32 accumulate, bf16 operands, both MN-major
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                             ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
      int s = 0;
      uint32_t phase = 0;
      uint32_t acc_parity = 0;  // of each accumulator's next use
      bool ok = true, issued_any = false;
      Schedule work(units, pair, pairs);
      Chunk c;
      while (ok && next_chunk(work, p, units, &c)) {
        const Tile& t = c.t;
        if (c.count == 0) continue;
        if (c.first == 0) {
          if (!mbar_wait_cluster(bar_tempty(c.acc), ((acc_parity >> c.acc) & 1u) ^ 1u, s_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        const uint32_t d = tmem_base + (uint32_t)(c.acc * kTile);
        for (int r = c.first * kBR; r < min((c.first + c.count) * kBR, t.rows); r += kBR) {
          if (!mbar_wait_cluster(bar_ready(s), phase, s_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = sbase + Smem::stage + s * kStageBytes, b = a + kBoxes * kBoxBytes;
          const int steps = (min(t.rows - r, kBR) + 15) / 16;
          for (int k = 0; k < steps; ++k)
            mma_issue_pair(d, desc_mn(a + k * 2048), desc_mn(b + k * 2048), idesc, (r | k) != 0);
          mma_commit_pair(bar_empty(s));
          issued_any = true;
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (c.first + c.count == c.blocks) {
          mma_commit_pair(bar_tfull(c.acc));
          acc_parity ^= 1u << c.acc;
        }
      }
      if (!ok) {
        flag_error(err, MOE_DEVERR_TIMEOUT);
        *s_abort = 1;
        if (issued_any) {  // the MMAs in flight finish before tensor memory is freed
          mma_commit_pair(bar_drain);
          mbar_wait(bar_drain, 0, nullptr, kDrainTimeoutNs);
        }
      }
    }
  } else {
    // ------------------------------------------------- epilogue (both CTAs)
    const int sub = warp & 3;  // TMEM lane quarter this warp may access
    uint8_t* stage = smem + Smem::epi + (warp - 2) * p.blocks * kEpiBlockBytes;
    const uint32_t tempty0 = map_to_rank(bar_tempty(0), 0);
    uint32_t acc_parity = 0;
    int blk = 0;
    Schedule work(units, pair, pairs);
    Chunk c;
    while (next_chunk(work, p, units, &c)) {
      if (c.first + c.count < c.blocks) continue;
      const int row = c.t.n0 + (int)rank * kHalf + 32 * sub;
      const int slot = SPLIT ? units.slot[c.t.unit] : kWhole;
      const int expert = SPLIT ? units.owner[c.t.unit] : c.t.unit;
      if (c.t.rows == 0) {
        if (!p.accumulate) store_tile<F32>(p, c.t, row, lane, 0, true, stage, &blk, &maps.dw, expert, false, [] {});
        continue;
      }
      if (!warp_wait(bar_tfull(c.acc), (acc_parity >> c.acc) & 1u, s_abort)) {
        if (lane == 0) flag_error(err, MOE_DEVERR_TIMEOUT);
        *s_abort = 1;
        break;
      }
      acc_parity ^= 1u << c.acc;
      tc_fence_after();
      const uint32_t tbase = tmem_base + ((uint32_t)(sub * 32) << 16) + (uint32_t)(c.acc * kTile);
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0 + (uint32_t)(c.acc * 8));
      };
      if (SPLIT && slot != kWhole)
        store_tile<true>(p, c.t, row, lane, tbase, false, stage, &blk, &maps.part, slot, false, release);
      else
        store_tile<F32>(p, c.t, row, lane, tbase, false, stage, &blk, &maps.dw, expert, p.accumulate, release);
    }
    if (lane == 0) bulk_wait_group0();  // this warp's stores are complete before the block exits
  }

  // the pair meets, then frees its tensor memory together
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
}

// dW of the experts that were cut.  32 float4 columns a block, 8 threads each, which add every
// eighth part in order and are then added in order.  n4: float4s of an expert's dW.
template <bool F32>
__global__ void __launch_bounds__(256) join_parts_kernel(const float4* __restrict__ parts,
                                                         const int* __restrict__ cut, int64_t n4, bool accumulate,
                                                         void* dw) {
  __shared__ float4 s[8][32];
  pdl_wait();
  const int c = threadIdx.x & 31, l = threadIdx.x >> 5;
  const int64_t per = n4 / 32, work = cut[0] * per;  // (n4 is a multiple of 64)
  for (int64_t u = blockIdx.x; u < work; u += gridDim.x) {
    const int* entry = cut + 1 + 3 * (u / per);
    const int expert = entry[0], slot = entry[1], count = entry[2];
    const int64_t i = u % per * 32 + c;
    const float4* p = parts + slot * n4 + i;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kAtOnce = 4;  // loads under way together
    for (int k = l; k < count; k += 8 * kAtOnce) {
      float4 a[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        a[j] = k + 8 * j < count ? __ldcs(p + (k + 8 * j) * n4) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) v = make_float4(v.x + a[j].x, v.y + a[j].y, v.z + a[j].z, v.w + a[j].w);
    }
    s[l][c] = v;
    __syncthreads();
    if (l == 0) {
      const int most = count < 8 ? count : 8;
      for (int k = 1; k < most; ++k) {
        const float4 b = s[k][c];
        v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
      }
      const int64_t at = expert * n4 + i;
      if (F32) {
        float4* o = static_cast<float4*>(dw) + at;
        if (accumulate) {
          const float4 b = *o;
          v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
        }
        *o = v;
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        static_cast<uint2*>(dw)[at] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- host

int64_t tiles_of(int n) { return (n + kTile - 1) / kTile; }

// Rows of a part, 0: experts are not cut.  A part for each pair when one expert has all the
// rows; dW of a tile for each pair needs none.
int part_rows(int a_max, int N, int K) {
  const int64_t tiles = tiles_of(N) * tiles_of(K);
  if (tiles >= kPairsGB300) return 0;
  int64_t rows = (a_max * tiles + kPairsGB300 - 1) / kPairsGB300;
  rows = (rows + kBR - 1) / kBR * kBR;
  if (rows < kMinPart) rows = kMinPart;
  return rows >= a_max ? 0 : (int)rows;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
size_t unpacked_bytes(int a_max, int K) { return up256((size_t)a_max * K * 2); }
// Slots: an expert that is cut has more than one part, of which all but the last are whole.
int64_t most_slots(int a_max, int part) { return 2 * (int64_t)a_max / part; }
size_t cut_bytes(int E) { return up256((size_t)(1 + 3 * E) * sizeof(int)); }

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

// Boxes of `rows` rows x 128 bytes of dY without a swizzle: read past its last row, they are
// zeros.  (N columns of 2 bytes; N may be below the box's 64.)
bool make_zero_map(CUtensorMap* map, const void* dy, int a_max, int N, int rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)a_max};
  cuuint64_t strides[1] = {(cuuint64_t)N * 2};
  cuuint32_t box[2] = {kBoxCols, (cuuint32_t)rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(dy), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t weight_grad_workspace_bytes(int E, int a_max, int N, int K, bool packed) {
  size_t n = packed ? unpacked_bytes(a_max, K) : 0;
  if (const int part = part_rows(a_max, N, K))
    n += cut_bytes(E) + (size_t)most_slots(a_max, part) * N * K * sizeof(float);
  return n;
}

cudaError_t launch_weight_grad(const WeightGradArgs& g, cudaStream_t s) {
  const void* x = g.x;
  char* ws = static_cast<char*>(g.ws);
  if (g.exponents && g.a_max > 0) {
    CheckpointArgs c{};
    c.a = g.a_max;
    c.W = g.K;
    c.codes = const_cast<void*>(g.x);
    c.exponents = const_cast<uint8_t*>(g.exponents);
    c.out = ws;
    c.sum_counts = g.counts;
    c.E = g.E;
    c.err = g.err;
    cudaError_t e = launch_checkpoint_unpack(c, s);
    if (e != cudaSuccess) return e;
    x = ws;
    ws += unpacked_bytes(g.a_max, g.K);
  }
  const int64_t mt = tiles_of(g.N), kt = tiles_of(g.K);
  const bool f32 = g.dw_dtype == MOE_DTYPE_F32;
  Shape p{};
  p.E = g.E;
  p.a_max = g.a_max;
  p.N = g.N;
  p.K = g.K;
  p.part = part_rows(g.a_max, g.N, g.K);
  p.units = g.E + (p.part ? g.a_max / p.part : 0);
  const int64_t tiles = p.units * mt * kt;  // at most
  if (tiles > INT32_MAX / 2) return cudaErrorNotSupported;
  p.mt = (int)mt;
  p.kt = (int)kt;
  p.per = divisor((int)(mt * kt));
  p.band = divisor((int)(kGroup * kt));
  p.last = divisor(mt % kGroup ? (int)(mt % kGroup) : kGroup);
  p.accumulate = g.accumulate;
  p.blocks = !p.part && g.E <= kTwoBlocksMaxE ? 2 : 1;
  int* cut = reinterpret_cast<int*>(ws);
  float* parts = reinterpret_cast<float*>(ws + cut_bytes(g.E));
  Maps maps;
  if (!make_dw_map(&maps.dw, g.dw, g.E, g.N, g.K, f32)) return cudaErrorInvalidValue;
  maps.part = maps.dw;  // without parts none are stored, without rows nothing is loaded
  if (p.part && !make_dw_map(&maps.part, parts, (int)most_slots(g.a_max, p.part), g.N, g.K, true))
    return cudaErrorInvalidValue;
  for (int h = 0; h < kLoadHeights; ++h) {
    maps.dy[h] = maps.x[h] = maps.dw;
    if (g.a_max > 0 && (!make_map_sw128(&maps.dy[h], g.dy, g.a_max, g.N, false, load_rows(h)) ||
                        !make_map_sw128(&maps.x[h], x, g.a_max, g.K, false, load_rows(h))))
      return cudaErrorInvalidValue;
  }
  for (int h = 0; h < kHeights; ++h) {
    maps.zero[h] = maps.dw;
    if (g.a_max > 0 && !make_zero_map(&maps.zero[h], g.dy, g.a_max, g.N, 1 << h)) return cudaErrorInvalidValue;
  }
  const int smem = Smem::bytes_for(p.units, p.part != 0, p.blocks) + 1024;
  auto kern = p.part ? (f32 ? weight_grad_kernel<true, true> : weight_grad_kernel<false, true>)
                     : (f32 ? weight_grad_kernel<true, false> : weight_grad_kernel<false, false>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(device_sm_count() / 2 * 2);
  int pairs = 0;
  e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
  if (e != cudaSuccess) return e;
  if (pairs < 1) return cudaErrorNotSupported;
  if (tiles < pairs) pairs = (int)tiles;
  cfg.gridDim = dim3(2 * pairs);
  e = cudaLaunchKernelEx(&cfg, kern, maps, g.counts, p, cut, g.err);
  if (e != cudaSuccess) return e;
  if (!p.part) return cudaGetLastError();
  const int64_t n4 = (int64_t)g.N * g.K / 4, want = n4 / 32 * g.E, most = 8 * (int64_t)device_sm_count();
  cudaLaunchConfig_t join = {};
  join.gridDim = dim3((unsigned)(want < most ? want : most));
  join.blockDim = dim3(256);
  join.stream = s;
  cudaLaunchAttribute pdl[1] = {pdl_attribute()};
  join.attrs = pdl;
  join.numAttrs = 1;
  auto jk = f32 ? join_parts_kernel<true> : join_parts_kernel<false>;
  e = cudaLaunchKernelEx(&join, jk, reinterpret_cast<const float4*>(parts), (const int*)cut, n4, g.accumulate,
                         g.dw);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace moe
