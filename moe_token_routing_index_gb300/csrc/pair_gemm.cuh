// A persistent GEMM on pairs of SMs for 16-bit operands, whose problem (tile list, operand
// boxes, epilogue) is a policy class: the gated feed-forward block and the orthogonalisation
// share it.
//
// A cluster of two CTAs computes a tile D[256, n] = A[256, k] B[n, k]^T, n a multiple of 32 up
// to 256, with tcgen05.mma.cta_group::2 (fp32 accumulation).  CTA r loads 128 rows of A and
// n / 2 of B, the MMAs of the leader (rank 0) read both CTAs' shared memory, and each CTA's
// tensor memory receives its 128 rows of the tile: one lane per row, one column per row of B.
// An operand lies K-major (its rows contiguous along the reduction: boxes of 64 k) or MN-major
// (rows of the reduction, contiguous along the tile: boxes of 64 columns).  10 warps:
//   warp 0     TMA producer of this CTA's halves, into a ring of stages of kBK of the
//              reduction; both CTAs' copies complete on the leader's barrier
//   warp 1     (leader) MMA issuer, into one of two 256-column accumulators
//   warps 2-9  the policy's epilogue: two warps for the 32 lanes of a quarter, which take its
//              columns by turns of kChunk
// Results go from registers to memory, without staging: where a column's lanes are contiguous there,
// neighbouring lanes deal two columns out among them and a warp stores two columns of 64 bytes at
// once; where a lane's columns are contiguous, a lane stores the 32 bytes of a chunk.
//
// 256 x 256 x 64 of products, 512 cycles, need 32 KB a CTA: 18 TB/s in all at 2390 TFLOP/s, by arithmetic.
// The main loop without an epilogue (an early form of it, one run): operands of zeros from L2, K = 4096, 2390
// TFLOP/s, at n = 192 2370, at 128 1760; random operands, K = 5120, one streamed from HBM and used twice, 2035,
// the same with zeros 2310.  M = 256 on pairs because a CTA by itself needs 48 KB for the same products.
//
// Every wait is bounded; on expiry the kernel records MOE_DEVERR_TIMEOUT, all roles stop,
// copies and MMAs in flight are drained, and tensor memory is freed.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace moe {
namespace pg {

using namespace tc;

constexpr int kTileM = 256, kHalfM = 128, kMaxN = 256;
// Of the reduction per stage.  (Stages twice as long, half as many: 128 experts of 344 rows, D = 4096,
// H = 1536, forward 950 us instead of 784.  Boxes brought into L2 8 stages ahead: 929, as the way from L2
// to the SMs is what binds next to DRAM.)
constexpr int kBK = 64;
constexpr int kOperandBytes = 128 * kBK * 2;             // of a CTA's half of A; room for its half of B
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kAccBufs = 2;
constexpr int kTmemCols = kAccBufs * kMaxN;
constexpr int kEpiWarps = 8, kEpiGroups = kEpiWarps / 4;
constexpr int kChunk = 16;                               // columns of an epilogue's step
constexpr int kThreads = 64 + 32 * kEpiWarps;
// Boxes of a K-major B, of 16, 32, ... 128 rows: a CTA loads its n / 2 rows and no more.  (With boxes of
// 16, 32, 64 and 128 rows, 128 experts of 344 rows loaded a third more of them than they used.)
constexpr int kHeights = 8;
__host__ __device__ constexpr int box_rows(int h) { return 16 * (h + 1); }
constexpr int kBoxBytes = 64 * 128;                      // of an MN-major box: 64 columns x kBK rows

template <int STAGES>
struct Smem {
  static constexpr int stage = 0;
  static constexpr int bars = stage + STAGES * kStageBytes;  // full[S], empty[S], tfull[2], tempty[2], drain
  static constexpr int misc = bars + (2 * STAGES + 2 * kAccBufs + 1) * 8;
  static constexpr int extra = (misc + 16 + 15) / 16 * 16;   // the policy's
  static constexpr int bytes(int more) { return extra + more + 1024; }  // (the base is aligned to 1024)
};
constexpr int kSmemMax = 227 * 1024;

// Shared-memory descriptor of an MN-major operand, 128B swizzle: 64-column blocks one box
// apart, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((64 * kBK * 2) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// The descriptor of an operand's half at addr, and how far on that of the 16 reduction steps from 16 * kk lies.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return MN ? desc_mn(addr) : smem_desc_sw128(addr);
}
template <bool MN>
__device__ __forceinline__ constexpr uint32_t operand_step(int kk) {
  return (MN ? kk * 2048                                      // 16 rows of 128 bytes
             : (kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;  // 64 k of 128 rows a box
}

// One lane of the (whole) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

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

// Arrive on the barrier at this shared-memory offset in both CTAs once the leader's MMAs have completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)0x3)
      : "memory");
}

// Arrival on the leader's barrier by a warp that has read its accumulator (tcgen05.wait::ld):
// nothing it wrote has to be seen, so no release at cluster scope, whose fence would wait.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// TMA loads into this CTA's shared memory that complete on the leader's barrier.
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                        int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// 128 rows of a K-major operand half, or 128 columns of an MN-major one, at reduction index k
// of matrix `at` of a 3-D map [at][rows][columns]: kBK of the reduction.
template <bool MN>
__device__ __forceinline__ void load_half(uint32_t dst, const CUtensorMap* map, uint32_t bar, int k, int row, int at) {
#pragma unroll
  for (int h = 0; h < (MN ? 2 : kBK / 64); ++h) {
    if (MN) load_3d(dst + h * kBoxBytes * (kBK / 64), map, bar, row + 64 * h, k, at);
    else load_3d(dst + h * 128 * 128, map, bar, k + 64 * h, row, at);
  }
}

// kChunk consecutive accumulator columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld_chunk(uint32_t taddr, float* v) {
  uint32_t r[kChunk];
  static_assert(kChunk == 16, "one load a chunk");
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kChunk; ++i) v[i] = __uint_as_float(r[i]);
}

// Columns 2j and 2j + 1 of two neighbouring lanes, dealt out so that the even lane has both lanes'
// column 2j and the odd one both lanes' column 2j + 1 (the even lane's value in x).
__device__ __forceinline__ float2 deal(const float* v, int j, bool odd) {
  const float other = __shfl_xor_sync(0xffffffffu, odd ? v[2 * j] : v[2 * j + 1], 1);
  return odd ? make_float2(other, v[2 * j + 1]) : make_float2(v[2 * j], other);
}

// An epilogue over `rows` columns of a tile: load(c, s) brings what column chunk c needs from memory
// into s, two chunks ahead (the first two before the accumulator is waited for); use(c, s, v)
// takes it with the accumulator's columns c .. c + kChunk - 1.
template <class Source, class Load, class Use, class Wait, class Release>
__device__ __forceinline__ void by_chunks(int rows, int group, uint32_t tbase, Load load, Use use, Wait wait,
                                          Release release) {
  constexpr int kStep = kEpiGroups * kChunk;
  int c = group * kChunk;
  Source s{}, next{};
  if (c < rows) load(c, s);
  if (c + kStep < rows) load(c + kStep, next);
  if (!wait()) return;
  while (c < rows) {
    float v[kChunk];
    tmem_ld_chunk(tbase + c, v);
    Source later{};
    if (c + 2 * kStep < rows) load(c + 2 * kStep, later);
    if (c + kStep >= rows) release();
    use(c, s, v);
    s = next;
    next = later;
    c += kStep;
  }
  if (group * kChunk >= rows) release();
}
struct NoSource {};

// A policy P has
//   kAMN, kBMN                       an operand is MN-major
//   kF16                             fp16 operands (else bf16)
//   Params                           kernel parameter, with unsigned int* err
//   Tile                             with int n (rows of B, a multiple of 32) and int k > 0, the reduction's length
//   setup(p, tables) -> int          the number of tiles, called by all threads (it may fill the tables)
//   tile(p, tables, i) -> Tile
//   narrow(t, part, parts)           makes t its part-th of `parts` parts along B (n = 0: there is none)
//   stage_bytes(p, t)                what both CTAs' loads of a stage complete
//   load(p, t, rank, block, a, b, bar)
//   epilogue(p, t, rank, sub, group, lane, tbase, wait, release)
//     wait() -> bool: the accumulator is whole (false: give up); release(): it has been read.
//     group: which of the quarter's two warps

// A pair's tiles, every pairs-th, the same for all of its roles.  Of `tiles` tiles the last round, which not
// every pair has one of, is cut into `parts` parts along B, as many as give each pair at most one: 640 tiles
// of 256 rows are 8 rounds and 32 tiles of 128 rows on either of 64 pairs, where 9 rounds were; a few tiles in
// all become so many smaller ones.  It is for those: 517 rows of 5 experts, D = 272, H = 208, gradient, 18.6 us
// against 24.9 uncut.  8192 rows of 16 experts, D = 5120, H = 8192, gradient, 1259 and 1281, 128 experts of 344
// rows 1211 and 1200, both within the spread of their runs; 64 rows, D = 256, H = 512, forward, lose: 15.1
// and 14.6.
template <class P>
struct Walk {
  const typename P::Params& p;
  const int* tables;
  int pair, pairs, whole, parts, count, step = 0;
  __device__ __forceinline__ Walk(const typename P::Params& p_, const int* tables_, int tiles, int pair_, int pairs_)
      : p(p_), tables(tables_), pair(pair_), pairs(pairs_) {
    whole = tiles / pairs * pairs;
    const int rest = tiles - whole;
    parts = rest ? min(kMaxN / 32, pairs / rest) : 1;
    const int total = whole + rest * parts;
    count = total > pair ? (total - pair + pairs - 1) / pairs : 0;
  }
  __device__ __forceinline__ bool next(typename P::Tile* t) {
    while (step < count) {
      const int i = pair + step++ * pairs;
      if (i < whole) {
        *t = P::tile(p, tables, i);
        return true;
      }
      const int j = (i - whole) / parts;
      *t = P::tile(p, tables, whole + j);
      P::narrow(t, i - whole - j * parts, parts);
      if (t->n > 0) return true;
    }
    return false;
  }
};

// What the roles of a CTA share.
template <int STAGES>
struct Block {
  using S = Smem<STAGES>;
  uint8_t* smem;
  uint32_t sbase, tmem;
  int warp, lane, rank, pair, pairs;
  volatile int* abort;
  unsigned int* err;

  __device__ __forceinline__ uint32_t bar(int i) const { return sbase + S::bars + 8 * i; }
  __device__ __forceinline__ uint32_t full(int s) const { return bar(s); }  // the leader's: both CTAs' stages are whole
  __device__ __forceinline__ uint32_t empty(int s) const { return bar(STAGES + s); }
  __device__ __forceinline__ uint32_t tfull(int b) const { return bar(2 * STAGES + b); }
  __device__ __forceinline__ uint32_t tempty(int b) const { return bar(2 * STAGES + kAccBufs + b); }
  __device__ __forceinline__ uint32_t drain() const { return bar(2 * STAGES + 2 * kAccBufs); }
  __device__ __forceinline__ int* tables() const { return reinterpret_cast<int*>(smem + S::extra); }

  // Barriers and tensor memory; then what the previous kernel of the stream wrote may be read.
  __device__ __forceinline__ void begin(uint8_t* raw, unsigned int* error) {
    const uint32_t raw_addr = smem_u32(raw);
    smem = raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    sbase = smem_u32(smem);
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    rank = (int)(cluster_ctarank() & 1u);
    pair = blockIdx.x >> 1;
    pairs = gridDim.x >> 1;
    abort = reinterpret_cast<volatile int*>(smem + S::misc + 4);
    err = error;
    pdl_launch_dependents();
    if (warp == 0 && lane == 0) {
      for (int s = 0; s < STAGES; ++s) {
        mbar_init(full(s), 1);
        mbar_init(empty(s), 1);
      }
      for (int b = 0; b < kAccBufs; ++b) {
        mbar_init(tfull(b), 1);
        mbar_init(tempty(b), 2 * kEpiWarps);  // of both CTAs
      }
      mbar_init(drain(), 1);
      *abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + S::misc),
                   "r"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
  }
  // Both CTAs' barriers exist before any arrival from the other.
  __device__ __forceinline__ void meet() {
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    tmem = *reinterpret_cast<const uint32_t*>(smem + S::misc);
  }
  // The pair meets, then frees its tensor memory together.
  __device__ __forceinline__ void end() {
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
  __device__ __forceinline__ void fail() const {
    flag_error(err, MOE_DEVERR_TIMEOUT);
    *abort = 1;
  }
};

// The TMA producer, one lane.
template <int STAGES>
struct Producer {
  const Block<STAGES>& b;
  uint32_t full0;
  int s = 0;
  uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
  __device__ __forceinline__ explicit Producer(const Block<STAGES>& b_) : b(b_), full0(map_to_rank(b_.full(0), 0)) {}

  template <class P>
  __device__ __forceinline__ bool run(const typename P::Params& p, Walk<P> walk) {
    typename P::Tile t;
    while (walk.next(&t)) {
      const uint32_t bytes = P::stage_bytes(p, t);
      const int blocks = (t.k + kBK - 1) / kBK;
      for (int kb = 0; kb < blocks; ++kb) {
        if (!mbar_wait(b.empty(s), phase ^ 1u, b.abort)) return false;
        if (b.rank == 0) mbar_arrive_expect_tx(b.full(s), bytes);
        const uint32_t a = b.sbase + s * kStageBytes;
        P::load(p, t, b.rank, kb, a, a + kOperandBytes, full0 + (uint32_t)(s * 8));
        issued_mask |= 1u << s;
        issued_parity = (issued_parity & ~(1u << s)) | (phase << s);
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    return true;
  }
  // Every stage this CTA filled has been read by the pair's MMAs before it exits.
  __device__ __forceinline__ void finish(bool ok) {
    for (int i = 0; i < STAGES && ok; ++i)
      if ((issued_mask >> i) & 1u && !mbar_wait(b.empty(i), (issued_parity >> i) & 1u, b.abort)) ok = false;
    if (ok) return;
    b.fail();
    const uint64_t t0 = global_timer_ns();  // copies in flight complete on the leader's barrier: let them land
    while (global_timer_ns() - t0 < kDrainTimeoutNs) {
    }
  }
};

// The leader's MMA issuer, a whole warp: it keeps the loop, so that its values are uniform, and one lane
// issues.  (With a lane that does it all, an MMA took 128 cycles to issue whatever its n, which left no
// slack for a late stage.)
template <int STAGES>
struct Issuer {
  const Block<STAGES>& b;
  int s = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool issued_any = false;
  __device__ __forceinline__ explicit Issuer(const Block<STAGES>& b_) : b(b_) {}

  template <class P>
  __device__ __forceinline__ bool run(Walk<P> walk) {
    const uint32_t fmt = P::kF16 ? 0u : 1u;
    const uint32_t base = (1u << 4) | (fmt << 7) | (fmt << 10) | ((P::kAMN ? 1u : 0u) << 15) |
                          ((P::kBMN ? 1u : 0u) << 16) | ((uint32_t)(kTileM >> 4) << 24);
    const uint64_t a0 = operand_desc<P::kAMN>(b.sbase);
    const uint64_t b0 = operand_desc<P::kBMN>(b.sbase + kOperandBytes);
    typename P::Tile t;
    while (walk.next(&t)) {
      const uint32_t idesc = base | ((uint32_t)(t.n >> 3) << 17);
      if (!__all_sync(0xffffffffu, mbar_wait_cluster(b.tempty(acc), acc_phase ^ 1u, b.abort))) return false;
      tc_fence_after();
      const uint32_t d = b.tmem + (uint32_t)(acc * kMaxN);
      for (int k = 0; k < t.k; k += kBK) {
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(b.full(s), phase, b.abort))) return false;
        tc_fence_after();
        const uint64_t da = a0 + (uint64_t)(s * (kStageBytes >> 4)), db = b0 + (uint64_t)(s * (kStageBytes >> 4));
        const int steps = (t.k - k + 15) / 16;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            if (kk < steps)
              mma_issue_pair(d, da + operand_step<P::kAMN>(kk), db + operand_step<P::kBMN>(kk), idesc, (k | kk) != 0);
          mma_commit_pair(b.empty(s));
        }
        __syncwarp();
        issued_any = true;
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (elect_one()) mma_commit_pair(b.tfull(acc));
      __syncwarp();
      if (++acc == kAccBufs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    return true;
  }
  __device__ __forceinline__ void finish(bool ok) {
    if (ok || !elect_one()) return;
    b.fail();
    if (issued_any) {  // the MMAs in flight finish before tensor memory is freed
      mma_commit_pair(b.drain());
      mbar_wait(b.drain(), 0, nullptr, kDrainTimeoutNs);
    }
  }
};

// An epilogue warp.
template <int STAGES>
struct Epilogue {
  const Block<STAGES>& b;
  uint32_t tempty0;
  int acc = 0;
  uint32_t acc_phase = 0;
  __device__ __forceinline__ explicit Epilogue(const Block<STAGES>& b_) : b(b_), tempty0(map_to_rank(b_.tempty(0), 0)) {}

  template <class P>
  __device__ __forceinline__ bool run(const typename P::Params& p, Walk<P> walk) {
    const int sub = b.warp & 3;  // TMEM lane quarter this warp may access
    typename P::Tile t;
    bool ok = true;
    while (ok && walk.next(&t)) {
      const uint32_t tbase = b.tmem + ((uint32_t)(sub * 32) << 16) + (uint32_t)(acc * kMaxN);
      P::epilogue(
          p, t, b.rank, sub, (b.warp - 2) >> 2, b.lane, tbase,
          [&] {
            ok = __all_sync(0xffffffffu, mbar_wait(b.tfull(acc), acc_phase, b.abort));
            if (!ok && b.lane == 0) b.fail();
            tc_fence_after();
            return ok;
          },
          [&] {
            tc_fence_before();
            __syncwarp();
            if (b.lane == 0) mbar_arrive_remote(tempty0 + (uint32_t)(acc * 8));
          });
      if (++acc == kAccBufs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    return ok;
  }
};

// One product.
template <class P, int STAGES>
__global__ void __launch_bounds__(kThreads, 1) pair_kernel(const __grid_constant__ typename P::Params p) {
  extern __shared__ uint8_t smem_raw[];
  Block<STAGES> b;
  b.begin(smem_raw, p.err);
  const Walk<P> walk(p, b.tables(), P::setup(p, b.tables()), b.pair, b.pairs);
  b.meet();
  if (b.warp == 0) {
    if (b.lane == 0) {
      Producer<STAGES> r(b);
      r.finish(r.template run<P>(p, walk));
    }
  } else if (b.warp == 1) {
    if (b.rank == 0) {
      Issuer<STAGES> r(b);
      r.finish(r.template run<P>(walk));
    }
  } else {
    Epilogue<STAGES> r(b);
    r.template run<P>(p, walk);
  }
  b.end();
}

// ------------------------------------------------------------------- host

// A map of 16-bit elements with boxes of 64 of them (128 bytes, 128B swizzle) along the first dimension.
inline bool make_map(CUtensorMap* map, const void* base, bool f16, int nd, const cuuint64_t* dims,
                     const cuuint64_t* strides, const cuuint32_t* box,
                     CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, nd,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [count][rows][cols], rows ld elements apart: boxes of box_rows rows of one matrix, of 64 columns or of 32
// (64 bytes, 64B swizzle).
inline bool make_map_3d(CUtensorMap* map, const void* base, bool f16, int64_t count, int64_t rows, int64_t cols,
                        int64_t ld, int box_rows, int box_cols = 64) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(rows * ld) * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  return make_map(map, base, f16, 3, dims, strides, box,
                  box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// The launch of a pair kernel: pairs of CTAs on all SMs, or fewer where there is not work for so many.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int pairs = 0;
  template <class Kernel>
  cudaError_t prepare(Kernel kern, int smem, int64_t most_pairs, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(device_sm_count() / 2 * 2);
    e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorNotSupported;
    if (most_pairs < pairs) pairs = (int)most_pairs;
    cfg.gridDim = dim3(2 * pairs);
    return cudaSuccess;
  }
};

template <class P, int STAGES>
cudaError_t launch_stages(const typename P::Params& p, int64_t tiles, int table_bytes, bool pdl, cudaStream_t s) {
  Launch l;
  const auto kern = pair_kernel<P, STAGES>;
  cudaError_t e = l.prepare(kern, Smem<STAGES>::bytes(table_bytes), tiles * (kMaxN / 32), s);
  if (e != cudaSuccess) return e;
  l.attr[1] = pdl_attribute();
  l.cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&l.cfg, kern, p);
}

// tiles: at most so many, before the last round is cut.  pdl: the launch may begin before the stream's
// previous kernel ends.  k: the reduction's length.  7 stages where the tables leave room for them (32768 rows
// on 128 fine-grained experts, forward: 2373 us, 2425 with 6 stages; 128 rows of 16 experts, D = 5120, H = 8192:
// 603 and 618), 6 where a tile is hardly more than that.
template <class P>
cudaError_t launch_pairs(const typename P::Params& p, int64_t tiles, int k, int table_bytes, bool pdl, cudaStream_t s) {
  if (tiles < 1) return cudaSuccess;
  return k > 8 * kBK && Smem<7>::bytes(table_bytes) <= kSmemMax ? launch_stages<P, 7>(p, tiles, table_bytes, pdl, s)
                                                                : launch_stages<P, 6>(p, tiles, table_bytes, pdl, s);
}

}  // namespace pg
}  // namespace moe
