// k_tree_tc.cu -- tree attention on the 5th-generation tensor cores (tcgen05.mma, accumulators in
// tensor memory), for bf16 queries over bf16 (head size 64 / 128) or e4m3 (128) pools of 16-position
// blocks.
//
// Work.  One CTA per SM walks its share of the items' key tiles (k_tree.cu cuts them).  An item is
// one (sequence, kv head) and up to two tiles of query rows; a row tile is whole nodes times the
// group's heads, at most 128 rows, one tensor-memory lane each.  Key tiles are 128 positions =
// eight pool blocks, fetched block by block with TMA from wherever the block table puts them.
//
// Two streams.  A softmax warpgroup (one thread per row, so no exchange between threads) and an
// S / P buffer and O accumulator in tensor memory make a stream; there are two.  An item with two
// row tiles gives each stream one, and both use the same key tiles: each K / V byte that reaches
// shared memory serves 256 rows.  An item with one row tile gives its key tiles to the
// streams in turn; the stream that takes the last one joins their states (m, l, O), while the
// other goes on with the next item.  Either way one stream's MMAs run while the other's
// exponentials do.
//
// Per key tile of a stream:  S = Q K^T (M 128, N 128, K = head size);  mask, running max (moved,
// with O rescaled, only when it grows by more than 2^8), p = 2^(s - m);  P written over S;
// O += P V.  Over bf16 pools P is a bf16 pair hi + lo (two products with V, weights good to
// 2^-16); over e4m3 pools it is one f16 value (2^-11), with V widened to f16 (exactly) in shared
// memory, while K's codes are used as they are: q is split into two e4m3 terms, hi + lo, with one
// power of two per row (exact down to 2^-9 of the row's largest element), two products for S.
// (Widening K too made the conversions bound the kernel.)  Row sums add the fp32 weights.
//
// Roles.  warp 0: TMA of K, warp 3: of Q (a ring of two row tiles) and V, into a ring of five
// 128-key stages (bf16) or three stages of codes for each (e4m3); warp 1: tensor-memory owner,
// issues S = Q K^T; warp 2: issues O += P V, and zeroes the V rows past the sequence's end (they may
// hold anything; K's are masked); warps 4..7 and 8..11: the streams' softmax and epilogue; warps
// 12..15 (e4m3 pools): split Q and widen V into one of two f16 tiles.
//
// Small calls (CL).  Instead of the planned shares, a cluster of 1 to 8 CTAs for each (sequence, kv
// head, item): each CTA plans its own part from the sequence's numbers (an even run of the key
// tiles), its softmax warps check the whole batch while the first tiles are on their way, and the
// CTAs' states are joined in key order through distributed shared memory.  One launch instead of
// three: a tree of 8 nodes over 700 positions takes 9.3 us instead of 16 (behind a table for 12 000
// positions or more, which the rule for the form leaves to the shares).
//
// What bounds it: up to 128 rows per kv head, the K / V bytes (a tile is 64 KB of bf16, 1.5 us of
// an SM's share of the measured copy bandwidth, against 0.8 us of tensor time): 64 sequences of up
// to 32 nodes x 4 heads over 512 to 4096 positions take 118 us, 5.9 TB/s, 0.88 of the copy
// bandwidth.  With two row tiles, the tensor cores and the chain of a stream (its S has to wait for
// the P V before it): 4 x 64 nodes x 8 heads over 65536 positions take 528 us at their best, 1040
// TFLOP/s of the formulas' work, 1560 with both terms of P, 0.81 of the measured peak; at full power
// the clock, and the time, depend on the box: up to 625 us.  Over e4m3 pools (half the bytes, V's
// widening on top) that chain, too: 48 x 16 nodes with a window take 94 us, 3.8 TB/s (52 us at the
// copy rate).  So does head size 64 (half the bytes over the same tiles): 64 sequences of up to 32
// nodes x 4 heads, a call of 90 us for 43 at the copy rate.  Items of up to 64 rows leave half of
// the lanes of S, P and O, and of the products, empty.
//
// Measured and left out: tiles of 64 keys with S and P double-buffered (Q is read twice as often:
// 160 -> 209 us for the first case above); straight-line loops in any role (the code runs out of
// the instruction cache); a pass over S saved by looking for larger scores 32 keys at a time, or
// S loaded ahead (no change: the softmax is not what the chain waits for most); eight converter
// warps, or widening by integer operations (no change, slower).
//
// Every mbarrier wait is bounded; one that runs out records PA_ETIMEOUT and raises an abort flag
// that ends the other roles' waits.  A softmax warp whose wait fails goes through the rest of its
// share without waiting or writing, so that no warp is left at the named barriers; the TMA
// issuers wait (bounded) for their copies in flight and the MMA issuers for their MMAs before the
// CTA gives its tensor memory back.
#include <algorithm>
#include <atomic>

#include "k_tree.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBN = 128;      // keys per tile
constexpr int kStages = 5;    // K / V ring (bf16 pools)
constexpr int kCodeStages = 3;  // e4m3 pools: a ring of codes for K, one for V

template <int D, bool FP8>
struct Shape {
  static constexpr int kHalves = D / 64;            // 64-dim halves of a tile: rows of 128 bytes
  static constexpr int kHalfBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // a 128-row tile of 16-bit values
  static constexpr int kStageBytes = FP8 ? kTileBytes / 2 : kTileBytes;  // a tile as it is loaded
  static constexpr int kThreads = FP8 ? 512 : 384;
  // K / V stages over bf16 pools: 8-row groups of (dim half, 8 rows of 128 bytes), as the 5-D
  // boxes write them; widened V and Q: dim half by dim half
  static constexpr int kRowGroup = FP8 ? 1024 : 1024 * kHalves;  // between 8-row groups
  static constexpr int kDimHalf = FP8 ? kHalfBytes : 1024;       // between dim halves
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffWide = kOffKV + 2 * kCodeStages * kStageBytes;  // e4m3: two tiles of V
  // [2][128] float2: a stream's m, l
  static constexpr int kOffX = FP8 ? kOffWide + 2 * kTileBytes : kOffKV + kStages * kTileBytes;
  static constexpr int kOffBad = kOffX + 2 * 128 * 8;          // [2][4] its warps' failed waits
  static constexpr int kOffBar = kOffBad + 2 * 4 * 4;
  static constexpr int kOffMisc = kOffBar + 48 * 8;
  // tensor-memory base, flags; e4m3: the rows' scale exponents of four Q tiles
  static constexpr int kOffExp = kOffMisc + 16;
  static constexpr int kOffSeg = kOffExp + (FP8 ? 4 * 128 : 0);  // clusters: the CTA's TreeSegment
  static constexpr int kSmem = kOffSeg + 64;
  // clusters: a CTA's state in the ring's place, once that is used up: O, rows padded by 16 bytes
  // (a warp's rows hit different banks), then (m, l)
  static constexpr int kStateLd = D + 4;
  static constexpr int kOffState = kOffKV;
  static constexpr int kOffML = kOffState + 256 * kStateLd * 4;
  static_assert(kOffML + 256 * 8 <= kOffX, "the state lies in the ring");
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

constexpr int kMostStages = 2 * kCodeStages;
static_assert(kMostStages >= kStages, "stage barriers");

// barriers (indices of consecutive 8-byte words)
enum : int {
  B_QFULL = 0,                     // Q buffer landed
  B_QEMPTY = B_QFULL + 2,          // its last S = Q K^T is done
  B_QCONV = B_QEMPTY + 2,          // e4m3: it has been split
  B_FULL = B_QCONV + 2,            // stage landed: K's copies, then V's (B_FULL + kMostStages + ..)
  B_EMPTY = B_FULL + 2 * kMostStages,  // its copy has been used up: K's copies, then V's
  B_WIDE = B_EMPTY + 2 * kMostStages,  // e4m3: a V tile is ready as f16
  B_WFREE = B_WIDE + 2,            // e4m3: its P V is done
  B_SFULL = B_WFREE + 2,           // per stream: S is ready
  B_PFULL = B_SFULL + 2,           // P is written
  B_PVDONE = B_PFULL + 2,          // P V is done: O is current, the S / P buffer is free
  B_OFREE = B_PVDONE + 2,          // the segment's O has been read
  B_FIN = B_OFREE + 2,
  B_NEVER = B_FIN + 2,             // nothing arrives on it (the debug_stall test hook)
  kNumBars = B_NEVER + 1
};
static_assert(kNumBars <= 48, "barrier area");

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int x) { return (uint32_t)x * 128; }
__device__ __forceinline__ uint32_t col_o(int x) { return 256 + (uint32_t)x * 128; }

// One CTA's MMAs (cta_group::1), issued by the one lane with `elect` of a warp in uniform control
// flow.
__device__ __forceinline__ void mma_ss(uint32_t elect, uint32_t d, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\tsetp.ne.u32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elect)
      : "memory");
}
// The same over e4m3 operands (K = 32).
__device__ __forceinline__ void mma_ss_e4m3(uint32_t elect, uint32_t d, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\tsetp.ne.u32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elect)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t elect, uint32_t d, uint32_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\tsetp.ne.u32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elect)
      : "memory");
}
// Arrive on `bar` once this thread's MMAs so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .u32 l;\n\t.reg .pred e;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

struct Ctx {
  uint8_t* sm;
  uint64_t* bar;
  volatile int* abort;
  int* status;
  uint64_t limit;
  bool work;  // false: an earlier error, nothing is done
  const TreeSegment* own;  // clusters: the CTA's part of its cluster's item
};

// The segments of a CTA: its share's, or the one it has in its cluster (CL).
template <bool CL>
struct Walk {
  TreeWalk w;
  __device__ __forceinline__ Walk(const Ctx& c, const TreeParams& p) : w(p, blockIdx.x) {}
  __device__ __forceinline__ bool next(const TreeParams& p, TreeSegment& g) { return w.next(p, g); }
};
template <>
struct Walk<true> {
  const TreeSegment* own;
  int left;
  __device__ __forceinline__ Walk(const Ctx& c, const TreeParams& p) : own(c.own) {
    // (not a constant to the compiler, which otherwise writes the roles' loops out several times)
    asm volatile("mov.u32 %0, 1;" : "=r"(left));
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreeSegment& g) {
    if (left == 0) return false;
    --left;
    g = *own;
    return g.t1 > g.t0;
  }
};

__device__ __forceinline__ bool wait_bar(const Ctx& c, int idx, uint32_t parity) {
  uint64_t* b = c.bar + idx;
  uint64_t t0 = 0;
  for (uint32_t i = 0; !mbar_try_wait(b, parity); ++i) {
    if ((i & 63u) != 63u) continue;
    const uint64_t now = globaltimer_ns();
    t0 = t0 ? t0 : now;
    const bool late = now - t0 > c.limit;
    if (late) {
      record_error(c.status, PA_ETIMEOUT);
      *c.abort = 1;
    }
    if (late || *c.abort) return false;
  }
  return true;
}
__device__ __forceinline__ bool wait_all(const Ctx& c, int idx, uint32_t parity) {
  return __all_sync(kFull, wait_bar(c, idx, parity));
}

// Over bf16 pools K and V share a ring.  The copies of a CTA's tiles 0, 1, 2, ... are numbered in
// the order in which they are needed: K0 V0 K1 V1 ... (K_t 2t, V_t 2t + 1) where an item may have
// two row tiles, and K0 - K1 V0 K2 V1 K3 ... (K_t 2t, V_t 2t + 3; `ahead`) where none has: the
// streams then work on two tiles at once, and tile t's V is needed after tile t + 1's K.  Copy n
// uses stage n % kStages, so K and V take turns in a stage, and an operand's copies come to the
// same stage every kStages tiles.
//
// A parity tells neighbouring phases of a barrier apart, no more, so every phase of a barrier is
// waited for, in order, by the one that goes on by it: a stage's "landed" barriers are one set per
// operand, and so are its "empty" ones.  K's producer waits for V's copies to leave a stage
// and V's for K's (copy n for copy n - 5's).  (One "empty" barrier for both, its phases waited for in
// turn by the two, let a producer mistake a phase two behind for the one before: a consumption
// counts when its issuer comes to say so, which can be later than what depends on its products.)
//
// Over e4m3 pools each operand has a ring of code stages of its own (0 .. 2 K, 3 .. 5 V), half as
// large.  V's codes are widened into one of two f16 tiles, and their stage is free as soon as they
// have been read: more bytes are on their way than when a stage held its V until P V was done.
__device__ __forceinline__ bool ring_ahead(const TreeParams& p) {
  return p.rows_per_item == p.tile_rows;
}
template <bool FP8>
struct Ring {
  static constexpr uint32_t kLen = FP8 ? kCodeStages : kStages;
  uint32_t st;         // stage of this operand's current copy
  uint32_t turn, par;  // tile t % kLen, and the parity of t / kLen: its visits to the stage
  __device__ __forceinline__ Ring(const TreeParams& p, int kv) {
    if constexpr (FP8)
      st = kv ? kCodeStages : 0;
    else
      st = kv ? (ring_ahead(p) ? 3 : 1) : 0;
    turn = par = 0;
  }
  __device__ __forceinline__ void next() {  // the next tile's copy of the same operand
    if constexpr (FP8) {
      ++st;
    } else {
      st += 2;
      if (st >= kStages) st -= kStages;
    }
    if (++turn == kLen) {
      turn = 0;
      par ^= 1;
      if constexpr (FP8) st -= kCodeStages;
    }
  }
};
static_assert(kStages == 5, "copies n and n - 5 are of different operands");

// Both streams take all key tiles of a segment with two row tiles.  With one row tile the streams
// alternate, over segments too: the stream that does not take a segment's last tile begins the
// next one, while the other finishes this one.
__device__ __forceinline__ bool two_tiles(const TreeParams& p, const TreeSegment& g) {
  return g.rows > p.tile_rows;
}

// ---- roles --------------------------------------------------------------------------------------

// Warp 0 brings K (kv = 0), warp 3 Q and V (kv = 1); both walk the whole share.  A block is one
// box, issued by a lane of its own: a warp's TMA instructions go out one lane after the other,
// and one warp issuing 32 half-size boxes per key tile was what bound this kernel.
template <int D, bool FP8, bool CL>
__device__ void producer(const Ctx& c, const TreeParams& p, const CUtensorMap* tkv,
                         const CUtensorMap* tq, int kv) {
  using S = Shape<D, FP8>;
  const int lane = threadIdx.x & 31;
  uint64_t* full = c.bar + B_FULL + kv * kMostStages;
  Ring<FP8> r(p, kv);
  // the stage's last copy is that of a tile `lag` before, of the other operand where they share
  uint64_t* empty = c.bar + B_EMPTY + (FP8 ? kv : kv ^ 1) * kMostStages;
  uint32_t lag = FP8 ? kCodeStages : kv ? (ring_ahead(p) ? 1 : 2) : (ring_ahead(p) ? 4 : 3);
  uint32_t gone = 0, gone_par = 0;  // that tile % kLen, the parity of its visit
  uint32_t issued = 0, nq = 0;  // this warp's stages; row tiles of Q (tile n uses buffer n % 2)
  bool ok = c.work;
  Walk<CL> walk(c, p);
  TreeSegment g;
  while (ok && walk.next(p, g)) {
    const int32_t* row = p.m.block_tables + (int64_t)g.s * p.m.max_blocks;
    const int blocks = (g.n + 15) / 16;
    const int b0 = g.kv0 / 16 + 8 * g.t0 + lane;
    int next = lane < 8 && b0 < blocks ? row[b0] : -1;
    const int tiles = kv ? (two_tiles(p, g) ? 2 : 1) : 0;
    for (int x = 0; ok && x < tiles; ++x) {
      if (lane == 0) {
        ok = wait_bar(c, B_QEMPTY + (nq & 1), ((nq >> 1) & 1) ^ 1);
        if (ok) {
          uint64_t* bar = c.bar + B_QFULL + (nq & 1);
          mbar_arrive_expect_tx(bar, (uint32_t)p.tile_rows * 128 * S::kHalves);
          // (an item's rows are those of whole row tiles)
          const int tok = g.qs + (ring_ahead(p) ? g.item : 2 * g.item + x) * p.tile_tokens;
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
            tma_load_3d(c.sm + (nq & 1) * S::kTileBytes + h * S::kHalfBytes, tq, 64 * h,
                        g.kvh * p.m.group, tok, bar);
        }
      }
      ok = __shfl_sync(kFull, (int)ok, 0);
      if (ok) ++nq;
    }
    for (int j = g.t0; ok && j < g.t1; ++j) {
      const int id = next;
      const int nb = b0 + 8 * (j + 1 - g.t0);
      if (j + 1 < g.t1) next = lane < 8 && nb < blocks ? row[nb] : -1;
      if (lane == 0) {
        if (issued >= lag) ok = wait_bar(c, (int)(empty - c.bar) + r.st, gone_par);
        if (ok) mbar_arrive_expect_tx(full + r.st, S::kStageBytes);
      }
      ok = __shfl_sync(kFull, (int)ok, 0);
      if (!ok) break;
      if (lane < 8) {  // a block past the end: rows outside the pool, which TMA fills with zeros
        uint8_t* dst = c.sm + S::kOffKV + r.st * S::kStageBytes + lane * (S::kStageBytes / 8);
        if constexpr (FP8)
          tma_load_3d(dst, tkv, 0, g.kvh, id >= 0 ? id * 16 : -16, full + r.st);
        else
          tma_load_5d(dst, tkv, 0, 0, 0, id >= 0 ? id * 2 : -2, g.kvh, full + r.st);
      }
      if (issued >= lag && ++gone == Ring<FP8>::kLen) {
        gone = 0;
        gone_par ^= 1;
      }
      ++issued;
      r.next();
    }
  }
  // the copies still in flight (after an abort; otherwise all have been consumed): the last ones
  // are the last of their barriers
  if (lane == 0) {
    Ring<FP8> d(p, kv);
    for (uint32_t k = 0; k < issued; ++k, d.next())
      if (k + Ring<FP8>::kLen >= issued) mbar_wait(full + d.st, d.par, c.limit);
    for (uint32_t k = nq > 2 ? nq - 2 : 0; k < nq; ++k)
      mbar_wait(c.bar + B_QFULL + (k & 1), (k >> 1) & 1u, c.limit);
  }
  __syncwarp();
}

template <int D, bool FP8, bool CL>
__device__ void s_issuer(const Ctx& c, const TreeParams& p, uint32_t tmem) {
  using S = Shape<D, FP8>;
  // (f8f6f4's descriptor has zeros where e4m3 operands are named)
  constexpr uint32_t kIdesc = idesc_f16kind(128, kBN, 0, FP8 ? 0 : 1);
  constexpr int kQ = FP8 ? B_QCONV : B_QFULL;
  const uint32_t sm = smem_u32(c.sm), elect = (threadIdx.x & 31) == 0;
  Ring<FP8> r(p, 0);
  uint32_t nq = 0, cnt[2] = {0, 0};  // row tiles used; tiles of each stream
  int turn = 0;                      // the stream whose turn it is
  if (!c.work) return;
  Walk<CL> walk(c, p);
  TreeSegment g;
  while (walk.next(p, g)) {
    const bool two = two_tiles(p, g);
    for (int j = g.t0; j < g.t1; ++j) {
      if (!wait_all(c, B_FULL + r.st, r.par)) return;
      const uint32_t kb = sm + S::kOffKV + r.st * S::kStageBytes;
#pragma unroll 1
      for (int y = 0; y < (two ? 2 : 1); ++y) {
        const int x = two ? y : turn;  // the stream
        const uint32_t q = nq + (two ? y : 0);
        if (j == g.t0 && !wait_all(c, kQ + (q & 1), (q >> 1) & 1)) return;
        const uint32_t n = x ? cnt[1] : cnt[0];
        if (!wait_all(c, B_PVDONE + x, (n & 1) ^ 1)) return;  // the buffer's last P is used up
        tc_fence_after();
        const uint32_t qb = sm + (q & 1) * S::kTileBytes;
        // (addresses of a descriptor advance in units of 16 bytes)
        uint64_t qd = sdesc(qb, 16, 1024), kd = sdesc(kb, 16, S::kRowGroup);
#pragma unroll 1
        for (int h = 0; h < S::kHalves; ++h) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (FP8)  // q's high codes, then its low ones, over all 128 dims of K
              mma_ss_e4m3(elect, tmem + col_s(x), qd + 2 * kk, kd + 2 * kk, kIdesc,
                          (h | kk) ? 1u : 0u);
            else
              mma_ss(elect, tmem + col_s(x), qd + 2 * kk, kd + 2 * kk, kIdesc, (h | kk) ? 1u : 0u);
          }
          qd += S::kHalfBytes / 16;
          if constexpr (!FP8) kd += S::kDimHalf / 16;
        }
        mma_commit(c.bar + B_SFULL + x);
        if (x) ++cnt[1]; else ++cnt[0];
      }
      if (!two) turn ^= 1;
      mma_commit(c.bar + B_EMPTY + r.st);
      __syncwarp();
      r.next();
    }
    for (int y = 0; y < (two ? 2 : 1); ++y) mma_commit(c.bar + B_QEMPTY + ((nq + y) & 1));
    nq += two ? 2 : 1;
  }
}

template <int D, bool FP8, bool CL>
__device__ void pv_issuer(const Ctx& c, const TreeParams& p, uint32_t tmem) {
  using S = Shape<D, FP8>;
  constexpr uint32_t kIdesc = idesc_f16kind(128, D, 1, FP8 ? 0 : 1);
  const int lane = threadIdx.x & 31;
  const uint32_t elect = lane == 0;
  Ring<FP8> r(p, 1);
  uint32_t wide = 0;  // e4m3: V tiles so far
  uint32_t cnt[2] = {0, 0}, seg = 0;
  int turn = 0;
  if (!c.work) return;
  Walk<CL> walk(c, p);
  TreeSegment g;
  for (; walk.next(p, g); ++seg) {
    const bool two = two_tiles(p, g);
    for (int j = g.t0; j < g.t1; ++j) {
      if (!(FP8 ? wait_all(c, B_WIDE + (wide & 1), (wide >> 1) & 1)
                : wait_all(c, B_FULL + kMostStages + r.st, r.par)))
        return;
      uint8_t* v = c.sm + (FP8 ? S::kOffWide + (wide & 1) * S::kTileBytes
                               : S::kOffKV + r.st * S::kStageBytes);
      if constexpr (!FP8) {  // (the converters do it over e4m3 pools)
        // rows of the last block past the sequence's end: zeros (whole blocks past it are)
        const int lim = g.n - (g.kv0 + j * kBN);
        if (lim < kBN && (lim & 15)) {
          for (int i = lane; i < (16 - (lim & 15)) * 8 * S::kHalves; i += 32) {
            const int row = lim + i / (8 * S::kHalves), h = (i >> 3) % S::kHalves;
            *reinterpret_cast<uint4*>(v + (row >> 3) * S::kRowGroup + h * S::kDimHalf +
                                      (row & 7) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      const uint32_t vb = smem_u32(v);
#pragma unroll 1
      for (int y = 0; y < (two ? 2 : 1); ++y) {
        const int x = two ? y : turn;
        const bool first = two ? j == g.t0 : j - g.t0 < 2;
        if (first && !wait_all(c, B_OFREE + x, (seg & 1) ^ 1)) return;
        const uint32_t n = x ? cnt[1] : cnt[0];
        if (!wait_all(c, B_PFULL + x, n & 1)) return;
        tc_fence_after();
        uint64_t vd = sdesc(vb, S::kDimHalf, S::kRowGroup);
        uint32_t pc = tmem + col_s(x), acc = first ? 0u : 1u;
        constexpr uint64_t kStep = 2 * S::kRowGroup / 16;  // 16 keys
#pragma unroll 1
        for (int kk = 0; kk < kBN / 32; ++kk) {  // 32 keys: hi, hi and lo, lo
          mma_ts(elect, tmem + col_o(x), pc, vd, kIdesc, acc);
          mma_ts(elect, tmem + col_o(x), pc + 8, vd + kStep, kIdesc, 1u);
          if constexpr (!FP8) {
            mma_ts(elect, tmem + col_o(x), pc + 16, vd, kIdesc, 1u);
            mma_ts(elect, tmem + col_o(x), pc + 24, vd + kStep, kIdesc, 1u);
          }
          vd += 2 * kStep;
          pc += 32;
          acc = 1;
        }
        mma_commit(c.bar + B_PVDONE + x);
        if (x) ++cnt[1]; else ++cnt[0];
      }
      if (!two) turn ^= 1;
      mma_commit(c.bar + (FP8 ? B_WFREE + (wide & 1) : B_EMPTY + kMostStages + r.st));
      __syncwarp();
      if constexpr (FP8)
        ++wide;
      else
        r.next();
    }
  }
}

// Widen a staged tile of 128 x 128 codes (rows of 128 bytes with the 128-byte swizzle) to f16, dim
// half by dim half.  A warp takes rows 32 w .. 32 w + 31, 16 at a time.  Rows at or past `lim`
// become zeros.
__device__ __forceinline__ void widen_rows(const uint8_t* codes, uint8_t* tile, int w, int lane,
                                           int lim) {
  constexpr int kHalf = 128 * 128;
#pragma unroll 1
  for (int r0 = 32 * w; r0 < 32 * w + 32; r0 += 16) {
    uint4 src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      src[i] = *reinterpret_cast<const uint4*>(codes + r0 * 128 + (lane + 32 * i) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = lane + 32 * i, r = r0 + (ch >> 3), sw = r & 7;
      const int L = (ch & 7) ^ sw;             // dims 16 L .. 16 L + 15
      const int h = L >> 2, c0 = 2 * (L & 3);  // dim half, first output chunk
      uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
      if (r < lim) {
        widen4(src[i].x, lo.x, lo.y);
        widen4(src[i].y, lo.z, lo.w);
        widen4(src[i].z, hi.x, hi.y);
        widen4(src[i].w, hi.z, hi.w);
      }
      uint8_t* row = tile + h * kHalf + r * 128;
      *reinterpret_cast<uint4*>(row + ((c0 ^ sw) << 4)) = lo;
      *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ sw) << 4)) = hi;
    }
  }
}

// Split the warp's 32 rows of a Q tile (bf16, dim half by dim half) into e4m3 codes, in place: hi
// in the first half's rows, lo in the second's (rows of 128 bytes, swizzled as they were).  With the
// row times 2^s, its largest magnitude in [128, 256), hi is the nearest code and lo the rest: eight
// significant bits in two of four, exactly, for elements down to 2^-9 of the row's largest (and to
// 2^-17 of it below that).  NaN elements give NaN codes, an infinite one the whole row.  Two lanes
// share a row, a dim half each.
__device__ __forceinline__ void split_q(uint8_t* tile, int8_t* exps, int w, int lane) {
  constexpr int kHalf = 128 * 128;
#pragma unroll 1
  for (int it = 0; it < 2; ++it) {
    const int r = 32 * w + 16 * it + (lane >> 1), h = lane & 1, sw = r & 7;
    uint4 v[8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // (chunk i of the row; the lanes start at different banks)
      v[i] = *reinterpret_cast<const uint4*>(tile + h * kHalf + r * 128 + ((i ^ sw) << 4));
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(x[e] << 16)),
                           fabsf(__uint_as_float(x[e] & 0xffff0000u))));
    }
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    const int exp = min(max(134 - (int)(__float_as_uint(m) >> 23), -120), 120);
    // (e4m3 has no infinity to saturate to: a row that holds one becomes NaN as a whole)
    const float up = m < INFINITY ? __uint_as_float((uint32_t)(127 + exp) << 23) : NAN;
    __syncwarp();  // both lanes of every row have loaded it
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t hw = 0, lw = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float a = __uint_as_float(x[2 * e + k] << 16) * up;
          const float b = __uint_as_float(x[2 * e + k] & 0xffff0000u) * up;
          const uint32_t c = f32x2_to_e4m3x2(a, b);
          const uint32_t f = e4m3x2_to_f16x2((uint16_t)c);
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&f));
          hw |= c << (16 * k);
          lw |= (uint32_t)f32x2_to_e4m3x2(a - back.x, b - back.y) << (16 * k);
        }
        hi[e] = hw;
        lo[e] = lw;
      }
      // dims 64 h + 8 i ..: 8 bytes of 16-byte chunk 4 h + i / 2
      uint8_t* to = tile + r * 128 + (((4 * h + (i >> 1)) ^ sw) << 4) + 8 * (i & 1);
      *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(to + kHalf) = make_uint2(lo[0], lo[1]);
    }
    if (h == 0) exps[r] = (int8_t)exp;
  }
}

// Warps 12 to 15 split Q and widen V, a quarter of every tile each.  K is used as it is.
template <int D, bool CL>
__device__ void converter(const Ctx& c, const TreeParams& p) {
  using S = Shape<D, true>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 12;
  Ring<true> r(p, 1);
  uint32_t nq = 0, wide = 0;
  if (!c.work) return;
  Walk<CL> walk(c, p);
  TreeSegment g;
  while (walk.next(p, g)) {
    const int tiles = two_tiles(p, g) ? 2 : 1;
#pragma unroll 1
    for (int x = 0; x < tiles; ++x, ++nq) {
      if (!wait_all(c, B_QFULL + (nq & 1), (nq >> 1) & 1)) return;
      split_q(c.sm + (nq & 1) * S::kTileBytes,
              reinterpret_cast<int8_t*>(c.sm + S::kOffExp) + (nq & 3) * 128, w, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar + B_QCONV + (nq & 1));
    }
    for (int j = g.t0; j < g.t1; ++j) {
      const uint32_t x = wide & 1;
      if (!wait_all(c, B_WFREE + x, ((wide >> 1) & 1) ^ 1)) return;
      if (!wait_all(c, B_FULL + kMostStages + r.st, r.par)) return;
      widen_rows(c.sm + S::kOffKV + r.st * S::kStageBytes, c.sm + S::kOffWide + x * S::kTileBytes, w,
                 lane, g.n - (g.kv0 + j * kBN));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(c.bar + B_EMPTY + kMostStages + r.st);
        mbar_arrive(c.bar + B_WIDE + x);
      }
      ++wide;
      r.next();
    }
  }
}

// Visible keys of one row in a tile's 128 positions from key0 on, 32 to a word.
__device__ __forceinline__ void visible_keys(const TreeParams& p, const TreeSegment& g, int tok,
                                             int pos, int key0, uint32_t (&see)[4]) {
  const int ctx = g.n - g.nodes;
  const int node0 = key0 - ctx;  // node of bit 0
  // the row's words that hold these bits, all requested at once
  uint32_t row[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    const int i = (node0 >> 5) + k;
    row[k] = i >= 0 && 32 * i < g.nodes ? (uint32_t)p.mask[(int64_t)tok * p.mask_words + i] : 0u;
  }
  const int far = max(pos - p.m.window, -1);  // (not so low that a key's distance overflows)
  // Nodes too far behind pos are looked for one by one, unless none can be: positions are not
  // negative, and a first key kv0 > 0 says that the sequence's lowest one is at least
  // kv0 + window - 1.
  const bool look = p.m.window > 0 && far >= 0 && !(g.kv0 > 0 && g.kv0 + p.m.window - 1 > far);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int key = key0 + 32 * q, node = node0 + 32 * q;
    uint32_t w = 0;
    if (key < ctx) {  // context positions from pos - window + 1 on
      const int hi = min(32, ctx - key);
      w = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
      if (p.m.window > 0) {
        const int lo = far + 1 - key;
        w = lo >= 32 ? 0u : lo > 0 ? w & (0xffffffffu << lo) : w;
      }
    }
    uint32_t t = __funnelshift_r(row[q], row[q + 1], node0 & 31);
    const int end = g.nodes - node;  // bits from there on are past the tree
    if (end < 32) t = end > 0 ? t & ((1u << end) - 1u) : 0u;
    see[q] = w | t;
  }
  if (!look) return;
#pragma unroll 1
  for (int i = max(0, -node0); i < kBN && node0 + i < g.nodes; ++i) {
    const uint32_t bit = 1u << (i & 31);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i >> 5 == q && (see[q] & bit) && p.m.positions[g.qs + node0 + i] <= far) see[q] &= ~bit;
  }
}

// The weights p = 2^(s * sl + nb) of 32 keys (packed pairs), added to `sum` and written to
// tensor memory for the product with V: bf16 hi in columns 0 .. 15 and lo in 16 .. 31, or f16 in
// columns 0 .. 15.
template <bool FP8>
__device__ __forceinline__ void weights32(uint32_t taddr, const uint32_t (&s)[32], uint64_t sl,
                                          uint64_t nb, uint64_t (&sum)[2]) {
  uint32_t w[FP8 ? 16 : 32];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a, b;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sl, nb), a,
              b);
    a = fast_exp2(a);
    b = fast_exp2(b);
    const uint64_t ab = f2_pack(a, b);
    sum[e & 1] = f2_add(sum[e & 1], ab);
    if constexpr (FP8) {
      w[e] = pack_f16x2(a, b);
    } else {
      w[e] = pack_bf16x2(a, b);
      // (a - hi is exact: hi is within half a bf16 step of a)
      f2_unpack(f2_fma(f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)),
                       f2_pack(-1.f, -1.f), ab), a, b);
      w[16 + e] = pack_bf16x2(a, b);
    }
  }
  if constexpr (FP8)
    tmem_st16(taddr, w);
  else
    tmem_st32(taddr, w);
}

// Handing a stream's state over at a segment's end: the warpgroup that finishes first arrives and
// goes on, the other waits for it.  Two barriers in turn.
__device__ __forceinline__ void state_given(int par) {
  __syncwarp();
  asm volatile("bar.arrive %0, 256;" ::"r"(1 + par) : "memory");
}
__device__ __forceinline__ void state_taken(int par) {
  __syncwarp();
  asm volatile("bar.sync %0, 256;" ::"r"(1 + par) : "memory");
}

// ---- small calls: a cluster for each item -------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// Address, in the cluster's shared window, of p's counterpart in CTA `rank`.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// One warp: this CTA's part of its cluster's item.  An item that the batch does not have, or
// whose sequence's numbers cannot be used as indices, has no rows and no tiles.
__device__ __forceinline__ void plan_own(const TreeParams& p, TreeSegment* out, int lane) {
  const VarlenMeta& m = p.m;
  const int rank = blockIdx.x % p.cluster;
  int u = blockIdx.x / p.cluster;
  TreeSegment g;
  g.kvh = u % m.num_kv_heads;
  u /= m.num_kv_heads;
  g.item = u % p.items;
  g.s = u / p.items;
  g.row0 = g.item * p.rows_per_item;
  g.qs = m.query_start_loc[g.s];
  const int qe = m.query_start_loc[g.s + 1];
  g.n = m.seq_lens[g.s];
  g.nodes = g.rows = g.kv0 = g.t0 = g.t1 = 0;
  g.slot = p.cluster > 1 ? 0 : -1;
  if (g.qs >= 0 && qe > g.qs && (int64_t)qe <= m.num_tokens && qe - g.qs <= 32 * (int64_t)p.mask_words &&
      g.n >= qe - g.qs && ((int64_t)g.n + 15) / 16 <= m.max_blocks) {
    g.nodes = qe - g.qs;
    const int rows = g.nodes * m.group;
    if (g.row0 < rows) {
      g.rows = min(p.rows_per_item, rows - g.row0);
      if (m.window > 0) {
        int lo = INT_MAX;
    #pragma unroll 1
        for (int t = lane; t < g.nodes; t += 32) lo = min(lo, m.positions[g.qs + t]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lo = min(lo, __shfl_xor_sync(kFull, lo, o));
        g.kv0 = min(max(max(lo, 0) - m.window + 1, 0), g.n - g.nodes);
        g.kv0 -= g.kv0 % 16;
      }
      const int tiles = (g.n - g.kv0 + kBN - 1) / kBN;
      g.t0 = (int)((int64_t)tiles * rank / p.cluster);
      g.t1 = (int)((int64_t)tiles * (rank + 1) / p.cluster);
    }
  }
  if (lane == 0) *out = g;
}

// Whether this thread (of 256) finds the batch not valid; what k_tree_plan checks.
__device__ __forceinline__ bool batch_refused(const TreeParams& p, int tid) {
  const VarlenMeta& m = p.m;
  bool bad = false;
#pragma unroll 1
  for (int g = tid; g < m.num_kv_heads; g += 256) {
    const float a = m.k_scales ? m.k_scales[g] : 1.f, b = m.v_scales ? m.v_scales[g] : 1.f;
    bad |= !(a > 0.f && a <= 3.402823466e38f) || !(b > 0.f && b <= 3.402823466e38f);
  }
#pragma unroll 1
  for (int s = tid; s < m.num_seqs; s += 256) {
    const int qs = m.query_start_loc[s], qe = m.query_start_loc[s + 1], n = m.seq_lens[s];
    bad |= qs < 0 || qe < qs || (int64_t)qe > m.num_tokens || (s == 0 && qs != 0) ||
           (s == m.num_seqs - 1 && (int64_t)qe != m.num_tokens);
    if (qe > qs)
      bad |= n < (int64_t)qe - qs || (int64_t)qe - qs > 32 * (int64_t)p.mask_words ||
             ((int64_t)n + 15) / 16 > m.max_blocks;
  }
  if (m.window > 0)
#pragma unroll 1
    for (int64_t t = tid; t < m.num_tokens; t += 256) bad |= m.positions[t] < 0;
  const int per = (m.max_blocks + 31) / 32;  // 32 entries of a table row: a warp's
#pragma unroll 1
  for (int i = tid >> 5; i < m.num_seqs * per; i += 8) {
    const int s = i / per, e = i % per * 32 + (tid & 31);
    const int qs = m.query_start_loc[s], qe = m.query_start_loc[s + 1], n = m.seq_lens[s];
    if (qe <= qs || n < 1) continue;
    if (e < (int)min(((int64_t)n + 15) / 16, (int64_t)m.max_blocks)) {
      const int id = m.block_tables[(int64_t)s * m.max_blocks + e];
      bad |= id < 0 || (int64_t)id >= m.num_blocks;
    }
  }
  return bad;
}

// The eight softmax warps, after the cluster's barrier: the CTA's share of its item's rows, from
// all CTAs' states in key order.
template <int D, bool FP8>
__device__ void cluster_merge(const Ctx& c, const TreeParams& p) {
  using S = Shape<D, FP8>;
  constexpr int E = D / 32;  // a lane's values of a row
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 4, C = p.cluster;
  const TreeSegment& g = *c.own;
  // (a failed wait in any CTA, or a batch that is not valid: nothing is written)
  const bool failed = lane < C && peer_load(peer_addr(const_cast<int*>(c.abort), lane)) != 0;
  if (__any_sync(kFull, failed)) return;
  // 8 / C rows at a time, so that eight loads are in flight whatever C: lane k < 8 has the (m, l)
  // of row k / C from CTA k % C
  const int lg = __ffs(C) - 1, low = C - 1, R = 8 >> lg, rank = (int)cluster_rank();
  const uint32_t ml = peer_addr(c.sm + S::kOffML, lane & low);
  const uint32_t o = smem_u32(c.sm + S::kOffState) + lane * E * 4;
#pragma unroll 1
  for (int i0 = R * warp; rank + C * i0 < g.rows; i0 += 8 * R) {  // rows rank + C i0, + C (i0 + 1) ..
    const int mine = rank + C * (i0 + (lane >> lg));
    const bool have = lane < 8 && mine < g.rows;
    const float2 st = have ? peer_load2(ml + mine * 8) : make_float2(-INFINITY, 0.f);
    float M = st.x;
#pragma unroll 1
    for (int k = 1; k < C; k <<= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, k));
    const float w = st.x == -INFINITY ? 0.f : exp2f(st.x - M);
    float L = w * st.y;
#pragma unroll 1
    for (int k = 1; k < C; k <<= 1) L += __shfl_xor_sync(kFull, L, k);
    float f = 0.f;
    int to = -1;  // row of the output
    if (have) {
      const int n = g.row0 + mine, tok = g.qs + n / m.group, h = g.kvh * m.group + n % m.group;
      f = tree_finish(p, g.kvh, h, tok, M, L, (lane & low) == 0);
      to = tok * m.num_heads + h;
    }
    float4 v[8];
    float wk[8];
    const uint32_t from = o + (rank + C * i0) * S::kStateLd * 4;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      wk[k] = __shfl_sync(kFull, w, k);
      if (wk[k] > 0.f) {  // (a row past the item's, or a CTA without a tile, left nothing)
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(a)
                     : "r"(from + (k >> lg << lg) * S::kStateLd * 4), "r"(k & low));
        if constexpr (E == 4) {
          v[k] = peer_load4(a);
        } else {
          const float2 h = peer_load2(a);
          v[k].x = h.x;
          v[k].y = h.y;
        }
      }
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[0] += wk[k] * v[k].x;
      acc[1] += wk[k] * v[k].y;
      acc[2] += wk[k] * v[k].z;
      acc[3] += wk[k] * v[k].w;
      if (((k + 1) & low) != 0) continue;  // not the row's last CTA
      const float fk = __shfl_sync(kFull, f, k);
      const int row = __shfl_sync(kFull, to, k);
      if (row >= 0) {
        const uint32_t lo = pack_bf16x2(acc[0] * fk, acc[1] * fk);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (int64_t)row * D + lane * E;
        if constexpr (E == 4)
          *reinterpret_cast<uint2*>(out) = make_uint2(lo, pack_bf16x2(acc[2] * fk, acc[3] * fk));
        else
          *reinterpret_cast<uint32_t*>(out) = lo;
      }
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
    }
  }
}

// The streams' threads: warpgroup x (warps 4 + 4x ..), thread = row = tensor-memory lane.
template <int D, bool FP8, bool CL>
__device__ void softmax_role(const Ctx& c, const TreeParams& p, uint32_t tmem, uint32_t stall) {
  using S = Shape<D, FP8>;
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 4;
  const int x = warp >> 2, quad = warp & 3;
  const int r = 32 * quad + lane;
  const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
  float2* xchg = reinterpret_cast<float2*>(c.sm + S::kOffX);
  int* bads = reinterpret_cast<int*>(c.sm + S::kOffBad);
  uint32_t cnt[2] = {0, 0};  // tiles of both streams so far
  uint32_t seg = 0, nq = 0;  // nq: row tiles of Q before this segment
  int turn = 0;  // the stream whose turn it is
  bool bad = false;
  if (!c.work) return;
  if constexpr (CL) {
    // (every CTA finds the same; the flag ends the other roles' waits)
    if (__any_sync(kFull, batch_refused(p, threadIdx.x - 128)) && lane == 0) {
      record_error(p.status, PA_EINVAL);
      *c.abort = 1;
    }
    __syncwarp();
    asm volatile("bar.sync 3, 256;" ::: "memory");  // both streams' warps have looked
    bad = __any_sync(kFull, *c.abort != 0);
    if (c.own->t1 <= c.own->t0 && threadIdx.x - 128 < c.own->rows)
      reinterpret_cast<float2*>(c.sm + S::kOffML)[threadIdx.x - 128] = make_float2(-INFINITY, 0.f);
  }
  Walk<CL> walk(c, p);
  TreeSegment g;
  for (; walk.next(p, g); ++seg) {
    const bool two = two_tiles(p, g);
    const int nt = g.t1 - g.t0;
    const int skip = two ? 0 : x ^ turn;                  // this stream's first tile
    const int mine = two ? nt : (nt + 1 - skip) >> 1;    // its tiles
    const int other = two ? nt : (nt + skip) >> 1;
    const int tile_row0 = two ? x * p.tile_rows : 0;     // of the item's rows
    const int rows = two ? (x ? g.rows - p.tile_rows : p.tile_rows) : g.rows;
    const bool valid = r < rows;
    const bool idle = 32 * quad >= rows;                 // no row in this warp (uniform)
    const int R = g.row0 + tile_row0 + (valid ? r : 0);
    const int tok = g.qs + R / m.group, h = g.kvh * m.group + R % m.group;
    const int pos = m.window > 0 ? m.positions[tok] : 0;
    float sl = head_scale(m.k_scales, g.kvh, p.scale) * kLog2e;
    const int8_t* exps = reinterpret_cast<const int8_t*>(c.sm + S::kOffExp) +
                         ((nq + (two ? x : 0)) & 3) * 128 + r;
    nq += two ? 2 : 1;
    const int ctx = g.n - g.nodes;
    // keys [free_lo, ctx) are visible to this row whatever its mask says
    const int free_lo = m.window > 0 ? pos - m.window + 1 : 0;
    float m_ref = -INFINITY, l = 0.f;
    uint32_t n = x ? cnt[1] : cnt[0];
    for (int i = 0; i < mine; ++i, ++n) {
      const int key0 = g.kv0 + (g.t0 + (two ? i : 2 * i + skip)) * kBN;
      const uint32_t sb = lanes + col_s(x);
      // a tile that hides keys from some row: which ones, while S is still being computed
      const bool hides = !__all_sync(kFull, key0 >= free_lo && key0 + kBN <= ctx) && !idle;
      uint32_t see[4] = {0, 0, 0, 0};
      if (hides) visible_keys(p, g, tok, pos, key0, see);
      if (!bad)
        bad = !wait_all(c, stall ? B_NEVER : B_SFULL + x, stall ? 0u : n & 1);
      // the row of q was multiplied by 2^exp when it was split (known once its first S is)
      if (FP8 && i == 0) sl *= __uint_as_float((uint32_t)(127 - *exps) << 23);
      // (a product that came to zero would make the hidden keys' -inf a NaN)
      if (i == 0) sl = fmaxf(sl, 1.17549435e-38f);
      if (!idle && !bad) {
        tc_fence_after();
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          uint32_t v[64];
          tmem_ld64(sb + 64 * q, v);
          tmem_wait_ld64(v);
          if (hides) {  // hidden keys' scores become -inf in place
            const uint32_t w0 = q ? see[2] : see[0], w1 = q ? see[3] : see[1];
            uint32_t u[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = v[e] = (w0 >> e) & 1u ? v[e] : 0xff800000u;
            tmem_st32(sb + 64 * q, u);
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = v[32 + e] = (w1 >> e) & 1u ? v[32 + e] : 0xff800000u;
            tmem_st32(sb + 64 * q + 32, u);
          }
#pragma unroll
          for (int e = 0; e < 64; e += 2)
            mx[(e >> 1) & 3] =
                fmaxf(mx[(e >> 1) & 3], fmaxf(__uint_as_float(v[e]), __uint_as_float(v[e + 1])));
        }
        if (hides) tmem_wait_st();
        // (the scale is positive on this path, so it commutes with the max)
        const float m_new = fmaxf(m_ref, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl);
        // (f16 weights are taken 2^7 times as large, up to 2^15: what rounds to a multiple of f16's
        // smallest step is off by 2^-32 of the row's largest weight, not by 2^-25)
        constexpr float kUp = FP8 ? 7.f : 0.f;
        const bool resc = m_new > m_ref + (8.f + kUp);
        float alpha = 1.f;
        if (resc) {
          alpha = fast_exp2(m_ref - (m_new - kUp));  // 0 when nothing was visible before
          m_ref = m_new - kUp;
          l *= alpha;
        }
        const float nb = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t sl2 = f2_pack(sl, sl), nb2 = f2_pack(nb, nb);
        uint64_t sum[2] = {0, 0};
        // P over the S columns it came from, 32 keys at a time (a loop: straight-line code for
        // all 128 keys ran out of the instruction cache and took 1.9 times as long)
        {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t s0[32];
            tmem_ld32(sb + 32 * q, s0);
            tmem_wait_ld(s0);
            weights32<FP8>(sb + 32 * q, s0, sl2, nb2, sum);
          }
        }
        {
          float a, b, d, e;
          f2_unpack(sum[0], a, b);
          f2_unpack(sum[1], d, e);
          l += (a + b) + (d + e);
        }
        // O is rescaled only when a reference moved, after the P V before it is done
        if (i > 0 && __any_sync(kFull, resc)) {
          if (!bad) bad = !wait_all(c, B_PVDONE + x, (n - 1) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(lanes + col_o(x) + 32 * q, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(lanes + col_o(x) + 32 * q, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar + B_PFULL + x);
    }
    cnt[0] += x ? other : mine;
    cnt[1] += x ? mine : other;

    // ---- the segment's end
    const int par = seg & 1;
    if (!two) turn = (turn + nt) & 1;
    if (!two && x == turn) {  // the other stream has the last tile: it gets this one's state
      if (mine) {
        xchg[par * 128 + r] = make_float2(m_ref, l);
        if (lane == 0) bads[par * 4 + quad] = bad ? 1 : 0;
        // (after a failed wait nothing holds this warp back: it must not come round to the same
        // barrier before the other stream has passed it)
        if (bad)
          state_taken(par);
        else
          state_given(par);
      }
      continue;
    }
    if (!bad && mine) bad = !wait_all(c, B_PVDONE + x, (n - 1) & 1);
    const bool join = !two && other > 0;
    if (join) {
      if (!bad) bad = !wait_all(c, B_PVDONE + (x ^ 1), ((x ? cnt[0] : cnt[1]) - 1) & 1);
      state_taken(par);
      bad |= bads[par * 4 + quad] != 0;  // (uniform across the warp)
    }
    // (the state goes over the ring: the other stream's last product has to be done with it)
    if (CL && two && !bad)
      bad = !wait_all(c, B_PVDONE + (x ^ 1), ((x ? cnt[0] : cnt[1]) - 1) & 1);
    // (a failed role's rows must not be written)
    if (!bad && __all_sync(kFull, *c.abort == 0)) {
      tc_fence_after();
      float a0 = 1.f, a1 = 0.f;
      if (join) {
        const float2 o = xchg[par * 128 + r];
        const float mn = fmaxf(m_ref, o.x), base = mn == -INFINITY ? 0.f : mn;
        a0 = fast_exp2(m_ref - base);
        a1 = fast_exp2(o.x - base);
        l = l * a0 + o.y * a1;
        m_ref = mn;
      }
      const int item_row = tile_row0 + r;
      float scale = 1.f;
      float* po = nullptr;
      __nv_bfloat16* out = nullptr;
      if (valid) {
        if (g.slot >= 0) {
          if constexpr (CL) {
            reinterpret_cast<float2*>(c.sm + S::kOffML)[item_row] = make_float2(m_ref, l);
            po = reinterpret_cast<float*>(c.sm + S::kOffState) + item_row * S::kStateLd;
          } else {
            const int64_t at = (int64_t)g.slot * p.rows_per_item + item_row;
            p.part_ml[at] = make_float2(m_ref, l);
            po = p.part_o + at * D;
          }
        } else {
          scale = tree_finish(p, g.kvh, h, tok, m_ref, l, true);
          out = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)tok * m.num_heads + h) * D;
        }
      }
      a0 *= scale;
      a1 *= scale;
      if (!idle) {
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(lanes + col_o(x) + 32 * q, o);
          tmem_wait_ld(o);
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * a0;
          if (join) {
            tmem_ld32(lanes + col_o(x ^ 1) + 32 * q, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] += __uint_as_float(o[e]) * a1;
          }
          if (po) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(po + 32 * q + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
          } else if (out) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(out + 32 * q + e) =
                  make_uint4(pack_bf16x2(f[e], f[e + 1]), pack_bf16x2(f[e + 2], f[e + 3]),
                             pack_bf16x2(f[e + 4], f[e + 5]), pack_bf16x2(f[e + 6], f[e + 7]));
          }
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(c.bar + B_OFREE + x);
      if (!two) mbar_arrive(c.bar + B_OFREE + (x ^ 1));
    }
  }
}

template <int D, bool FP8, bool CL>
__global__ void __launch_bounds__(Shape<D, FP8>::kThreads, 1)
    k_tree_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
              const __grid_constant__ CUtensorMap tv, const TreeParams p, uint64_t wait_limit,
              uint32_t stall) {
  using S = Shape<D, FP8>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::kOffMisc);
  int* flags = reinterpret_cast<int*>(sm + S::kOffMisc + 4);  // [0] skip, [1] abort
  TreeSegment* own = reinterpret_cast<TreeSegment*>(sm + S::kOffSeg);
  static_assert(sizeof(TreeSegment) <= 64, "kOffSeg");
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    flags[1] = 0;
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if ((i >= B_QCONV && i < B_QCONV + 2) || (i >= B_WIDE && i < B_WIDE + 2)) n = 4;
      // e4m3: four warps read V's codes
      if (FP8 && i >= B_EMPTY + kMostStages && i < B_EMPTY + 2 * kMostStages) n = 4;
      if (i >= B_PFULL && i < B_PFULL + 2) n = 4;
      if (i >= B_OFREE && i < B_OFREE + 2) n = 4;
      mbar_init(bar + i, n);
    }
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  fence_mbar_init();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // everything above overlaps the kernel ahead (shares: the planning kernel)
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    // (the swizzled tiles need the 1024-byte alignment that the declaration asks for)
    const bool off = (smem_u32(sm) & 1023u) != 0;
    if (off) record_error(p.status, PA_ECUDA);
    flags[0] = off || status_set(p.status) ? 1 : 0;
  }
  if (CL && warp == 2) plan_own(p, own, threadIdx.x & 31);
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const Ctx c{sm,         bar,        reinterpret_cast<volatile int*>(flags + 1), p.status,
              wait_limit, flags[0] == 0, own};
  const bool joined = CL && p.cluster > 1;  // the cluster's CTAs join their states
  // (a CTA that does nothing tells the others)
  if (CL && !c.work && threadIdx.x == 0) flags[1] = 1;

  // register shares of the warps: bf16 4 x 72 + 8 x 216, e4m3 4 x 72 + 8 x 176 + 4 x 88
  static_assert(4 * 72 + 8 * 216 <= 12 * 168 && 4 * 72 + 8 * 176 + 4 * 88 <= 16 * 128, "registers");
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
    if constexpr (FP8) converter<D, CL>(c, p);
    __syncthreads();
    if (joined) {
      cluster_sync();
      cluster_sync();
    }
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
    if (warp == 0 || warp == 3) {
      producer<D, FP8, CL>(c, p, warp ? &tv : &tk, &tq, warp ? 1 : 0);
    } else {
      if (warp == 1)
        s_issuer<D, FP8, CL>(c, p, tmem);
      else
        pv_issuer<D, FP8, CL>(c, p, tmem);
      __syncwarp();
      // every MMA of this warp is done before the tensor memory goes (bounded)
      mma_commit(bar + B_FIN + (warp - 1));
      if ((threadIdx.x & 31) == 0) mbar_wait(bar + B_FIN + (warp - 1), 0, 1000000000ull);
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (joined) cluster_sync();
    if (warp == 1) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemCols)
                   : "memory");
    }
    if (joined) cluster_sync();
  } else {
    if constexpr (FP8)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 176;" ::: "memory");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
    softmax_role<D, FP8, CL>(c, p, tmem, stall);
    tc_fence_before();
    __syncthreads();
    if (joined) {
      cluster_sync();
      cluster_merge<D, FP8>(c, p);
      cluster_sync();  // every CTA stays until its state has been read
    }
  }
}

template <int D, bool FP8, bool CL>
cudaError_t launch_as(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const TreeParams& p, uint64_t limit, uint32_t stall, cudaStream_t stream) {
  using S = Shape<D, FP8>;
  auto kern = k_tree_tc<D, FP8, CL>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  if constexpr (!CL)
    return launch_pdl(kern, dim3(p.grid), dim3(S::kThreads), S::kSmem, stream, tq, tk, tv, p, limit,
                      stall);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p, limit, stall);
}

template <int D, bool FP8>
int resident(int c) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c);
  cfg.blockDim = dim3(Shape<D, FP8>::kThreads);
  cfg.dynamicSmemBytes = Shape<D, FP8>::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = c;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kern = k_tree_tc<D, FP8, true>;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<D, FP8>::kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

template <int D, bool FP8>
cudaError_t launch_mode(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const TreeParams& p, uint64_t limit, uint32_t stall, cudaStream_t stream) {
  return p.cluster ? launch_as<D, FP8, true>(tq, tk, tv, p, limit, stall, stream)
                   : launch_as<D, FP8, false>(tq, tk, tv, p, limit, stall, stream);
}

}  // namespace

int tree_clusters_resident(int device, bool fp8, int head_dim, int c) {
  // [device][variant][cluster size 2, 4, 8]: number + 1, 0 while it is not known
  static std::atomic<int> known[64][3][3];
  const int variant = fp8 ? 2 : head_dim == 128, at = c == 2 ? 0 : c == 4 ? 1 : 2;
  if (device < 0 || device >= 64) return 0;
  const int k = known[device][variant][at].load(std::memory_order_relaxed);
  if (k) return k - 1;
  const int n = fp8 ? resident<128, true>(c) : variant ? resident<128, false>(c) : resident<64, false>(c);
  known[device][variant][at].store(n + 1, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_tree_tc(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const TreeParams& p, bool fp8, uint64_t wait_limit, uint32_t stall,
                           cudaStream_t stream) {
  if (fp8) return launch_mode<128, true>(tq, tk, tv, p, wait_limit, stall, stream);
  if (p.m.head_dim == 128) return launch_mode<128, false>(tq, tk, tv, p, wait_limit, stall, stream);
  return launch_mode<64, false>(tq, tk, tv, p, wait_limit, stall, stream);
}

}  // namespace pa
