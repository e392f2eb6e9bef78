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
// shared memory serves 256 rows.  An item with one row tile gives its even key tiles to stream 0
// and its odd ones to stream 1, whose states (m, l, O) are joined at the end.  Either way one
// stream's MMAs run while the other's exponentials do.
//
// Per key tile of a stream:  S = Q K^T (M 128, N 128, K = head size);  mask, running max (moved,
// with O rescaled, only when it grows by more than 2^8), p = 2^(s - m);  P written over S;
// O += P V.  Over bf16 pools P is a bf16 pair hi + lo (two products with V, weights good to
// 2^-16); over e4m3 pools it is one f16 value (2^-11), with q, K and V widened to f16 (exactly,
// for the codes) in shared memory.  Row sums add the fp32 weights.
//
// Roles.  warp 0: TMA of K and V through a ring of five 128-key stages, K and V alternating;
// warp 1: tensor-memory owner, issues S = Q K^T; warp 2: issues O += P V, and zeroes the V rows
// past the sequence's end (they may hold anything; K's are masked); warp 3: TMA of Q, a ring of
// two row tiles; warps 4..7 and 8..11: the streams' softmax and epilogue; warps 12..15 (e4m3
// pools): widen Q, K and V in shared memory.
//
// What bounds it: up to 128 rows per kv head, the K / V bytes (a tile is 64 KB of bf16, 1.5 us of
// an SM's share of the measured copy bandwidth, against 1.0 us of tensor time); with two row
// tiles, the tensor cores (2.0 us a tile).
//
// Every mbarrier wait is bounded; one that runs out records PA_ETIMEOUT and raises an abort flag
// that ends the other roles' waits.  The softmax warps meet at a named barrier at the end of each
// segment, where they agree on leaving; the TMA issuers wait (bounded) for their copies in flight
// and the MMA issuers for their MMAs before the CTA gives its tensor memory back.
#include <algorithm>

#include "k_tree.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBN = 128;      // keys per tile
constexpr int kStages = 5;    // K / V ring

template <int D, bool FP8>
struct Shape {
  static constexpr int kHalves = D / 64;            // 64-dim halves of a tile: rows of 128 bytes
  static constexpr int kHalfBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // a 128-row tile of 16-bit values
  static constexpr int kLoadBytes = FP8 ? kTileBytes / 2 : kTileBytes;
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffX = kOffKV + kStages * kTileBytes;  // [2][128] float2: stream 1's m, l
  static constexpr int kOffBad = kOffX + 2 * 128 * 8;          // [2][8] failed-wait flags
  static constexpr int kOffBar = kOffBad + 2 * 8 * 4;
  static constexpr int kOffMisc = kOffBar + 40 * 8;
  static constexpr int kSmem = kOffMisc + 16;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

// barriers (indices of consecutive 8-byte words)
enum : int {
  B_QFULL = 0,                     // Q buffer landed
  B_QEMPTY = B_QFULL + 2,          // its last S = Q K^T is done
  B_QCONV = B_QEMPTY + 2,          // e4m3: its f16 form is ready
  B_FULL = B_QCONV + 2,            // K / V stage landed
  B_EMPTY = B_FULL + kStages,
  B_CONV = B_EMPTY + kStages,      // e4m3: the stage's f16 form is ready
  B_SFULL = B_CONV + kStages,      // per stream: S is ready
  B_PFULL = B_SFULL + 2,           // P is written
  B_PVDONE = B_PFULL + 2,          // P V is done: O is current, the S / P buffer is free
  B_OFREE = B_PVDONE + 2,          // the segment's O has been read
  B_FIN = B_OFREE + 2,
  B_NEVER = B_FIN + 2,             // nothing arrives on it (the debug_stall test hook)
  kNumBars = B_NEVER + 1
};
static_assert(kNumBars <= 40, "barrier area");

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int x) { return (uint32_t)x * 128; }
__device__ __forceinline__ uint32_t col_o(int x) { return 256 + (uint32_t)x * 128; }

// One CTA's MMAs (cta_group::1), issued by lane 0 of a warp in uniform control flow.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .u32 l;\n\t.reg .pred e, p;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .u32 l;\n\t.reg .pred e, p;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
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
};

__device__ __forceinline__ bool wait_bar(const Ctx& c, int idx, uint32_t parity) {
  uint64_t* b = c.bar + idx;
  if (mbar_try_wait(b, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(b, parity)) return true;
    if ((i & 31u) == 0) {
      if (*c.abort) return false;
      if (globaltimer_ns() - t0 > c.limit) {
        record_error(c.status, PA_ETIMEOUT);
        *c.abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_all(const Ctx& c, int idx, uint32_t parity) {
  return __all_sync(kFull, wait_bar(c, idx, parity));
}

// Position in the K / V ring.
struct Ring {
  uint32_t st = 0, par = 0;
  __device__ __forceinline__ void next() {
    if (++st == kStages) {
      st = 0;
      par ^= 1;
    }
  }
};

// Tiles of stream x in a segment of nt key tiles: both streams all of them (two row tiles), or
// the even and the odd ones.
__device__ __forceinline__ bool two_tiles(const TreeParams& p, const TreeSegment& g) {
  return g.rows > p.tile_rows;
}

// ---- roles --------------------------------------------------------------------------------------

template <int D, bool FP8>
__device__ void kv_producer(const Ctx& c, const TreeParams& p, const CUtensorMap* tk,
                            const CUtensorMap* tv) {
  using S = Shape<D, FP8>;
  const int lane = threadIdx.x & 31;
  constexpr int kBoxes = FP8 ? 8 : 8 * S::kHalves;  // one box per lane
  const int blk = lane & 7, half = lane >> 3;
  Ring r;
  uint32_t issued = 0;
  bool ok = c.work;
  TreeWalk walk(p, blockIdx.x);
  TreeSegment g;
  while (ok && walk.next(p, g)) {
    const int32_t* row = p.m.block_tables + (int64_t)g.s * p.m.max_blocks;
    const int blocks = (g.n + 15) / 16;
    const int b0 = g.kv0 / 16 + 8 * g.t0 + blk;
    int next = b0 < blocks ? row[b0] : -1;
    for (int j = g.t0; ok && j < g.t1; ++j) {
      const int id = next;
      const int nb = b0 + 8 * (j + 1 - g.t0);
      if (j + 1 < g.t1) next = nb < blocks ? row[nb] : -1;
      const int coord = id >= 0 ? id * 16 : -16;  // past the end: rows outside the pool, zeros
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (lane == 0) {
          ok = wait_bar(c, B_EMPTY + r.st, r.par ^ 1);
          if (ok) mbar_arrive_expect_tx(c.bar + B_FULL + r.st, S::kLoadBytes);
        }
        ok = __shfl_sync(kFull, (int)ok, 0);
        if (!ok) break;
        if (lane < kBoxes) {
          uint8_t* dst = c.sm + S::kOffKV + r.st * S::kTileBytes;
          if constexpr (FP8)  // the codes go where the second dim half's rows will be
            tma_load_3d(dst + S::kHalfBytes + blk * 2048, kv ? tv : tk, 0, g.kvh, coord,
                        c.bar + B_FULL + r.st);
          else
            tma_load_3d(dst + half * S::kHalfBytes + blk * 2048, kv ? tv : tk, 64 * half, g.kvh,
                        coord, c.bar + B_FULL + r.st);
        }
        ++issued;
        r.next();
      }
    }
  }
  // the copies still in flight (after an abort; otherwise all have been consumed)
  if (lane == 0)
    for (uint32_t k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
      mbar_wait(c.bar + B_FULL + k % kStages, (k / kStages) & 1u, c.limit);
  __syncwarp();
}

template <int D, bool FP8>
__device__ void q_producer(const Ctx& c, const TreeParams& p, const CUtensorMap* tq) {
  using S = Shape<D, FP8>;
  const int lane = threadIdx.x & 31;
  uint32_t n = 0;  // row tiles loaded; tile n uses buffer n % 2
  bool ok = c.work;
  TreeWalk walk(p, blockIdx.x);
  TreeSegment g;
  while (ok && walk.next(p, g)) {
    const int tiles = two_tiles(p, g) ? 2 : 1;
    for (int x = 0; ok && x < tiles; ++x) {
      if (lane == 0) {
        ok = wait_bar(c, B_QEMPTY + (n & 1), ((n >> 1) & 1) ^ 1);
        if (ok) {
          uint64_t* bar = c.bar + B_QFULL + (n & 1);
          mbar_arrive_expect_tx(bar, (uint32_t)p.tile_rows * 128 * S::kHalves);
          const int tok = g.qs + (g.row0 + x * p.tile_rows) / p.m.group;
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
            tma_load_3d(c.sm + (n & 1) * S::kTileBytes + h * S::kHalfBytes, tq, 64 * h,
                        g.kvh * p.m.group, tok, bar);
        }
      }
      ok = __shfl_sync(kFull, (int)ok, 0);
      if (ok) ++n;
    }
  }
  if (lane == 0)
    for (uint32_t k = n > 2 ? n - 2 : 0; k < n; ++k)
      mbar_wait(c.bar + B_QFULL + (k & 1), (k >> 1) & 1u, c.limit);
  __syncwarp();
}

template <int D, bool FP8>
__device__ void s_issuer(const Ctx& c, const TreeParams& p, uint32_t tmem) {
  using S = Shape<D, FP8>;
  constexpr uint32_t kIdesc = idesc_f16kind(128, kBN, 0, FP8 ? 0 : 1);
  constexpr int kQ = FP8 ? B_QCONV : B_QFULL, kKV = FP8 ? B_CONV : B_FULL;
  const uint32_t sm = smem_u32(c.sm);
  Ring r;
  uint32_t nq = 0, cnt[2] = {0, 0};  // row tiles used; tiles of each stream
  if (!c.work) return;
  TreeWalk walk(p, blockIdx.x);
  TreeSegment g;
  while (walk.next(p, g)) {
    const bool two = two_tiles(p, g);
    for (int j = g.t0; j < g.t1; ++j) {
      if (!wait_all(c, kKV + r.st, r.par)) return;
      const uint32_t kb = sm + S::kOffKV + r.st * S::kTileBytes;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int x = two ? y : (j - g.t0) & 1;  // the stream
        if (!two && y) break;
        const uint32_t q = nq + (two ? y : 0);
        if (j == g.t0 && !wait_all(c, kQ + (q & 1), (q >> 1) & 1)) return;
        const uint32_t n = x ? cnt[1] : cnt[0];
        if (!wait_all(c, B_PVDONE + x, (n & 1) ^ 1)) return;  // the buffer's last P is used up
        tc_fence_after();
        const uint32_t qb = sm + (q & 1) * S::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + col_s(x), sdesc(qb + (kk >> 2) * S::kHalfBytes + (kk & 3) * 32, 16, 1024),
                 sdesc(kb + (kk >> 2) * S::kHalfBytes + (kk & 3) * 32, 16, 1024), kIdesc,
                 kk > 0 ? 1u : 0u);
        mma_commit(c.bar + B_SFULL + x);
        if (x) ++cnt[1]; else ++cnt[0];
      }
      mma_commit(c.bar + B_EMPTY + r.st);
      __syncwarp();
      r.next();
      r.next();  // V's stage
    }
    for (int y = 0; y < (two ? 2 : 1); ++y) mma_commit(c.bar + B_QEMPTY + ((nq + y) & 1));
    nq += two ? 2 : 1;
  }
}

template <int D, bool FP8>
__device__ void pv_issuer(const Ctx& c, const TreeParams& p, uint32_t tmem) {
  using S = Shape<D, FP8>;
  constexpr uint32_t kIdesc = idesc_f16kind(128, D, 1, FP8 ? 0 : 1);
  constexpr int kKV = FP8 ? B_CONV : B_FULL;
  const int lane = threadIdx.x & 31;
  const uint32_t sm = smem_u32(c.sm);
  Ring r;
  uint32_t cnt[2] = {0, 0}, seg = 0;
  if (!c.work) return;
  TreeWalk walk(p, blockIdx.x);
  TreeSegment g;
  for (; walk.next(p, g); ++seg) {
    const bool two = two_tiles(p, g);
    for (int j = g.t0; j < g.t1; ++j) {
      r.next();  // K's stage
      if (!wait_all(c, kKV + r.st, r.par)) return;
      uint8_t* v = c.sm + S::kOffKV + r.st * S::kTileBytes;
      if constexpr (!FP8) {  // (the converters do it over e4m3 pools)
        // rows of the last block past the sequence's end: zeros (whole blocks past it are)
        const int lim = g.n - (g.kv0 + j * kBN);
        if (lim < kBN && (lim & 15)) {
          const int rows = 16 - (lim & 15);
          for (int i = lane; i < rows * 8 * S::kHalves; i += 32) {
            const int h = i / (rows * 8), e = i % (rows * 8);
            *reinterpret_cast<uint4*>(v + h * S::kHalfBytes + lim * 128 + e * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      const uint32_t vb = smem_u32(v);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int x = two ? y : (j - g.t0) & 1;
        if (!two && y) break;
        const bool first = two ? j == g.t0 : j - g.t0 < 2;
        if (first && !wait_all(c, B_OFREE + x, (seg & 1) ^ 1)) return;
        const uint32_t n = x ? cnt[1] : cnt[0];
        if (!wait_all(c, B_PFULL + x, n & 1)) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk) {
          const uint64_t vd = sdesc(vb + kk * 2048, S::kHalfBytes, 1024);
          mma_ts(tmem + col_o(x), tmem + col_s(x) + kk * 8, vd, kIdesc,
                 (!first || kk > 0) ? 1u : 0u);
          if constexpr (!FP8) mma_ts(tmem + col_o(x), tmem + col_s(x) + 64 + kk * 8, vd, kIdesc, 1u);
        }
        mma_commit(c.bar + B_PVDONE + x);
        if (x) ++cnt[1]; else ++cnt[0];
      }
      mma_commit(c.bar + B_EMPTY + r.st);
      __syncwarp();
      r.next();
    }
  }
}

// Widen a staged tile of 128 x 128 codes to f16, in place: the codes lie in the second dim half's
// 16 KB, in rows of 128 bytes with the 128-byte swizzle; warp w takes blocks 2w and 2w + 1.  A
// round's stores overwrite only codes of its own four rows, loaded by all lanes before.  Rows at
// or past `lim` become zeros.
__device__ __forceinline__ void widen_tile(uint8_t* tile, int w, int lane, int lim) {
  constexpr int kHalf = 128 * 128;
#pragma unroll 2
  for (int i = 0; i < 8; ++i) {
    const int b = 2 * w + (i >> 2), ch = lane + 32 * (i & 3);
    const uint4 src = *reinterpret_cast<const uint4*>(tile + kHalf + b * 2048 + ch * 16);
    __syncwarp();
    const int rr = ch >> 3, L = (ch & 7) ^ (rr & 7);  // row of the block, dims 16 L .. 16 L + 15
    const int h = L >> 2, c0 = 2 * (L & 3);           // dim half, first output chunk
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (b * 16 + rr < lim) {
      widen4(src.x, lo.x, lo.y);
      widen4(src.y, lo.z, lo.w);
      widen4(src.z, hi.x, hi.y);
      widen4(src.w, hi.z, hi.w);
    }
    uint8_t* row = tile + h * kHalf + b * 2048 + rr * 128;
    *reinterpret_cast<uint4*>(row + ((c0 ^ (rr & 7)) << 4)) = lo;
    *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (rr & 7)) << 4)) = hi;
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <int D>
__device__ void converter(const Ctx& c, const TreeParams& p) {
  using S = Shape<D, true>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 12;
  Ring r;
  uint32_t nq = 0;
  if (!c.work) return;
  TreeWalk walk(p, blockIdx.x);
  TreeSegment g;
  while (walk.next(p, g)) {
    const int tiles = two_tiles(p, g) ? 2 : 1;
    for (int x = 0; x < tiles; ++x, ++nq) {
      if (!wait_all(c, B_QFULL + (nq & 1), (nq >> 1) & 1)) return;
      uint4* q = reinterpret_cast<uint4*>(c.sm + (nq & 1) * S::kTileBytes) + w * (S::kTileBytes / 64);
#pragma unroll 4
      for (int i = 0; i < S::kTileBytes / 64 / 32; ++i) {
        uint4 v = q[lane + 32 * i];
        v.x = bf16x2_to_f16x2(v.x);
        v.y = bf16x2_to_f16x2(v.y);
        v.z = bf16x2_to_f16x2(v.z);
        v.w = bf16x2_to_f16x2(v.w);
        q[lane + 32 * i] = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar + B_QCONV + (nq & 1));
    }
    for (int j = g.t0; j < g.t1; ++j) {
      const int lim = g.n - (g.kv0 + j * kBN);
      for (int kv = 0; kv < 2; ++kv) {
        if (!wait_all(c, B_FULL + r.st, r.par)) return;
        widen_tile(c.sm + S::kOffKV + r.st * S::kTileBytes, w, lane, lim);
        if (lane == 0) mbar_arrive(c.bar + B_CONV + r.st);
        r.next();
      }
    }
  }
}

// Visible keys of one row in the 32 positions from key0 on.
__device__ __forceinline__ uint32_t visible_word(const TreeParams& p, const TreeSegment& g, int tok,
                                                 int pos, int key0) {
  const int ctx = g.n - g.nodes;
  uint32_t w = 0;
  if (key0 < ctx) {  // context positions from pos - window + 1 on
    const int hi = min(32, ctx - key0);
    w = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
    if (p.m.window > 0) {
      const int lo = pos - p.m.window + 1 - key0;
      w = lo >= 32 ? 0u : lo > 0 ? w & (0xffffffffu << lo) : w;
    }
  }
  const int node0 = key0 - ctx;  // node of bit 0
  if (node0 > -32 && node0 < g.nodes) {
    const int32_t* row = p.mask + (int64_t)tok * p.mask_words;
    uint32_t t;
    if (node0 < 0) {
      t = (uint32_t)row[0] << -node0;
    } else {
      const int i = node0 >> 5, s = node0 & 31;
      const uint32_t a = (uint32_t)row[i], b = i + 1 < p.mask_words ? (uint32_t)row[i + 1] : 0u;
      t = __funnelshift_r(a, b, s);
    }
    const int end = g.nodes - node0;  // bits from there on are past the tree
    if (end < 32) t &= (1u << end) - 1u;
    if (p.m.window > 0)
      for (uint32_t m = t; m; m &= m - 1) {
        const int i = __ffs(m) - 1;
        if (p.m.positions[g.qs + node0 + i] <= pos - p.m.window) t &= ~(1u << i);
      }
    w |= t;
  }
  return w;
}

__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

// The streams' threads: warpgroup x (warps 4 + 4x ..), thread = row = tensor-memory lane.
template <int D, bool FP8>
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
  uint32_t seg = 0;
  bool bad = false;
  if (!c.work) return;
  TreeWalk walk(p, blockIdx.x);
  TreeSegment g;
  for (; walk.next(p, g); ++seg) {
    const bool two = two_tiles(p, g);
    const int nt = g.t1 - g.t0;
    const int mine = two ? nt : (nt + 1 - x) >> 1;       // this stream's tiles
    const int other = two ? nt : (nt + x) >> 1;
    const int tile_row0 = two ? x * p.tile_rows : 0;     // of the item's rows
    const int rows = two ? (x ? g.rows - p.tile_rows : p.tile_rows) : g.rows;
    const bool valid = r < rows;
    const bool idle = 32 * quad >= rows;                 // no row in this warp (uniform)
    const int R = g.row0 + tile_row0 + (valid ? r : 0);
    const int tok = g.qs + R / m.group, h = g.kvh * m.group + R % m.group;
    const int pos = m.window > 0 ? m.positions[tok] : 0;
    const float sl = head_scale(m.k_scales, g.kvh, p.scale) * kLog2e;
    const int ctx = g.n - g.nodes;
    // keys [free_lo, ctx) are visible to this row whatever its mask says
    const int free_lo = m.window > 0 ? pos - m.window + 1 : 0;
    float m_ref = -INFINITY, l = 0.f;
    uint32_t n = x ? cnt[1] : cnt[0];
    for (int i = 0; i < mine; ++i, ++n) {
      const int key0 = g.kv0 + (g.t0 + (two ? i : 2 * i + x)) * kBN;
      const uint32_t sb = lanes + col_s(x);
      if (!bad)
        bad = !wait_all(c, stall ? B_NEVER : B_SFULL + x, stall ? 0u : n & 1);
      if (!idle && !bad) {
        tc_fence_after();
        float v[kBN];
        {
          uint32_t a[64], b[64];
          tmem_ld64(sb, a);
          tmem_ld64(sb + 64, b);
          tmem_wait_ld64(a);
          tmem_wait_ld64(b);
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            v[e] = __uint_as_float(a[e]);
            v[64 + e] = __uint_as_float(b[e]);
          }
        }
        if (!__all_sync(kFull, key0 >= free_lo && key0 + kBN <= ctx)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t w = visible_word(p, g, tok, pos, key0 + 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              v[32 * q + e] = (w >> e) & 1u ? v[32 * q + e] : -INFINITY;
          }
        }
        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int e = 4; e < kBN; e += 4) {
          mx[0] = fmaxf(mx[0], v[e]);
          mx[1] = fmaxf(mx[1], v[e + 1]);
          mx[2] = fmaxf(mx[2], v[e + 2]);
          mx[3] = fmaxf(mx[3], v[e + 3]);
        }
        // (the scale is positive on this path, so it commutes with the max)
        const float m_new = fmaxf(m_ref, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl);
        const bool resc = m_new > m_ref + 8.f;
        float alpha = 1.f;
        if (resc) {
          alpha = fast_exp2(m_ref - m_new);  // 0 when nothing was visible before
          m_ref = m_new;
          l *= alpha;
        }
        const float nb = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t sl2 = f2_pack(sl, sl), nb2 = f2_pack(nb, nb);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // 64 keys at a time: P over their S columns
          uint32_t ph[32], pl[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int k = 64 * part + 2 * e;
            float a, b;
            f2_unpack(f2_fma(f2_pack(v[k], v[k + 1]), sl2, nb2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum[e & 1] = f2_add(sum[e & 1], f2_pack(a, b));
            if constexpr (FP8) {
              ph[e] = pack_f16x2(a, b);
            } else {
              ph[e] = pack_bf16x2(a, b);
              pl[e] = pack_bf16x2(a - __uint_as_float(ph[e] << 16),
                                  b - __uint_as_float(ph[e] & 0xffff0000u));
            }
          }
          tmem_st32(sb + 32 * part, ph);
          if constexpr (!FP8) tmem_st32(sb + 64 + 32 * part, pl);
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
#pragma unroll
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
    // both streams' last P V, as far as this warpgroup reads their O
    if (!bad && mine) bad = !wait_all(c, B_PVDONE + x, (n - 1) & 1);
    if (!two && x == 0 && other) {
      if (!bad) bad = !wait_all(c, B_PVDONE + 1, (cnt[1] - 1) & 1);
    }
    if (!two && x == 1) xchg[par * 128 + r] = make_float2(m_ref, l);
    if (lane == 0) bads[par * 8 + warp] = bad ? 1 : 0;
    softmax_sync();
    int any = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) any |= bads[par * 8 + e];
    if (any) return;  // all eight warps alike, before anything is written
    if (two || x == 0) {
      tc_fence_after();
      float a0 = 1.f, a1 = 0.f;
      const bool join = !two && other > 0;
      if (join) {  // stream 1's state
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
          const int64_t at = (int64_t)g.slot * p.rows_per_item + item_row;
          p.part_ml[at] = make_float2(m_ref, l);
          po = p.part_o + at * D;
        } else {
          scale = tree_finish(p, g.kvh, h, tok, m_ref, l, true);
          out = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)tok * m.num_heads + h) * D;
        }
      }
      a0 *= scale;
      a1 *= scale;
      if (!idle) {
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(lanes + col_o(x) + 32 * q, o);
          tmem_wait_ld(o);
          float f[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * a0;
          if (join) {
            tmem_ld32(lanes + col_o(1) + 32 * q, o);
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
    if (lane == 0) {  // (a stream's next O waits for all eight warps, whoever read it)
      mbar_arrive(c.bar + B_OFREE);
      mbar_arrive(c.bar + B_OFREE + 1);
    }
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Shape<D, FP8>::kThreads, 1)
    k_tree_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
              const __grid_constant__ CUtensorMap tv, const TreeParams p, uint64_t wait_limit,
              uint32_t stall) {
  using S = Shape<D, FP8>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::kOffMisc);
  int* flags = reinterpret_cast<int*>(sm + S::kOffMisc + 4);  // [0] skip, [1] abort
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    flags[1] = 0;
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if ((i >= B_QCONV && i < B_QCONV + 2) || (i >= B_CONV && i < B_CONV + kStages)) n = 4;
      if (i >= B_PFULL && i < B_PFULL + 2) n = 4;
      if (i >= B_OFREE && i < B_OFREE + 2) n = 8;
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
  // everything above overlaps the planning kernel
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    // (the swizzled tiles need the 1024-byte alignment that the declaration asks for)
    const bool off = (smem_u32(sm) & 1023u) != 0;
    if (off) record_error(p.status, PA_ECUDA);
    flags[0] = off || status_set(p.status) ? 1 : 0;
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const Ctx c{sm, bar, reinterpret_cast<volatile int*>(flags + 1), p.status, wait_limit,
              flags[0] == 0};

  // register shares: bf16 4 x 72 + 8 x 216, e4m3 4 x 64 + 8 x 184 + 4 x 80 warps' worth
  static_assert(4 * 72 + 8 * 216 <= 12 * 168 && 4 * 64 + 8 * 184 + 4 * 80 <= 16 * 128, "registers");
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" ::: "memory");
    if constexpr (FP8) converter<D>(c, p);
    __syncthreads();
  } else if (warp < 4) {
    if constexpr (FP8)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
    if (warp == 0) {
      kv_producer<D, FP8>(c, p, &tk, &tv);
    } else if (warp == 3) {
      q_producer<D, FP8>(c, p, &tq);
    } else {
      if (warp == 1)
        s_issuer<D, FP8>(c, p, tmem);
      else
        pv_issuer<D, FP8>(c, p, tmem);
      __syncwarp();
      // every MMA of this warp is done before the tensor memory goes (bounded)
      mma_commit(bar + B_FIN + (warp - 1));
      if ((threadIdx.x & 31) == 0) mbar_wait(bar + B_FIN + (warp - 1), 0, 1000000000ull);
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemCols)
                   : "memory");
    }
  } else {
    if constexpr (FP8)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 184;" ::: "memory");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
    softmax_role<D, FP8>(c, p, tmem, stall);
    tc_fence_before();
    __syncthreads();
  }
}

template <int D, bool FP8>
cudaError_t launch_as(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const TreeParams& p, uint64_t limit, uint32_t stall, cudaStream_t stream) {
  using S = Shape<D, FP8>;
  auto kern = k_tree_tc<D, FP8>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.grid), dim3(S::kThreads), S::kSmem, stream, tq, tk, tv, p, limit,
                    stall);
}

}  // namespace

cudaError_t launch_tree_tc(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const TreeParams& p, bool fp8, uint64_t wait_limit, uint32_t stall,
                           cudaStream_t stream) {
  if (fp8) return launch_as<128, true>(tq, tk, tv, p, wait_limit, stall, stream);
  if (p.m.head_dim == 128) return launch_as<128, false>(tq, tk, tv, p, wait_limit, stall, stream);
  return launch_as<64, false>(tq, tk, tv, p, wait_limit, stall, stream);
}

}  // namespace pa
