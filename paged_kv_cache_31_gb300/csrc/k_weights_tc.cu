// k_weights_tc.cu -- the attention weight that every cached key receives (k_key_weights.cu has the
// formula and the general kernel), on the 5th-generation tensor cores: bf16 queries over bf16 (head size
// 64 / 128) or e4m3 (128) pools of 16-position blocks.
//
// Math.  With the attention's log-sum-exps at hand a weight needs no running maximum: exp(s - lse) is
// final, so only S is computed again, a third of the attention's products over bf16 pools (which
// multiplies V by both terms of P).  It is taken transposed, S^T = K Q^T: keys are the rows of the
// accumulator, a key is a thread, and the sum over the queries stays in its registers: no exchange, no
// atomics, one add to memory for a key in the end.  -lse is added by the products, too: a row's, divided by
// the scale, as three bf16 whose sum it is, times ones (each thread reading the rows' numbers from shared
// memory kept that busy for a third of the time).
//
// Work.  An item is 256 keys of one (sequence, kv head), which stay in tensor memory, against the row
// tiles (128 rows: whole tokens times the group's heads) that see any of them, which stream past.  The
// items' row tiles, laid end to end with a weight for an item's keys, are cut evenly over one CTA per SM;
// the pieces of a cut item leave partial sums, which k_weights_join adds in order.
//
// Roles.  warp 0: TMA of K (256 keys) and Q (a ring of three row tiles); warp 1: tensor-memory owner,
// issues S^T; warp 2: the rows' log-sum-exps into the ring and their positions; warps 4..19: exponentials
// and sums, two warpgroups for 128 keys each, which take the row tiles in turn, from three S^T buffers (half of
// every row tile to each: 9 us more; one warpgroup for 128 keys left the schedulers idle half of the time); at
// an item's start they take K from shared to tensor memory, e4m3 codes widened to bf16 exactly.
//
// What bounds it: three buffers.  A row tile of a prompt of 8191 tokens (8 x 4 heads, 237 us in all) takes some
// 1900 cycles, of which its products take 1150, its 32768 exponentials 1024 of the SFU and its instructions
// 1100 of the schedulers; but a buffer is held by the products into it, a wait, and half of its sums.  K from
// shared memory, a fourth buffer, with log-sum-exps read by each thread: 275 us, shared memory four fifths
// busy.  Tried without gain: two issuing warps, a look at the next tile's waits between products, 32 columns
// loaded while the 32 before are summed (311: the buffers are held longer).
#include <algorithm>

#include "k_tree.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kKeys = kWeightKeys;  // of an item
constexpr int kRows = 128;          // of a row tile, at most
constexpr int kPos = 8;             // ring of the rows' positions
constexpr int kQueries = 3;         // ring of row tiles: queries and log-sum-exps
constexpr int kSums = 3;            // S^T buffers (128 keys, a row tile) in tensor memory, then K
constexpr uint32_t kColK = kSums * kRows;

template <int D, bool FP8>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;  // 128 rows of 16-bit values
  static constexpr int kThreads = 640;
  static constexpr int kHalf = FP8 ? 128 * 128 : kTile;  // of a stage: 128 keys as the pool has them
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kOffK + 2 * kHalf;
  // 128 rows of 64 bf16: 16 of a row for each of the ring's stages (its log-sum-exp), then K's ones
  static constexpr int kOffLse = kOffQ + kQueries * kTile;
  static_assert(kQueries == 3, "the stages and the ones fill a row");
  static constexpr int kOffPos = kOffLse + 128 * 128;          // [kPos][128]
  static constexpr int kOffInfo = kOffPos + kPos * kRows * 4;  // [kPos] int4
  static constexpr int kOffHalf = kOffInfo + kPos * 16;  // [key half][128]: sums of the second warpgroups
  static constexpr int kOffBar = kOffHalf + 2 * 128 * 4;
  static constexpr int kOffMisc = kOffBar + 40 * 8;
  static constexpr int kSmem = kOffMisc + 16;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

enum : int {
  B_KFULL = 0,              // K's keys (or codes) landed
  B_KEMPTY = B_KFULL + 1,   // they have been read
  B_KREADY = B_KEMPTY + 1,  // K is in tensor memory
  B_KDONE = B_KREADY + 1,   // all its products are done
  B_QFULL = B_KDONE + 1,        // a row tile's queries landed, its numbers are there
  B_QEMPTY = B_QFULL + kQueries,
  B_SFULL = B_QEMPTY + kQueries,  // [key half][warpgroup][its tiles in turn]
  B_SFREE = B_SFULL + 8,          // of a buffer
  B_PFREE = B_SFREE + kSums,    // positions have been read
  B_HALF = B_PFREE + kPos,  // per key half: the second warpgroup's sums are there
  B_TAKEN = B_HALF + 2,     // they have been added
  B_FIN = B_TAKEN + 2,
  B_NEVER = B_FIN + 1,  // nothing arrives on it (the debug_stall test hook)
  kNumBars = B_NEVER + 1
};
static_assert(kNumBars <= 40, "barrier area");

constexpr uint32_t kTmemCols = 512;

// Whole warp, in uniform control flow; lane 0 issues.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .u32 l;\n\t.reg .pred e, p;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Same with A in tensor memory (row r in lane r, two values to a column).
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t at, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .u32 l;\n\t.reg .pred e, p;\n\tmov.u32 l, %%laneid;\n\tsetp.eq.u32 e, l, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(at), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {  // whole warp; arrives once its MMAs are done
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

// A counter of a ring's stages: stage and parity of the current use.
template <int N>
struct Ring {
  uint32_t st = 0, par = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      par ^= 1;
    }
  }
};

// One CTA's piece of an item: row tiles [r0, r1) of the sequence's counted rows.
struct Piece {
  int s, kvh, key0, keys;  // keys that the sequence has there
  int qs, tokens;          // first counted token, their number
  int r0, r1;
  int slot;  // of its partial sums, or -1: the item is whole
};

struct Walk {
  int4 at, end;  // (sequence, kv head, item, row tile) where the next piece begins, the share ends
  int slot;
  __device__ __forceinline__ Walk(const TreeParams& p, int cta) {
    at = p.w.starts[cta];
    end = p.w.starts[cta + 1];
    slot = 2 * cta;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, Piece& g) {
    if (at.x >= p.m.num_seqs) return false;
    int4 q = p.w.seqs[2 * at.x];
    while (q.y == 0) {  // sequences without items
      if (++at.x >= p.m.num_seqs) return false;
      q = p.w.seqs[2 * at.x];
    }
    const int4 t = p.w.seqs[2 * at.x + 1];
    const int4 it = p.w.items[q.x + at.z];
    const bool last = at.x == end.x && at.y == end.y && at.z == end.z;
    g.s = at.x;
    g.kvh = at.y;
    g.key0 = it.x * kKeys;
    g.keys = min(kKeys, t.z - g.key0);
    g.qs = t.x;
    g.tokens = t.y;
    g.r0 = at.w;
    g.r1 = last ? end.w : it.z;
    if (g.r1 <= g.r0) return false;
    g.slot = at.w > it.y || g.r1 < it.z ? slot : -1;
    slot |= 1;  // a share's first piece has the even slot
    if (last) {
      at.x = p.m.num_seqs;
    } else {
      if (++at.z == q.y) {
        at.z = 0;
        if (++at.y == p.m.num_kv_heads) {
          at.y = 0;
          do {
            if (++at.x >= p.m.num_seqs) return true;
            q = p.w.seqs[2 * at.x];
          } while (q.y == 0);
        }
      }
      at.w = p.w.items[q.x + at.z].y;
    }
    return true;
  }
};

template <int D, bool FP8>
__device__ void producer(const Ctx& c, const TreeParams& p, const CUtensorMap* tk, const CUtensorMap* tq) {
  using S = Shape<D, FP8>;
  const int lane = threadIdx.x & 31;
  Ring<1> k;
  Ring<kQueries> q;
  uint32_t nk = 0, nq = 0;  // stages issued
  bool ok = true;
  Walk walk(p, blockIdx.x);
  Piece g;
  while (ok && walk.next(p, g)) {
    // 16 blocks: a lane each.  Blocks that no counted token reaches may have any entry, and what they
    // give is not used; those outside the pool (or past the end) are taken from outside, as zeros.
    const int32_t* row = p.m.block_tables + (int64_t)g.s * p.m.max_blocks;
    int id = -1;
    if (lane < 16 && 16 * lane < g.keys) {
      id = row[g.key0 / 16 + lane];
      if (id < 0 || (int64_t)id >= p.m.num_blocks) id = -1;
    }
    const int halves = g.keys > 128 ? 2 : 1;
    if (lane == 0) {
      if (nk >= 1) ok = wait_bar(c, B_KEMPTY, k.par ^ 1);
      if (ok) mbar_arrive_expect_tx(c.bar + B_KFULL, halves * S::kHalf);
    }
    ok = __shfl_sync(kFull, (int)ok, 0);
    if (!ok) break;
    if (lane < 8 * halves) {
      if constexpr (FP8)
        tma_load_3d(c.sm + S::kOffK + lane * 2048, tk, 0, g.kvh, id >= 0 ? id * 16 : -16, c.bar + B_KFULL);
      else
        tma_load_5d(c.sm + S::kOffK + lane * (S::kTile / 8), tk, 0, 0, 0, id >= 0 ? id * 2 : -2, g.kvh,
                    c.bar + B_KFULL);
    }
    ++nk;
    k.next();
    if (lane == 0) {
      for (int r = g.r0; ok && r < g.r1; ++r) {
        if (nq >= kQueries) ok = wait_bar(c, B_QEMPTY + q.st, q.par ^ 1);
        if (!ok) break;
        uint64_t* bar = c.bar + B_QFULL + q.st;
        mbar_arrive_expect_tx(bar, (uint32_t)p.tile_rows * 128 * S::kHalves);
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h)
          tma_load_3d(c.sm + S::kOffQ + q.st * S::kTile + h * 128 * 128, tq, 64 * h,
                      g.kvh * p.m.group, g.qs + r * p.tile_tokens, bar);
        ++nq;
        q.next();
      }
    }
    ok = __shfl_sync(kFull, (int)ok, 0);
  }
  // the copies still in flight (after an abort; otherwise all have been consumed)
  if (lane == 0) {
    if (nk > 0) mbar_wait(c.bar + B_KFULL, (nk - 1) & 1, c.limit);
    for (uint32_t i = nq > kQueries ? nq - kQueries : 0; i < nq; ++i)
      mbar_wait(c.bar + B_QFULL + i % kQueries, i / kQueries & 1, c.limit);
  }
  __syncwarp();
}

// Tile `tile` of a key half goes to warpgroup tile & 1 of the half, as its tile number tile / 2.
__device__ __forceinline__ int sum_bar(int x, uint32_t tile) {
  return B_SFULL + 4 * x + 2 * (tile & 1) + ((tile >> 1) & 1);
}

template <int D, bool FP8>
__device__ void issuer(const Ctx& c, const TreeParams& p, uint32_t tmem_base) {
  using S = Shape<D, FP8>;
  constexpr uint32_t kIdesc = idesc_f16kind(128, kRows, 0, 1);
  const uint32_t sm = smem_u32(c.sm);
  Ring<1> k;
  Ring<kQueries> q;
  Ring<kSums> s;
  uint32_t n = 0, tiles[2] = {0, 0};  // S^T tiles so far; of each key half
  const uint32_t tmem = __shfl_sync(kFull, tmem_base, 0);
  const uint64_t ones = sdesc(sm + S::kOffLse + kQueries * 32, 16, 1024);
  Walk walk(p, blockIdx.x);
  Piece g;
  while (walk.next(p, g)) {
    // (one value for the warp, as the compiler can see: in control flow that it takes for divergent, an
    // MMA's issue took 110 cycles instead of 65)
    const int halves = __shfl_sync(kFull, g.keys > 128 ? 2 : 1, 0);
    if (!wait_all(c, B_KREADY, k.par)) return;
    for (int left = __shfl_sync(kFull, g.r1 - g.r0, 0); left > 0; --left) {
      if (!wait_all(c, B_QFULL + q.st, q.par)) return;
#pragma unroll 1
      for (int x = 0; x < halves; ++x, ++n) {
        if (n >= kSums && !wait_all(c, B_SFREE + s.st, s.par ^ 1)) return;
        tc_fence_after();
        const uint64_t qd = sdesc(sm + S::kOffQ + q.st * S::kTile, 16, 1024);
        const uint32_t d = tmem + s.st * kRows, kt = tmem + kColK + x * (D / 2);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ta(d, kt + 8 * kk, qd + (kk >> 2) * (128 * 128 / 16) + 2 * (kk & 3), kIdesc, kk ? 1u : 0u);
        // (last: one rounding at the log-sum-exp's magnitude)
        mma(d, ones, sdesc(sm + S::kOffLse + q.st * 32, 16, 1024), kIdesc, 1u);
        const uint32_t tile = x ? tiles[1]++ : tiles[0]++;
        commit(c.bar + sum_bar(x, tile));
        s.next();
      }
      commit(c.bar + B_QEMPTY + q.st);
      __syncwarp();
      q.next();
    }
    commit(c.bar + B_KDONE);
    __syncwarp();
    k.next();
  }
}

// The rows' numbers: for row r of a row tile -lse in the products' units, as three bf16 whose sum it is (for
// the products with K's ones), and its position (-1: no row), and (lowest position, highest, rows) of the tile.  A tile's are
// requested while the warp waits for the place of the one before (a load's latency to each row tile had
// bound this kernel).
__device__ void row_loader(const Ctx& c, const TreeParams& p, uint8_t* lse, int* pos, int4* info) {
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31;
  float a[4], scale = 1.f;  // scale: -1 over the kv head's
  int b[4], cols = 0, token[4], head[4];  // of the lane's rows in a tile
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = lane + 32 * i;
    token[i] = col < p.tile_rows ? col / m.group : INT_MAX / 2;
    head[i] = col % m.group;
  }
  uint32_t tile = 0;  // row tiles so far
  Ring<kQueries> q;
  auto store = [&]() {  // the tile before
    const uint32_t st = (tile - 1) % kPos, turn = (tile - 1) / kPos;
    if (tile > kQueries && !wait_all(c, B_QEMPTY + q.st, q.par ^ 1)) return false;
    if (turn > 0 && !wait_all(c, B_PFREE + st, (turn & 1) ^ 1)) return false;
    int lo = INT_MAX, hi = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = lane + 32 * i;
      lo = min(lo, b[i] >= 0 ? b[i] : INT_MAX);
      hi = max(hi, b[i]);
      // (a row without a finite score, lse -inf, gives no weight)
      const float x = a[i] == -INFINITY ? -INFINITY : a[i] * scale;
      const float x1 = __bfloat162float(__float2bfloat16_rn(x)), rest = fabsf(x1) < INFINITY ? x - x1 : 0.f;
      const float x2 = __bfloat162float(__float2bfloat16_rn(rest));
      *reinterpret_cast<uint2*>(lse + col * 128 + (((2 * q.st) ^ (col & 7)) << 4)) =
          make_uint2(pack_bf16x2(x1, x2), pack_bf16x2(rest - x2, 0.f));
      pos[st * kRows + col] = b[i];
    }
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    if (lane == 0) info[st] = make_int4(lo, hi, cols, 0);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar + B_QFULL + q.st);
    q.next();
    return true;
  };
  Walk walk(p, blockIdx.x);
  Piece g;
  while (walk.next(p, g)) {
    const float of_head = -1.f / head_scale(m.k_scales, g.kvh, p.scale);
    for (int r = g.r0; r < g.r1; ++r, ++tile) {
      if (tile > 0 && !store()) return;
      const int first = r * p.tile_tokens;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = first + token[i];
        const bool in = t < g.tokens;
        a[i] = in ? m.lse[(int64_t)(g.kvh * m.group + head[i]) * m.num_tokens + g.qs + t] : 0.f;
        b[i] = in ? m.positions[g.qs + t] : -1;
      }
      scale = of_head;
      cols = min(p.tile_rows, (g.tokens - first) * m.group);
    }
  }
  if (tile > 0) store();
}

// 64 of a key's dims (half h) from a stage in shared memory, as pairs of bf16; codes are widened (exactly).
template <int D, bool FP8>
__device__ __forceinline__ void key_dims(const uint8_t* stage, int row, int h, uint32_t (&v)[32]) {
  using S = Shape<D, FP8>;
  const int sw = row & 7;
  if constexpr (FP8) {
    const uint8_t* at = stage + row * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 src = *reinterpret_cast<const uint4*>(at + (((4 * h + i) ^ sw) << 4));
      const uint32_t in[4] = {src.x, src.y, src.z, src.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t lo, hi;
        widen4(in[e], lo, hi);
        const float2 fl = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        v[8 * i + 2 * e] = pack_bf16x2(fl.x, fl.y);
        v[8 * i + 2 * e + 1] = pack_bf16x2(fh.x, fh.y);
      }
    }
  } else {
    const uint8_t* at = stage + (row >> 3) * 1024 * S::kHalves + h * 1024 + sw * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 src = *reinterpret_cast<const uint4*>(at + ((i ^ sw) << 4));
      v[4 * i] = src.x;
      v[4 * i + 1] = src.y;
      v[4 * i + 2] = src.z;
      v[4 * i + 3] = src.w;
    }
  }
}

// A warpgroup's 128 keys and every other row tile: thread = key.
template <int D, bool FP8>
__device__ void summer(const Ctx& c, const TreeParams& p, uint32_t tmem, uint32_t stall, const int* pos,
                        const int4* info, float* sums) {
  using S = Shape<D, FP8>;
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 4, x = warp >> 3, quad = warp & 3;
  const uint32_t half = (warp >> 2) & 1;  // warpgroup of the key half
  const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
  Ring<1> k;
  Ring<kPos> l;
  Ring<kSums> s;
  uint32_t pieces = 0, tile = 0;  // of this key half so far
  bool first = true;
  Walk walk(p, blockIdx.x);
  Piece g;
  while (walk.next(p, g)) {
    const bool both = g.keys > 128, mine = x == 0 || both;
    const int low = g.key0 + 128 * x, key = low + 32 * quad + lane;
    const float sl = head_scale(m.k_scales, g.kvh, p.scale) * kLog2e;
    const uint64_t sl2 = f2_pack(sl, sl);
    // the last position that sees the key
    const int last = m.window > 0 && key >= p.first ? (int)min((int64_t)key + m.window - 1, (int64_t)INT_MAX) : INT_MAX;
    // K to tensor memory, where all of the item's products read it; each warp half of its keys' dims
    if (!wait_all(c, B_KFULL, k.par)) return;
    if (!first && !wait_all(c, B_KDONE, k.par ^ 1)) return;
    if (mine && half < S::kHalves) {
      uint32_t v[32];
      key_dims<D, FP8>(c.sm + S::kOffK + x * S::kHalf, 32 * quad + lane, half, v);
      tc_fence_after();
      tmem_st32(lanes + kColK + x * (D / 2) + 32 * half, v);
      tmem_wait_st();
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(c.bar + B_KEMPTY);
      mbar_arrive(c.bar + B_KREADY);
    }
    k.next();
    first = false;
    uint64_t sum[4] = {0, 0, 0, 0};
    if (!mine) {  // (the first half's warps arrive for the second's)
      for (int r = g.r0; r < g.r1; ++r) {
        s.next();
        l.next();
      }
      continue;
    }
    for (int r = g.r0; r < g.r1; ++r, ++tile) {
      if (x) s.next();
      if ((tile & 1) == half) {
        // (the issuer has waited for the rows' numbers)
        if (!wait_all(c, stall ? B_NEVER : sum_bar(x, tile), stall ? 0u : (tile >> 2) & 1)) return;
        tc_fence_after();
        const int4 t = info[l.st];
        // every row of the tile sees all of the warpgroup's keys
        const bool all = t.x >= low + 127 && (m.window <= 0 || low > t.y - m.window || low + 127 < p.first);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t v[64];
          tmem_ld64(lanes + s.st * kRows + 64 * h, v);
          const int* tp = pos + l.st * kRows + 64 * h;
          tmem_wait_ld64(v);
          if (h) {  // the buffer has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar + B_SFREE + s.st);
          }
          if (all && t.z >= 64 * h + 64) {
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float a, b;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sl2), a, b);
              sum[(e >> 1) & 3] = f2_add(sum[(e >> 1) & 3], f2_pack(fast_exp2(a), fast_exp2(b)));
            }
          } else if (t.z > 64 * h) {
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const int4 ps = *reinterpret_cast<const int4*>(tp + e);
              auto one = [&](int at, int i) {  // (-1, no row, is below every key)
                return at >= key && at <= last ? fast_exp2(__uint_as_float(v[e + i]) * sl) : 0.f;
              };
              sum[0] = f2_add(sum[0], f2_pack(one(ps.x, 0), one(ps.y, 1)));
              sum[1] = f2_add(sum[1], f2_pack(one(ps.z, 2), one(ps.w, 3)));
            }
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(c.bar + B_PFREE + l.st);
          if (!both) mbar_arrive(c.bar + B_PFREE + l.st);
        }
      }
      s.next();
      if (!x && both) s.next();
      l.next();
    }
    float a, b, d, e;
    f2_unpack(f2_add(sum[0], sum[1]), a, b);
    f2_unpack(f2_add(sum[2], sum[3]), d, e);
    float total = (a + b) + (d + e);
    // the second warpgroup's sums go to the first
    float* other = sums + 128 * x + 32 * quad + lane;
    if (half) {
      if (pieces >= 1 && !wait_all(c, B_TAKEN + x, (pieces & 1) ^ 1)) return;
      *other = total;
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar + B_HALF + x);
      ++pieces;
      continue;
    }
    if (!wait_all(c, B_HALF + x, pieces & 1)) return;
    const float add = *other;
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar + B_TAKEN + x);
    ++pieces;
    total += add;
    if (key < g.key0 + g.keys && !*c.abort) {
      if (g.slot >= 0) {
        p.w.part[(int64_t)g.slot * kKeys + key - g.key0] = total;
      } else if (total != 0.f) {
        float* at = p.key_weights + ((int64_t)g.s * m.num_kv_heads + g.kvh) * p.weights_len + key;
        *at += total;
      }
    }
    __syncwarp();
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Shape<D, FP8>::kThreads, 1)
    k_weights_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const TreeParams p, uint64_t wait_limit, uint32_t stall) {
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
      if (i == B_KEMPTY || i == B_KREADY) n = 16;
      if (i >= B_SFREE && i < B_SFREE + kSums) n = 4;
      if (i >= B_QFULL && i < B_QFULL + kQueries) n = 2;
      if (i >= B_PFREE && i < B_PFREE + kPos) n = 8;
      if (i >= B_HALF && i < B_TAKEN + 2) n = 4;
      mbar_init(bar + i, n);
    }
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
  }
  for (int i = threadIdx.x; i < 128 * 8; i += S::kThreads) {  // the rows of log-sum-exps and ones
    const int chunk = (i & 7) ^ ((i >> 3) & 7);
    *reinterpret_cast<uint4*>(sm + S::kOffLse + 16 * i) =
        chunk == 2 * kQueries ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
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
  pdl_wait();  // (the attention's log-sum-exps)
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    const bool off = (smem_u32(sm) & 1023u) != 0;
    if (off) record_error(p.status, PA_ECUDA);
    flags[0] = off || status_set(p.status) ? 1 : 0;
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const Ctx c{sm, bar, reinterpret_cast<volatile int*>(flags + 1), p.status, wait_limit};
  int* pos = reinterpret_cast<int*>(sm + S::kOffPos);
  int4* info = reinterpret_cast<int4*>(sm + S::kOffInfo);
  if (flags[0] == 0) {
    if (warp == 0) {
      producer<D, FP8>(c, p, &tk, &tq);
    } else if (warp == 1) {
      issuer<D, FP8>(c, p, tmem);
      __syncwarp();
      // every MMA is done before the tensor memory goes (bounded)
      commit(bar + B_FIN);
      if ((threadIdx.x & 31) == 0) mbar_wait(bar + B_FIN, 0, 1000000000ull);
      __syncwarp();
    } else if (warp == 2) {
      row_loader(c, p, sm + S::kOffLse, pos, info);
    } else if (warp >= 4) {
      summer<D, FP8>(c, p, tmem, stall, pos, info, reinterpret_cast<float*>(sm + S::kOffHalf));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
  }
}

// Block b: the item that the boundary between CTA b and b + 1 cuts, when that is the item's first cut.
// Its pieces are CTA b's last one and the first ones of the CTAs behind it whose shares begin inside it.
__global__ void __launch_bounds__(kKeys) k_weights_join(const TreeParams p) {
  const int b = blockIdx.x, key = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (__syncthreads_or(status_set(p.status))) return;
  const int4 cut = p.w.starts[b + 1], from = p.w.starts[b];
  if (cut.x < 0 || cut.x >= p.m.num_seqs) return;
  const int4 q = p.w.seqs[2 * cut.x], t = p.w.seqs[2 * cut.x + 1];
  const int4 it = p.w.items[q.x + cut.z];
  if (cut.w <= it.y) return;  // the boundary lies between items
  const bool same = from.x == cut.x && from.y == cut.y && from.z == cut.z;
  if (same && from.w > it.y) return;  // a later cut of the item
  if (it.x * kKeys + key >= t.z) return;
  float sum = p.w.part[(int64_t)(same ? 2 * b : 2 * b + 1) * kKeys + key];
  for (int c = b + 1; c < p.w.grid; ++c) {
    const int4 s0 = p.w.starts[c], s1 = p.w.starts[c + 1];
    if (s0.x != cut.x || s0.y != cut.y || s0.z != cut.z) break;
    // (a CTA whose share is empty left nothing)
    if (s1.x != s0.x || s1.y != s0.y || s1.z != s0.z || s1.w != s0.w)
      sum += p.w.part[(int64_t)(2 * c) * kKeys + key];
  }
  if (sum != 0.f) {
    float* at = p.key_weights + ((int64_t)cut.x * p.m.num_kv_heads + cut.y) * p.weights_len +
                it.x * kKeys + key;
    *at += sum;
  }
}

template <int D, bool FP8>
cudaError_t launch_as(const CUtensorMap& tq, const CUtensorMap& tk, const TreeParams& p, uint64_t limit,
                      uint32_t stall, cudaStream_t stream) {
  using S = Shape<D, FP8>;
  auto kern = k_weights_tc<D, FP8>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.w.grid), dim3(S::kThreads), S::kSmem, stream, tq, tk, p, limit, stall);
}

}  // namespace

cudaError_t launch_weights_tc(const CUtensorMap& tq, const CUtensorMap& tk, const TreeParams& p, bool fp8,
                              uint64_t wait_limit, uint32_t stall, cudaStream_t stream) {
  const cudaError_t e = fp8 ? launch_as<128, true>(tq, tk, p, wait_limit, stall, stream)
                        : p.m.head_dim == 128 ? launch_as<128, false>(tq, tk, p, wait_limit, stall, stream)
                                              : launch_as<64, false>(tq, tk, p, wait_limit, stall, stream);
  if (e != cudaSuccess || p.w.grid < 2) return e;
  return launch_pdl(k_weights_join, dim3(p.w.grid - 1), dim3(kKeys), 0, stream, p);
}

}  // namespace pa
