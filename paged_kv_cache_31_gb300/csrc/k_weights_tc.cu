// k_weights_tc.cu -- the attention weight that every cached key receives (k_key_weights.cu has the
// formula and the general kernel), on the 5th-generation tensor cores: bf16 queries over bf16 (head size
// 64 / 128) or e4m3 (128) pools of 16-position blocks.
//
// Math.  With the attention's log-sum-exps at hand a weight needs no running maximum: exp(s - lse) is
// final, so only S is computed again, a third of the attention's products over bf16 pools (which
// multiplies V by both terms of P).  It is taken transposed, S^T = K Q^T: keys are the rows of the
// accumulator, a key is a thread, and the sum over the queries stays in its registers: no exchange, no
// atomics, one add to memory for a key in the end.
//
// Work.  An item is 256 keys of one (sequence, kv head), which stay in shared memory, against the row
// tiles (128 rows: whole tokens times the group's heads) that see any of them, which stream past.  The
// items' row tiles, laid end to end with a weight for an item's keys, are cut evenly over one CTA per SM;
// the pieces of a cut item leave partial sums, which k_weights_join adds in order.
//
// Roles.  warp 0: TMA of K (two stages of 256 keys) and Q (a ring of two row tiles); warp 1:
// tensor-memory owner, issues S^T; warps 2 and 3: the rows' log-sum-exps and positions into a ring of four;
// warps 4..19: exponentials and sums, a warpgroup for 128 keys and 64 rows of a row tile each, from two S^T
// buffers for each 128 keys (two warpgroups, of all rows, left the schedulers idle half of the time: 312 us
// for a prompt of 8191 tokens, 8 x 4 heads); warps 20..23 (e4m3 pools): widen K to bf16, exactly, once an
// item.
//
// What bounds it: a row tile's 32768 exponentials (2^x on the SFU and two packed fp32 instructions for
// a pair) beside 1230 cycles of products.
#include <algorithm>

#include "k_tree.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kKeys = kWeightKeys;  // of an item
constexpr int kRows = 128;          // of a row tile, at most
constexpr int kLse = 4;             // ring of the rows' numbers

template <int D, bool FP8>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;  // 128 rows of 16-bit values
  static constexpr int kCodes = 128 * 128;           // 128 keys of codes
  static constexpr int kThreads = FP8 ? 768 : 640;
  // K as it is multiplied: two stages of 256 keys (bf16, as the 5-D boxes write it), or one of widened
  // ones (dim half by dim half)
  static constexpr int kWide = FP8 ? 1 : 2;
  static constexpr int kRowGroup = FP8 ? 1024 : 1024 * kHalves;  // between 8-row groups
  static constexpr int kDimHalf = FP8 ? 128 * 128 : 1024;        // between dim halves
  static constexpr int kOffK = 0;
  static constexpr int kOffCodes = kOffK + kWide * 2 * kTile;  // e4m3: two stages of 256 keys' codes
  static constexpr int kOffQ = kOffCodes + (FP8 ? 4 * kCodes : 0);
  static constexpr int kOffRow = kOffQ + 2 * kTile;  // [kLse][2][128]: -lse in log2 units, positions
  static constexpr int kOffInfo = kOffRow + kLse * 2 * kRows * 4;  // [kLse] int4
  static constexpr int kOffHalf = kOffInfo + kLse * 16;  // [key half][128]: sums of the second row halves
  static constexpr int kOffBar = kOffHalf + 2 * 128 * 4;
  static constexpr int kOffMisc = kOffBar + 32 * 8;
  static constexpr int kSmem = kOffMisc + 16;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

enum : int {
  B_KFULL = 0,              // K's keys (or codes) landed
  B_KEMPTY = B_KFULL + 2,   // all products (or the widening) of the stage are done
  B_WIDE = B_KEMPTY + 2,    // e4m3: K is widened
  B_WFREE = B_WIDE + 1,     // e4m3: its products are done
  B_QFULL = B_WFREE + 1,
  B_QEMPTY = B_QFULL + 2,
  B_SFULL = B_QEMPTY + 2,   // [key half][buffer]
  B_SFREE = B_SFULL + 4,
  B_LFULL = B_SFREE + 4,
  B_LFREE = B_LFULL + kLse,
  B_HALF = B_LFREE + kLse,  // per key half: the second row half's sums are there
  B_TAKEN = B_HALF + 2,     // they have been added
  B_FIN = B_TAKEN + 2,
  B_NEVER = B_FIN + 1,  // nothing arrives on it (the debug_stall test hook)
  kNumBars = B_NEVER + 1
};
static_assert(kNumBars <= 32, "barrier area");

constexpr uint32_t kTmemCols = 512;

__device__ __forceinline__ void mma(uint32_t elect, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\tsetp.ne.u32 e, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elect)
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
  Ring<2> k, q;
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
      if (nk >= 2) ok = wait_bar(c, B_KEMPTY + k.st, k.par ^ 1);
      if (ok) mbar_arrive_expect_tx(c.bar + B_KFULL + k.st, halves * (FP8 ? S::kCodes : S::kTile));
    }
    ok = __shfl_sync(kFull, (int)ok, 0);
    if (!ok) break;
    if (lane < 8 * halves) {
      if constexpr (FP8)
        tma_load_3d(c.sm + S::kOffCodes + k.st * 2 * S::kCodes + lane * 2048, tk, 0, g.kvh,
                    id >= 0 ? id * 16 : -16, c.bar + B_KFULL + k.st);
      else
        tma_load_5d(c.sm + S::kOffK + k.st * 2 * S::kTile + lane * (S::kTile / 8), tk, 0, 0, 0,
                    id >= 0 ? id * 2 : -2, g.kvh, c.bar + B_KFULL + k.st);
    }
    ++nk;
    k.next();
    if (lane == 0) {
      for (int r = g.r0; ok && r < g.r1; ++r) {
        if (nq >= 2) ok = wait_bar(c, B_QEMPTY + q.st, q.par ^ 1);
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
    for (uint32_t i = nk > 2 ? nk - 2 : 0; i < nk; ++i) mbar_wait(c.bar + B_KFULL + (i & 1), (i >> 1) & 1, c.limit);
    for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq; ++i) mbar_wait(c.bar + B_QFULL + (i & 1), (i >> 1) & 1, c.limit);
  }
  __syncwarp();
}

template <int D, bool FP8>
__device__ void issuer(const Ctx& c, const TreeParams& p, uint32_t tmem) {
  using S = Shape<D, FP8>;
  constexpr uint32_t kIdesc = idesc_f16kind(128, kRows, 0, 1);
  const uint32_t sm = smem_u32(c.sm), elect = (threadIdx.x & 31) == 0;
  Ring<2> k, q;
  Ring<1> w;
  uint32_t n[2] = {0, 0};  // tiles of each half so far
  Walk walk(p, blockIdx.x);
  Piece g;
  while (walk.next(p, g)) {
    const int halves = g.keys > 128 ? 2 : 1;
    if (!(FP8 ? wait_all(c, B_WIDE, w.par) : wait_all(c, B_KFULL + k.st, k.par))) return;
    const uint32_t kb = sm + S::kOffK + (FP8 ? 0 : k.st * 2 * S::kTile);
    for (int r = g.r0; r < g.r1; ++r) {
      if (!wait_all(c, B_QFULL + q.st, q.par)) return;
#pragma unroll 1
      for (int x = 0; x < halves; ++x) {
        const uint32_t use = x ? n[1] : n[0], buf = use & 1;
        if (use >= 2 && !wait_all(c, B_SFREE + 2 * x + buf, ((use >> 1) & 1) ^ 1)) return;
        tc_fence_after();
        uint64_t kd = sdesc(kb + x * S::kTile, 16, S::kRowGroup);
        uint64_t qd = sdesc(sm + S::kOffQ + q.st * S::kTile, 16, 1024);
#pragma unroll 1
        for (int h = 0; h < S::kHalves; ++h) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma(elect, tmem + (2 * x + buf) * kRows, kd + 2 * kk, qd + 2 * kk, kIdesc, (h | kk) ? 1u : 0u);
          kd += S::kDimHalf / 16;
          qd += 128 * 128 / 16;
        }
        commit(c.bar + B_SFULL + 2 * x + buf);
        if (x) ++n[1]; else ++n[0];
      }
      commit(c.bar + B_QEMPTY + q.st);
      __syncwarp();
      q.next();
    }
    commit(c.bar + (FP8 ? B_WFREE : B_KEMPTY + k.st));
    __syncwarp();
    k.next();
    w.next();
  }
}

// The rows' numbers: for column r of a row tile -lse in log2 units and its position (-1: no row), and
// (lowest position, highest, rows) of the tile.  Two warps take the tiles in turn, and a warp requests a
// tile's before it stores those of the one before: one warp without either was what bound this kernel (a
// load's latency to each row tile: 1.4 us a tile of 0.6 us).
__device__ void row_loader(const Ctx& c, const TreeParams& p, int which, float* nl, int* pos, int4* info) {
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31;
  float a[4];
  int b[4], cols = 0;
  uint32_t tile = 0, held = 0;  // row tiles so far; the one whose numbers are held
  bool have = false;
  auto store = [&]() {
    const uint32_t st = held % kLse, turn = held / kLse;
    int lo = INT_MAX, hi = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo = min(lo, b[i] >= 0 ? b[i] : INT_MAX);
      hi = max(hi, b[i]);
    }
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    if (turn > 0 && !wait_all(c, B_LFREE + st, (turn & 1) ^ 1)) return false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = lane + 32 * i;
      // (a row without a finite score, lse -inf, gives no weight)
      nl[st * 2 * kRows + col] = a[i] == -INFINITY ? -INFINITY : -a[i] * kLog2e;
      pos[st * 2 * kRows + col] = b[i];
    }
    if (lane == 0) info[st] = make_int4(lo, hi, cols, 0);
    __syncwarp();
    if (lane == 0) mbar_arrive(c.bar + B_LFULL + st);
    return true;
  };
  Walk walk(p, blockIdx.x);
  Piece g;
  while (walk.next(p, g)) {
    for (int r = g.r0; r < g.r1; ++r, ++tile) {
      if ((int)(tile & 1) != which) continue;
      float na[4];
      int nb[4];
      const int first = r * p.tile_tokens;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = lane + 32 * i, t = first + col / m.group;
        const bool in = col < p.tile_rows && t < g.tokens;
        na[i] = in ? m.lse[(int64_t)(g.kvh * m.group + col % m.group) * m.num_tokens + g.qs + t] : 0.f;
        nb[i] = in ? m.positions[g.qs + t] : -1;
      }
      if (have && !store()) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = na[i];
        b[i] = nb[i];
      }
      cols = min(p.tile_rows, (g.tokens - first) * m.group);
      held = tile;
      have = true;
    }
  }
  if (have) store();
}

// Warps 20 to 23: codes to bf16 (exact), a quarter of the keys each; 128 keys at a time as in
// k_tree_tc.cuh, dim half by dim half.
template <int D>
__device__ void widener(const Ctx& c, const TreeParams& p) {
  using S = Shape<D, true>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 20;
  Ring<2> k;
  Ring<1> wd;
  uint32_t use = 0;
  Walk walk(p, blockIdx.x);
  Piece g;
  for (; walk.next(p, g); ++use) {
    const int halves = g.keys > 128 ? 2 : 1;
    if (use >= 1 && !wait_all(c, B_WFREE, wd.par ^ 1)) return;
    if (!wait_all(c, B_KFULL + k.st, k.par)) return;
    for (int x = 0; x < halves; ++x) {
      const uint8_t* codes = c.sm + S::kOffCodes + (2 * k.st + x) * S::kCodes;
      uint8_t* tile = c.sm + S::kOffK + x * S::kTile;
#pragma unroll 1
      for (int i0 = 0; i0 < 8; ++i0) {
        const int ch = lane + 32 * i0, r = 32 * w + (ch >> 3), sw = r & 7;
        const uint4 src = *reinterpret_cast<const uint4*>(codes + 32 * w * 128 + ch * 16);
        const int L = (ch & 7) ^ sw, h = L >> 2, c0 = 2 * (L & 3);
        const uint32_t in[4] = {src.x, src.y, src.z, src.w};
        uint32_t out[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t a, b;
          widen4(in[e], a, b);
          const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
          const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
          out[2 * e] = pack_bf16x2(fa.x, fa.y);
          out[2 * e + 1] = pack_bf16x2(fb.x, fb.y);
        }
        uint8_t* row = tile + h * 128 * 128 + r * 128;
        *reinterpret_cast<uint4*>(row + ((c0 ^ sw) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ sw) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(c.bar + B_KEMPTY + k.st);
      mbar_arrive(c.bar + B_WIDE);
    }
    k.next();
    wd.next();
  }
}

// A warpgroup's 128 keys and half of the rows: thread = key.
template <int D, bool FP8>
__device__ void summer(const Ctx& c, const TreeParams& p, uint32_t tmem, uint32_t stall, const float* nl,
                       const int* pos, const int4* info, float* sums) {
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 4, x = warp >> 3, quad = warp & 3;
  const int half = (warp >> 2) & 1;  // of a row tile's columns
  const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + 2 * x * kRows;
  Ring<kLse> l;
  uint32_t use = 0, pieces = 0;  // row tiles and pieces of this key half so far
  Walk walk(p, blockIdx.x);
  Piece g;
  while (walk.next(p, g)) {
    const bool mine = x == 0 || g.keys > 128;
    const int low = g.key0 + 128 * x, key = low + 32 * quad + lane;
    const float sl = head_scale(m.k_scales, g.kvh, p.scale) * kLog2e;
    const uint64_t sl2 = f2_pack(sl, sl);
    uint64_t sum[2] = {0, 0};
    for (int r = g.r0; r < g.r1; ++r) {
      if (!wait_all(c, B_LFULL + l.st, l.par)) return;
      if (mine) {
        const uint32_t buf = use & 1;
        if (!wait_all(c, stall ? B_NEVER : B_SFULL + 2 * x + buf, stall ? 0u : (use >> 1) & 1)) return;
        tc_fence_after();
        const int4 t = info[l.st];
        // every row of the tile sees all of the warpgroup's keys
        const bool all = t.x >= low + 127 && (m.window <= 0 || low > t.y - m.window || low + 127 < p.first);
        const float* tl = nl + l.st * 2 * kRows;
        const int* tp = pos + l.st * 2 * kRows;
#pragma unroll 1
        for (int q = 2 * half; q < 2 * half + 2; ++q) {
          uint32_t v[32];
          tmem_ld32(lanes + buf * kRows + 32 * q, v);
          tmem_wait_ld(v);
          if (q & 1) {  // this half of the buffer has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar + B_SFREE + 2 * x + buf);
          }
          if (all && 32 * q + 32 <= t.z) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 n4 = *reinterpret_cast<const float4*>(tl + 32 * q + e);
              float a, b;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sl2,
                               f2_pack(n4.x, n4.y)), a, b);
              sum[0] = f2_add(sum[0], f2_pack(fast_exp2(a), fast_exp2(b)));
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), sl2,
                               f2_pack(n4.z, n4.w)), a, b);
              sum[1] = f2_add(sum[1], f2_pack(fast_exp2(a), fast_exp2(b)));
            }
          } else if (32 * q < t.z) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int ps = tp[32 * q + e];
              const bool see = ps >= 0 && window_visible(p, ps, key);
              const float a = see ? fast_exp2(fmaf(__uint_as_float(v[e]), sl, tl[32 * q + e])) : 0.f;
              sum[0] = f2_add(sum[0], f2_pack(e & 1 ? 0.f : a, e & 1 ? a : 0.f));
            }
          }
        }
        ++use;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(c.bar + B_LFREE + l.st);
      l.next();
    }
    float a, b, d, e;
    f2_unpack(sum[0], a, b);
    f2_unpack(sum[1], d, e);
    float total = (a + b) + (d + e);
    if (!mine) continue;
    // the second half's sums go to the first
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
      if ((FP8 && i >= B_KEMPTY && i < B_KEMPTY + 2) || i == B_WIDE) n = 4;
      if (i >= B_SFREE && i < B_SFREE + 4) n = 8;
      if (i >= B_LFREE && i < B_LFREE + kLse) n = 16;
      if (i >= B_HALF && i < B_TAKEN + 2) n = 4;
      mbar_init(bar + i, n);
    }
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
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
  float* nl = reinterpret_cast<float*>(sm + S::kOffRow);
  int* pos = reinterpret_cast<int*>(sm + S::kOffRow) + kRows;
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
    } else if (warp == 2 || warp == 3) {
      row_loader(c, p, warp - 2, nl, pos, info);
    } else if (warp >= 20) {
      if constexpr (FP8) widener<D>(c, p);
    } else if (warp >= 4) {
      summer<D, FP8>(c, p, tmem, stall, nl, pos, info, reinterpret_cast<float*>(sm + S::kOffHalf));
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
