// k_window_decode.cu -- attention behind a window with first tokens, and the attention weights that keys
// receive, for batches of decoding tokens: bf16 queries over bf16 (head size 64 / 128) or e4m3 (128)
// pools of 16-position blocks.
//
// Work.  A cluster of CTAs for each (sequence, kv head) shares the visible blocks (k_window.cu counts
// them without the gap) in even, contiguous runs; a CTA's warps take the run's blocks in turn, each
// through its own ring of TMA stages, so every key is read once.  The warps' and then the CTAs' softmax
// states (m, l, O) are joined in fixed order, through shared memory and the cluster's.  The metadata are
// checked by a kernel in front (k_window_check), beside which this one loads and computes already: it
// waits for it before it writes, and bounds its own indices until then.  Two launches instead of the
// three of a planned call, and no partial states in memory.
//
// Math.  As k_decode_mma.cu: S = Q K^T on the m16n8k16 warp MMA (bf16), rows = (token, head) pairs, an
// online softmax over 16 keys at a time, P as a bf16 pair; e4m3 pools swap the operands, S^T = K Q^T and
// O^T = V^T P^T in f16, with the codes widened in registers and the dimensions in a permuted order that
// makes a lane's bytes contiguous.
//
// Weights.  exp(s - lse) needs a row's final log-sum-exp, so a CTA keeps the scores of its keys in shared
// memory (14 KB: 872 keys of 4 heads) or, where they are more, in the workspace (they stay in L2) until
// the states have been joined, and adds each key's sum to memory then: K is read once, where a second
// pass over it would read half as many bytes again.  Keys past that room are multiplied once more.  One
// thread adds to a key, so the order of the sums is fixed.
//
// Where the scores lie in the workspace, K and V leave L2 first: left to itself L2 wrote the scores out
// before they came back (64 sequences of 512 to 4096 keys, the same ones again: 22 MB written and 21 read beside
// 624 MB of K and V, 109.6 us; so 102).
//
// What bounds it: the K / V bytes for large batches (64 sequences behind a window of 4096, 1027 MB: 159 us, 0.95
// of the copy rate; 64 of 512 to 4096 keys with their weights 104 us, 0.90 of it), for small ones a chain of
// latencies (metadata, table, keys, joins: 1 sequence, window 4096: 11.7 us), over e4m3 pools both (48
// sequences, window 1024: 24.7 us for 15, or 22.2 from L2 where the same 103 MB are read again).
#include <algorithm>
#include <cfloat>

#include "k_tree.cuh"
#include "k_window.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBlk = 16;

// Shapes: two CTAs to an SM; kNarrow: half as many warps, four CTAs; kBroad (bf16): twice as many, one.
enum : int { kPlain = 0, kNarrow = 1, kBroad = 2 };
template <int D, bool FP8, int KIND>
struct Shape {
  static constexpr bool NARROW = KIND == kNarrow;
  static constexpr int NW = NARROW ? (FP8 ? 4 : 2) : FP8 || KIND == kBroad ? 8 : 4;  // warps
  static constexpr int kPerSm = NARROW ? 4 : KIND == kBroad ? 1 : 2;
  static constexpr int NS = KIND == kBroad ? 2 : 3;  // stages of a warp's ring
  static constexpr int TR = FP8 ? 8 : 16;  // query rows of a tile
  static constexpr int kHalves = FP8 ? 1 : D / 64;
  static constexpr int kTile = kHalves * kBlk * 128;  // a block's K (or V) of one kv head
  static constexpr int kStage = 2 * kTile;
  static constexpr int kNT = D / 8, kKS = D / 16;
  static constexpr int kRing = NW * NS * kStage;
  // scores of a CTA's keys, and the states that are joined (in the ring's place)
  static constexpr int kScores = NARROW ? 0 : 14336;
  static constexpr int kLd = D + 4;
  static constexpr int kOffState = NW * 16 * kLd * 4;  // behind the warps' O: the CTA's
  static_assert(kOffState + 16 * kLd * 4 <= kRing, "states lie in the ring");
  static constexpr int kOffSmall = kRing;  // struct Small
  static constexpr int kOffScores = kOffSmall + 2816;
  static constexpr int smem(bool weigh) { return kOffScores + (weigh ? kScores : 0); }
  static_assert(kPerSm * (1024 + kOffScores + kScores) <= 228 * 1024, "CTAs of an SM");
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// TMA loads whose lines leave L2 before others.
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                        uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void load_5d(void* dst, const CUtensorMap* map, int32_t c3, int32_t c4,
                                        uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c3), "r"(c4), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Byte offset of 16-byte chunk `chunk` (along D) of row `row` of a block written by a 5-D box: 8-row
// groups of (dim half, 8 rows of 128 bytes), 128-byte swizzle.
template <int HALVES>
__device__ __forceinline__ uint32_t tile_off(int row, int chunk) {
  return (uint32_t)((row >> 3) * HALVES * 1024 + (chunk >> 3) * 1024 + (row & 7) * 128 +
                    (((chunk & 7) ^ (row & 7)) << 4));
}

template <int NW, int NS>
struct Small {
  uint64_t full[NW * NS + 1];  // the last: nothing arrives on it (the debug_stall test hook)
  float2 warp_ml[NW][16];
  float2 ml[16];  // the CTA's state, read by its cluster
  int seq;        // the sequence that is this CTA's
  float lse[16], norm[16];
  float factor[16][16];  // of each CTA's part of a row
  int fail;
  int nan;  // row0 + 1 of a tile with a row of NaN
};

template <int D, bool FP8, bool WEIGH, int KIND>
__global__ void __launch_bounds__(Shape<D, FP8, KIND>::NW * 32, Shape<D, FP8, KIND>::kPerSm)
    k_window_decode(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const TreeParams p, uint64_t limit, uint32_t stall) {
  using S = Shape<D, FP8, KIND>;
  constexpr bool NARROW = S::NARROW;
  constexpr int NW = S::NW, NS = S::NS, TR = S::TR, LD = S::kLd;
  extern __shared__ __align__(1024) uint8_t ring[];
  using Sm = Small<NW, NS>;
  static_assert(sizeof(Sm) <= S::kOffScores - S::kOffSmall, "kOffScores");
  Sm& sh = *reinterpret_cast<Sm*>(ring + S::kOffSmall);
  float* mrg_o = reinterpret_cast<float*>(ring);
  float* state = reinterpret_cast<float*>(ring + S::kOffState);
  uint64_t* full = sh.full;
  const VarlenMeta& m = p.m;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.cluster, rank = C > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / C, kvh = unit % m.num_kv_heads;
  const int H = m.num_heads, G = m.group;
  int s = unit / m.num_kv_heads;
  // (the kernel in front lets this one start once it has waited for all work before it)
  int qs = 0, qe = 0, n = 0, guess = 0;
  auto numbers = [&]() {
    qs = m.query_start_loc[s];
    qe = m.query_start_loc[s + 1];
    n = m.seq_lens[s];
  };
  if (!p.ordered) {
    numbers();
    // (mostly token s is sequence s's: its position is there when that is known)
    guess = m.positions[min((int64_t)s, m.num_tokens - 1)];
  }
  if (tid <= NW * NS) mbar_init(&full[tid], 1);
  if (tid == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    // (the swizzled tiles need the alignment that the declaration asks for)
    sh.fail = (smem_u32(ring) & 1023u) != 0;
    sh.nan = 0;
    if (sh.fail) record_error(p.status, PA_ECUDA);
  }
  fence_mbar_init();
  __syncthreads();
  bool waited = false;
  if (p.ordered) {
    // more units than are resident at once: those with the most keys first (the s-th longest sequence)
    int* keys = reinterpret_cast<int*>(ring);
    auto seen = [&](int n) { return m.window > 0 ? min(n, (int)min((int64_t)m.window + p.first, (int64_t)INT_MAX)) : n; };
    for (int i = tid; i < m.num_seqs; i += NW * 32) keys[i] = seen(m.seq_lens[i]);
    __syncthreads();
    for (int i = tid; i < m.num_seqs; i += NW * 32) {
      const int mine = keys[i];
      int before = 0;
#pragma unroll 8
      for (int j = 0; j < m.num_seqs; ++j) before += keys[j] > mine || (keys[j] == mine && j < i);
      if (before == s) sh.seq = i;
    }
    __syncthreads();
    s = sh.seq;
    fence_proxy_async_smem();
    __syncthreads();  // (the ring is free)
    numbers();
  }
  // numbers that cannot be used as indices: no rows (the check records the error)
  const bool usable = qs >= 0 && qe >= qs && (int64_t)qe <= m.num_tokens && n >= 1 &&
                      ((int64_t)n + kBlk - 1) / kBlk <= m.max_blocks &&
                      (!WEIGH || (int64_t)n <= p.weights_len);
  int rows = usable && !sh.fail ? (qe - qs) * G : 0;
  // beside the prefill kernel: the sequences that it leaves; the plan was complete before it started
  // (and left no tokens to a batch that is not valid)
  if (p.after_tc && (rows > kWindowDecodeRows || p.seqs[2 * s].y == 0)) rows = 0;
  const int counted0 = WEIGH && p.observed > 0 ? max(0, qe - qs - p.observed) * G : 0;  // row
  const int32_t* table = m.block_tables + (int64_t)s * m.max_blocks;
  const float sl = p.scale * kLog2e;
  uint32_t ring_pos = 0;
  const uint64_t policy = evict_first();
  for (int row0 = 0; row0 < rows; row0 += TR) {
    const int nrow = min(TR, rows - row0);
    // q's rows are requested first, their values are used last
    uint32_t qa[S::kKS][4];
    {
      const int g = lane >> 2, c = lane & 3;
      const int r0 = min(g, nrow - 1) + row0, r1 = min(g + 8, nrow - 1) + row0;
      const uint32_t* q0 = reinterpret_cast<const uint32_t*>(
          static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)(qs + r0 / G) * H + kvh * G + r0 % G) * D);
      const uint32_t* q1 = reinterpret_cast<const uint32_t*>(
          static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)(qs + r1 / G) * H + kvh * G + r1 % G) * D);
      const bool v0 = g < nrow, v1 = g + 8 < nrow;
#pragma unroll
      for (int kk = 0; kk < S::kKS; ++kk) {
        if constexpr (FP8) {  // dims 32c + 4kk + {0, 1} and {2, 3} of row g (the permuted order)
          const uint2 w = v0 ? *reinterpret_cast<const uint2*>(q0 + 16 * c + 2 * kk) : make_uint2(0u, 0u);
          qa[kk][0] = w.x;
          qa[kk][2] = w.y;
        } else {
          qa[kk][0] = v0 ? q0[kk * 8 + c] : 0u;
          qa[kk][1] = v1 ? q1[kk * 8 + c] : 0u;
          qa[kk][2] = v0 ? q0[kk * 8 + 4 + c] : 0u;
          qa[kk][3] = v1 ? q1[kk * 8 + 4 + c] : 0u;
        }
      }
    }
    auto position = [&](int t) {
      return min(max(!p.ordered && qs + t == s ? guess : m.positions[qs + t], 0), n - 1);
    };
    const int low = position(row0 / G);
    const int high = max(position((row0 + nrow - 1) / G), low);
    // the tile's blocks, counted without the gap, and this CTA's run of them
    const int front = p.front;
    const int gap = m.window > 0 ? max(max(low - m.window + 1, 0) / kBlk - front, 0) : 0;
    const int vn = n - gap * kBlk;
    const int nblk = (high - gap * kBlk) / kBlk + 1;
    const int run0 = (int)((int64_t)nblk * rank / C), run1 = (int)((int64_t)nblk * (rank + 1) / C);
    const int count = run1 - run0;
    const int mine = count > warp ? (count - warp + NW - 1) / NW : 0;  // blocks run0 + warp + NW x
    auto pos_of = [&](int r) {  // counted without the gap; -1: no row
      const int R = row0 + r;
      return r < nrow ? position(R / G) - gap * kBlk : -1;
    };

    int win = -1, ids = 0;
    auto block_id = [&](int x) -> int {  // whole warp
      if ((x >> 5) != win) {
        win = x >> 5;
        const int i = (win << 5) + lane;
        ids = -1;
        if (i < mine) {
          int b = run0 + warp + NW * i;
          if (b >= front) b += gap;
          ids = table[b];
          if (ids < 0 || (int64_t)ids >= m.num_blocks) ids = -1;
        }
      }
      return __shfl_sync(kFull, ids, x & 31);
    };
    auto issue = [&](int x, uint32_t at, bool with_v) {  // whole warp: its block x as copy `at`
      const int id = block_id(x);
      if (lane == 0) {
        const uint32_t slot = at % NS;
        uint64_t* bar = &full[warp * NS + slot];
        uint8_t* dst = ring + (size_t)(warp * NS + slot) * S::kStage;
        mbar_arrive_expect_tx(bar, with_v ? S::kStage : S::kTile);
        // (an id outside the pool reads zeros from outside it)
        if (WEIGH && p.ordered) {
          if constexpr (FP8) {
            load_3d(dst, &tk, 0, kvh, id >= 0 ? id * kBlk : -kBlk, bar, policy);
            if (with_v) load_3d(dst + S::kTile, &tv, 0, kvh, id >= 0 ? id * kBlk : -kBlk, bar, policy);
          } else {
            load_5d(dst, &tk, id >= 0 ? id * 2 : -2, kvh, bar, policy);
            if (with_v) load_5d(dst + S::kTile, &tv, id >= 0 ? id * 2 : -2, kvh, bar, policy);
          }
        } else if constexpr (FP8) {
          tma_load_3d(dst, &tk, 0, kvh, id >= 0 ? id * kBlk : -kBlk, bar);
          if (with_v) tma_load_3d(dst + S::kTile, &tv, 0, kvh, id >= 0 ? id * kBlk : -kBlk, bar);
        } else {
          tma_load_5d(dst, &tk, 0, 0, 0, id >= 0 ? id * 2 : -2, kvh, bar);
          if (with_v) tma_load_5d(dst + S::kTile, &tv, 0, 0, 0, id >= 0 ? id * 2 : -2, kvh, bar);
        }
      }
    };
    int issued = 0;
    for (; issued < min(mine, NS); ++issued) issue(issued, ring_pos + issued, true);
    // scores to log2 units, of this lane's rows
    float sk[2];
    sk[0] = sk[1] = head_scale(m.k_scales, kvh, sl);
    // ---- q fragments and the rows' visible keys
    int pos[2], lo[2];  // of this lane's rows: bf16 lane / 4 (+ 8), e4m3 2 (lane % 4) (+ 1)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      pos[i] = pos_of(FP8 ? 2 * (lane & 3) + i : (lane >> 2) + 8 * i);
      lo[i] = m.window > 0 ? max(pos[i] - m.window, -1) + 1 : 0;
    }
    if constexpr (FP8) {
      // f16 with a power of two a row that brings its largest element to [2^14, 2^15): exact down to
      // 2^-28 of that.  An infinity makes the whole row NaN.
      float big = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        big = fmaxf(big, fmaxf(fmaxf(fabsf(__uint_as_float(qa[kk][0] << 16)),
                                     fabsf(__uint_as_float(qa[kk][0] & 0xffff0000u))),
                               fmaxf(fabsf(__uint_as_float(qa[kk][2] << 16)),
                                     fabsf(__uint_as_float(qa[kk][2] & 0xffff0000u)))));
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
      const int up = min(max(141 - (int)(__float_as_uint(big) >> 23), -113), 120);
      const float f = big < INFINITY ? __uint_as_float((uint32_t)(127 + up) << 23) : NAN;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          qa[kk][i] = pack_f16x2(__uint_as_float(qa[kk][i] << 16) * f,
                                 __uint_as_float(qa[kk][i] & 0xffff0000u) * f);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        sk[e] *= __uint_as_float((uint32_t)(127 - __shfl_sync(kFull, up, (2 * (lane & 3) + e) * 4)) << 23);
    }
    // keys that every row sees: [.., all_hi), and from all_lo on (the first tokens apart)
    const int all_hi = low - gap * kBlk + 1;
    const int all_lo = m.window > 0 ? max(high - gap * kBlk - m.window, -1) + 1 : 0;
    auto seen_by_all = [&](int key) {
      return key + kBlk <= all_hi && (key >= all_lo || key + kBlk <= p.first);
    };

    // S of a block in log2 units: bf16 [key tile][row 2, key 2] of rows g, g + 8 and keys 2c + {0, 1}
    // (+ 8); e4m3 in [0]: keys g (+ 8 in the upper two), rows 2c + {0, 1}
    auto scores_of = [&](const uint8_t* kt, int key0, float (&sc)[2][4]) {
      const uint32_t kbase = smem_u32(kt);
      const int g = lane >> 2, c = lane & 3;
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[0][i] = sc[1][i] = 0.f;
      if constexpr (FP8) {
        uint4 kw[2][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int key = g + mt * 8;
          kw[mt][0] = lds128(kbase + key * 128 + (((2 * c) ^ (key & 7)) << 4));
          kw[mt][1] = lds128(kbase + key * 128 + (((2 * c + 1) ^ (key & 7)) << 4));
        }
#pragma unroll
        for (int kk = 0; kk < S::kKS; ++kk) {  // (two accumulators: even and odd steps)
          const uint4& k0 = kw[0][kk >> 2];
          const uint4& k1 = kw[1][kk >> 2];
          const int sel = kk & 3;
          uint32_t a[4];
          e4m3x4_to_f16(sel == 0 ? k0.x : sel == 1 ? k0.y : sel == 2 ? k0.z : k0.w, a[0], a[2]);
          e4m3x4_to_f16(sel == 0 ? k1.x : sel == 1 ? k1.y : sel == 2 ? k1.z : k1.w, a[1], a[3]);
          mma_f16_16816(sc[kk & 1], a, qa[kk][0], qa[kk][2]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[0][i] = (sc[0][i] + sc[1][i]) * sk[i & 1];
        if (!seen_by_all(key0)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + g + 8 * (i >> 1), e = i & 1;
            if (!(key <= pos[e] && (key >= lo[e] || key < p.first))) sc[0][i] = -INFINITY;
          }
        }
      } else {
        const int mi = lane >> 3, rr = lane & 7;
        const int row = rr + ((mi >> 1) << 3);
#pragma unroll
        for (int kk = 0; kk < S::kKS; ++kk) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(kbase + tile_off<S::kHalves>(row, kk * 2 + (mi & 1)), b0, b1, b2, b3);
          mma_bf16_16816(sc[0], qa[kk], b0, b1);
          mma_bf16_16816(sc[1], qa[kk], b2, b3);
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[nt][i] *= sk[0];
        if (!seen_by_all(key0)) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key0 + 2 * c + 8 * nt + (i & 1), r = i >> 1;
              if (!(key <= pos[r] && (key >= lo[r] || key < p.first))) sc[nt][i] = -INFINITY;
            }
        }
      }
    };

    // ---- one pass over the keys
    float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.f, 0.f};
    constexpr int NO = FP8 ? 8 : S::kNT;
    float o[NO][4];
#pragma unroll
    for (int j = 0; j < NO; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    // room for the scores of the CTA's first `kept` blocks, [row][key]: shared memory (rows 8 words apart
    // in the banks) where all the cluster's fit, else the workspace
    float* scores = reinterpret_cast<float*>(ring + S::kOffScores);
    int ld = WEIGH && !NARROW ? S::kScores / 4 / nrow / 32 * 32 - 24 : 0;
    const int most = (nblk + C - 1) / C;  // blocks of a CTA
    if (WEIGH && most > ld / kBlk && p.w.room / nrow > ld) {
      ld = p.w.room / nrow / 32 * 32;
      scores = p.w.part + (int64_t)blockIdx.x * p.w.room;
    }
    const int kept = WEIGH ? min(count, ld / kBlk) : 0;
    bool late = false;
    for (int x = 0; x < mine; ++x) {
      const uint32_t cnt = ring_pos + x, slot = cnt % NS;
      // (one answer for the warp: a lane's own wait may run out just before the copy lands)
      if (!__all_sync(kFull, mbar_wait(&full[stall ? NW * NS : warp * NS + slot],
                                       stall ? 0u : (cnt / NS) & 1u, limit))) {
        late = true;
        break;
      }
      uint8_t* kt = ring + (size_t)(warp * NS + slot) * S::kStage;
      uint8_t* vt = kt + S::kTile;
      const int b = warp + NW * x, key0 = (run0 + b) * kBlk;
      const int g = lane >> 2, c = lane & 3;
      if (!FP8 && key0 + kBlk > vn) {
        // V rows past the sequence's end hold anything: zeros, so that 0 x NaN does not show
        const int first = vn - key0;
        for (int i = lane; i < (kBlk - first) * S::kHalves * 8; i += 32) {
          const int r = first + i / (S::kHalves * 8), ch = i % (S::kHalves * 8);
          *reinterpret_cast<uint4*>(vt + tile_off<S::kHalves>(r, ch)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      float sc[2][4];
      scores_of(kt, key0, sc);
      if (WEIGH && b < kept) {
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (2 * c + (i & 1) < nrow) scores[(2 * c + (i & 1)) * ld + b * kBlk + g + 8 * (i >> 1)] = sc[0][i];
        } else {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (g + 8 * r < nrow)
                *reinterpret_cast<float2*>(scores + (g + 8 * r) * ld + b * kBlk + 8 * nt + 2 * c) =
                    make_float2(sc[nt][2 * r], sc[nt][2 * r + 1]);
        }
      }
      float alpha[2];
      bool grew = false;  // a row's running maximum rose: its O needs the rescale (else alpha = 1)
      if constexpr (FP8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(sc[0][e], sc[0][2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
          const float mn = fmaxf(mrow[e], mx), base = mn == -INFINITY ? 0.f : mn;
          alpha[e] = exp2f(mrow[e] - base);
          grew |= mn > mrow[e];
          mrow[e] = mn;
          sc[0][e] = exp2f(sc[0][e] - base);
          sc[0][2 + e] = exp2f(sc[0][2 + e] - base);
          lrow[e] = lrow[e] * alpha[e] + (sc[0][e] + sc[0][2 + e]);
        }
        if (__any_sync(kFull, grew)) {
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            o[t][0] *= alpha[0];
            o[t][1] *= alpha[1];
            o[t][2] *= alpha[0];
            o[t][3] *= alpha[1];
          }
        }
        // (weights are taken 2^15 times as large, the row's largest so far just inside f16: what rounds
        // to a multiple of f16's smallest step is off by 2^-40 of it)
        constexpr float kUp = 32768.f;
        const uint32_t pb0 = movmatrix_trans(pack_f16x2(sc[0][0] * kUp, sc[0][1] * kUp));
        const uint32_t pb1 = movmatrix_trans(pack_f16x2(sc[0][2] * kUp, sc[0][3] * kUp));
        const uint32_t vbase = smem_u32(vt);
        const int lim = vn - key0;  // rows at or past it: zeros
        uint4 vr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * c + (i & 1) + (i >> 1) * 8;
          vr[i] = lds128(vbase + r * 128 + ((g ^ (r & 7)) << 4));
          if (r >= lim) vr[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        const uint32_t ra[4] = {vr[0].x, vr[0].y, vr[0].z, vr[0].w};
        const uint32_t rb[4] = {vr[1].x, vr[1].y, vr[1].z, vr[1].w};
        const uint32_t rc[4] = {vr[2].x, vr[2].y, vr[2].z, vr[2].w};
        const uint32_t rd[4] = {vr[3].x, vr[3].y, vr[3].z, vr[3].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo01 = __byte_perm(ra[i], rb[i], 0x5140), hi01 = __byte_perm(ra[i], rb[i], 0x7362);
          const uint32_t lo89 = __byte_perm(rc[i], rd[i], 0x5140), hi89 = __byte_perm(rc[i], rd[i], 0x7362);
          const uint32_t a0[4] = {e4m3x2_to_f16x2((uint16_t)(lo01 & 0xffffu)),
                                  e4m3x2_to_f16x2((uint16_t)(lo01 >> 16)),
                                  e4m3x2_to_f16x2((uint16_t)(lo89 & 0xffffu)),
                                  e4m3x2_to_f16x2((uint16_t)(lo89 >> 16))};
          const uint32_t a1[4] = {e4m3x2_to_f16x2((uint16_t)(hi01 & 0xffffu)),
                                  e4m3x2_to_f16x2((uint16_t)(hi01 >> 16)),
                                  e4m3x2_to_f16x2((uint16_t)(hi89 & 0xffffu)),
                                  e4m3x2_to_f16x2((uint16_t)(hi89 >> 16))};
          mma_f16_16816(o[2 * i], a0, pb0, pb1);
          mma_f16_16816(o[2 * i + 1], a1, pb0, pb1);
        }
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
          const float mn = fmaxf(mrow[r], mx), base = mn == -INFINITY ? 0.f : mn;
          alpha[r] = exp2f(mrow[r] - base);
          grew |= mn > mrow[r];
          mrow[r] = mn;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            sc[nt][2 * r] = exp2f(sc[nt][2 * r] - base);
            sc[nt][2 * r + 1] = exp2f(sc[nt][2 * r + 1] - base);
          }
          lrow[r] = lrow[r] * alpha[r] + ((sc[0][2 * r] + sc[0][2 * r + 1]) + (sc[1][2 * r] + sc[1][2 * r + 1]));
        }
        uint32_t ph[4], pl[4];  // P as a bf16 pair: the weights keep 2^-17
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = sc[i >> 1][(i & 1) * 2], d = sc[i >> 1][(i & 1) * 2 + 1];
          ph[i] = pack_bf16x2(a, d);
          const float2 hv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ph[i]));
          pl[i] = pack_bf16x2(a - hv.x, d - hv.y);
        }
        if (__any_sync(kFull, grew)) {
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            o[j][0] *= alpha[0];
            o[j][1] *= alpha[0];
            o[j][2] *= alpha[1];
            o[j][3] *= alpha[1];
          }
        }
        const int mi = lane >> 3, rr = lane & 7;
        const int row = rr + ((mi & 1) << 3);
        const uint32_t vbase = smem_u32(vt);
#pragma unroll
        for (int dd = 0; dd < D / 16; ++dd) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_trans(vbase + tile_off<S::kHalves>(row, dd * 2 + (mi >> 1)), b0, b1, b2, b3);
          mma_bf16_16816(o[2 * dd], ph, b0, b1);
          mma_bf16_16816(o[2 * dd + 1], ph, b2, b3);
          mma_bf16_16816(o[2 * dd], pl, b0, b1);
          mma_bf16_16816(o[2 * dd + 1], pl, b2, b3);
        }
      }
      __syncwarp();
      if (issued < mine) {
        issue(issued, ring_pos + issued, true);
        ++issued;
      }
    }
    if (late) {
      if (lane == 0) {
        record_error(p.status, PA_ETIMEOUT);
        atomicExch(&sh.fail, 1);
      }
      // wait (bounded) for this warp's copies still in flight
      for (int x = max(0, issued - NS); x < issued; ++x)
        mbar_wait(&full[warp * NS + (ring_pos + x) % NS], ((ring_pos + x) / NS) & 1u, 100000000ull);
    }
    ring_pos += issued;

    // ---- the warps' states
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (FP8) {
        lrow[r] += __shfl_xor_sync(kFull, lrow[r], 4);
        lrow[r] += __shfl_xor_sync(kFull, lrow[r], 8);
        lrow[r] += __shfl_xor_sync(kFull, lrow[r], 16);
      } else {
        lrow[r] += __shfl_xor_sync(kFull, lrow[r], 1);
        lrow[r] += __shfl_xor_sync(kFull, lrow[r], 2);
      }
    }
    __syncthreads();  // every warp is done with its ring
    {
      float* ob = mrg_o + (size_t)warp * 16 * LD;
      const int g = lane >> 2, c = lane & 3;
      if constexpr (FP8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 2 * c + e;
          if (g == 0) sh.warp_ml[warp][row] = make_float2(mrow[e], lrow[e]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(ob + row * LD + 16 * g + 4 * i) =
                make_float4(o[2 * i][e] * (1.f / 32768.f), o[2 * i][2 + e] * (1.f / 32768.f),
                            o[2 * i + 1][e] * (1.f / 32768.f), o[2 * i + 1][2 + e] * (1.f / 32768.f));
        }
      } else {
        if (c == 0) {
          sh.warp_ml[warp][g] = make_float2(mrow[0], lrow[0]);
          sh.warp_ml[warp][g + 8] = make_float2(mrow[1], lrow[1]);
        }
#pragma unroll
        for (int j = 0; j < S::kNT; ++j) {
          const int col = j * 8 + c * 2;
          *reinterpret_cast<float2*>(ob + g * LD + col) = make_float2(o[j][0], o[j][1]);
          *reinterpret_cast<float2*>(ob + (g + 8) * LD + col) = make_float2(o[j][2], o[j][3]);
        }
      }
    }
    if (!waited && !p.after_tc) {
      // the check of the batch is complete; whatever follows on the stream may be prepared
      pdl_wait();
      pdl_launch_dependents();
      waited = true;
    }
    if (tid == 0 && row0 == 0 && status_set(p.status)) atomicExch(&sh.fail, 1);
    __syncthreads();
    // (a row with scores of NaN keeps l NaN: a warp without a finite score has m -inf, and its factor 0
    // makes 0 x NaN)
    if (tid < nrow) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, sh.warp_ml[w][tid].x);
      const float base = M == -INFINITY ? 0.f : M;
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = exp2f(sh.warp_ml[w][tid].x - base);
        L += f * sh.warp_ml[w][tid].y;
        sh.warp_ml[w][tid].x = f;
      }
      sh.ml[tid] = make_float2(M, L);
    }
    __syncthreads();
    for (int i = tid; i < nrow * (D / 4); i += NW * 32) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = sh.warp_ml[w][r].x;
        const float4 v = *reinterpret_cast<const float4*>(mrg_o + ((size_t)w * 16 + r) * LD + d);
        a.x += f * v.x;
        a.y += f * v.y;
        a.z += f * v.z;
        a.w += f * v.w;
      }
      *reinterpret_cast<float4*>(state + r * LD + d) = a;
    }
    if (C > 1) cluster_sync(); else __syncthreads();

    // ---- the cluster's
    bool fail = sh.fail != 0;
    if (C > 1) {
      fail = lane < C && peer_u32(peer(&sh.fail, lane)) != 0;
      fail = __any_sync(kFull, fail);
    }
    // a warp to a row, a lane to a CTA: all states of a row are requested at once
    for (int r = warp; r < nrow; r += NW) {
      const float2 st = lane >= C ? make_float2(-INFINITY, 0.f)
                        : C > 1   ? peer_f2(peer(&sh.ml[r], lane))
                                  : sh.ml[r];
      float M = st.x;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, k));
      const float base = M == -INFINITY ? 0.f : M;
      const float f = exp2f(st.x - base);
      float L = f * st.y;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) L += __shfl_xor_sync(kFull, L, k);
      if (lane < 16) sh.factor[r][lane] = f;
      if (lane == 0) {
        const int R = row0 + r, t = qs + R / G, h = kvh * G + R % G;
        // tree_finish takes the sink into the sum; the log-sum-exp with it, in log2 units, is the weights'
        const float sink = m.sinks ? m.sinks[h] * kLog2e : -INFINITY;
        float M2 = fmaxf(M, sink);
        if (M2 == -INFINITY) M2 = 0.f;
        const float total = L * exp2f(M - M2) + exp2f(sink - M2);
        // (a row without a finite score gives no weight; one of NaN infinite ones, which become NaN when they
        // are added, but nothing to the keys that it does not see, of score -inf)
        const float lse = L == 0.f ? INFINITY : M2 + log2f(total);
        sh.lse[r] = lse == lse ? lse : -FLT_MAX;
        if (WEIGH && lse != lse) sh.nan = row0 + 1;
        sh.norm[r] = tree_finish(p, kvh, h, t, M, L, rank == 0 && !fail);
      }
    }
    __syncthreads();
    if (!fail) {
      const int items = nrow * (D / 4);
      for (int i = items * rank / C + tid; i < items * (rank + 1) / C; i += NW * 32) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (C > 1) {
          for (int k0 = 0; k0 < C; k0 += 8) {
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[k] = k0 + k < C ? peer_f4(peer(state + r * LD + d, k0 + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float f = sh.factor[r][k0 + k];
              a.x += f * v[k].x;
              a.y += f * v[k].y;
              a.z += f * v[k].z;
              a.w += f * v[k].w;
            }
          }
        } else {
          a = *reinterpret_cast<const float4*>(state + r * LD + d);
        }
        const float f = sh.norm[r];
        const int R = row0 + r;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                  ((int64_t)(qs + R / G) * H + kvh * G + R % G) * D + d) =
            make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
      }
    }
    // the states have been read
    fence_proxy_async_smem();
    if (C > 1) cluster_arrive();
    bool reused = false;  // the ring: every CTA of the cluster has read the states
    if constexpr (WEIGH) {
      float* w = p.key_weights + ((int64_t)s * m.num_kv_heads + kvh) * p.weights_len;
      auto real = [&](int key) { return key >= front * kBlk ? key + gap * kBlk : key; };
      // One thread adds to a key, a row tile after the other (another CTA's, perhaps, behind the cluster's
      // barrier): atomic only so that L2 adds, and nobody waits for the sum that was there.
      auto add = [&](int key, float v) {
        if (v != 0.f && key < vn) atomicAdd(w + real(key), fmaf(v, 0.f, v));
      };
      const int r0 = max(0, counted0 - row0);
      constexpr int kU = 4;
      if (!fail)
        // four keys of one block to a step, kU steps' loads in flight
        for (int i0 = tid; i0 < kept * 4; i0 += kU * NW * 32) {
          float4 v[kU];
          int at[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int i = i0 + u * NW * 32, key = run0 * kBlk + 4 * i;
            at[u] = i < kept * 4 ? real(key) : INT_MAX;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          for (int r = r0; r < nrow; r += 4) {
            float4 x[4][kU];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int u = 0; u < kU; ++u)
                x[k][u] = at[u] < n && r + k < nrow
                              ? *reinterpret_cast<const float4*>(scores + (r + k) * ld + 4 * (i0 + u * NW * 32))
                              : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float l = sh.lse[min(r + k, nrow - 1)];
#pragma unroll
              for (int u = 0; u < kU; ++u) {
                v[u].x += exp2f(x[k][u].x - l);
                v[u].y += exp2f(x[k][u].y - l);
                v[u].z += exp2f(x[k][u].z - l);
                v[u].w += exp2f(x[k][u].w - l);
              }
            }
          }
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const float y[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (at[u] < n - k && y[k] != 0.f) atomicAdd(w + at[u] + k, fmaf(y[k], 0.f, y[k]));
          }
        }
      if (most > ld / kBlk) {  // (one answer for the cluster)
        // the blocks whose scores did not fit: K once more
        if (C > 1) cluster_wait(); else __syncthreads();  // (the states in the ring have been read)
        reused = true;
        const int x0 = kept > warp ? (kept - warp + NW - 1) / NW : 0;  // this warp's first
        int sent = x0;
        for (; sent < min(mine, x0 + NS); ++sent) issue(sent, ring_pos + sent - x0, false);
        bool stop = fail;
        for (int x = x0; x < mine && !stop; ++x) {
          const uint32_t cnt = ring_pos + x - x0, slot = cnt % NS;
          if (!__all_sync(kFull, mbar_wait(&full[warp * NS + slot], (cnt / NS) & 1u, limit))) {
            if (lane == 0) {
              record_error(p.status, PA_ETIMEOUT);
              atomicExch(&sh.fail, 1);
            }
            break;
          }
          const int key0 = (run0 + warp + NW * x) * kBlk, g = lane >> 2, c = lane & 3;
          float sc[2][4];
          scores_of(ring + (size_t)(warp * NS + slot) * S::kStage, key0, sc);
          __syncwarp();
          if (sent < mine) {
            issue(sent, ring_pos + sent - x0, false);
            ++sent;
          }
          if constexpr (FP8) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              v[h] = 0.f;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = 2 * c + e;
                if (r >= r0 && r < nrow) v[h] += exp2f(sc[0][2 * h + e] - sh.lse[r]);
              }
              v[h] += __shfl_xor_sync(kFull, v[h], 1);
              v[h] += __shfl_xor_sync(kFull, v[h], 2);
            }
            if (c < 2) add(key0 + g + 8 * c, c ? v[1] : v[0]);
          } else {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i] = 0.f;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h;
                if (r >= r0 && r < nrow) v[i] += exp2f(sc[i >> 1][2 * h + (i & 1)] - sh.lse[r]);
              }
              v[i] += __shfl_xor_sync(kFull, v[i], 4);
              v[i] += __shfl_xor_sync(kFull, v[i], 8);
              v[i] += __shfl_xor_sync(kFull, v[i], 16);
            }
            // lanes 0 .. 3 of row group i have key 2c + (i & 1) + 8 (i >> 1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (g == i) add(key0 + 2 * c + (i & 1) + 8 * (i >> 1), v[i]);
          }
        }
        // (copies in flight when it stopped early)
        for (int x = max(x0, sent - NS); x < sent; ++x)
          mbar_wait(&full[warp * NS + (ring_pos + x - x0) % NS], ((ring_pos + x - x0) / NS) & 1u, 100000000ull);
        ring_pos += sent - x0;
      }
      // a row of NaN spoils all that it sees, keys of score -inf (q or K with an infinity) among them
      if (sh.nan == row0 + 1 && !fail)
        for (int r = r0; r < nrow; ++r) {
          if (sh.lse[r] != -FLT_MAX) continue;
          const int at = pos_of(r);
          for (int key = run0 * kBlk + tid; key < min(run1 * kBlk, at + 1); key += NW * 32)
            if (m.window <= 0 || key > at - m.window || key < p.first) atomicAdd(w + real(key), NAN);
        }
    }
    // the ring, or the CTA, may go when all have read
    if (reused)
      fence_proxy_async_smem();
    else if (C > 1)
      cluster_wait();
    __syncthreads();
  }
  if (!waited) {
    // a sequence without rows; beside the prefill kernel one CTA stays for it, so that what follows on
    // the stream finds both done
    pdl_launch_dependents();
    if (!p.after_tc || blockIdx.x == gridDim.x - 1) pdl_wait();
  }
}

template <int D, bool FP8, bool WEIGH, int KIND>
cudaError_t launch_as(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, uint64_t limit,
                      uint32_t stall, cudaStream_t stream) {
  using S = Shape<D, FP8, KIND>;
  auto kern = k_window_decode<D, FP8, WEIGH, KIND>;
  const int smem = (int)S::smem(WEIGH);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && p.cluster > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.m.num_seqs * p.m.num_kv_heads * p.cluster));
  cfg.blockDim = dim3(S::NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, p, limit, stall);
}
template <int D, bool FP8>
cudaError_t launch_sum(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, uint64_t limit,
                       uint32_t stall, cudaStream_t stream) {
  const bool w = p.key_weights != nullptr;
  if (p.shape == kNarrow)
    return w ? launch_as<D, FP8, true, kNarrow>(tk, tv, p, limit, stall, stream)
             : launch_as<D, FP8, false, kNarrow>(tk, tv, p, limit, stall, stream);
  if constexpr (!FP8)
    if (p.shape == kBroad)
      return w ? launch_as<D, FP8, true, kBroad>(tk, tv, p, limit, stall, stream)
               : launch_as<D, FP8, false, kBroad>(tk, tv, p, limit, stall, stream);
  return w ? launch_as<D, FP8, true, kPlain>(tk, tv, p, limit, stall, stream)
           : launch_as<D, FP8, false, kPlain>(tk, tv, p, limit, stall, stream);
}

}  // namespace

cudaError_t launch_window_decode(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                                 bool fp8, uint64_t limit, uint32_t stall, cudaStream_t stream) {
  if (fp8) return launch_sum<128, true>(tk, tv, p, limit, stall, stream);
  if (p.m.head_dim == 128) return launch_sum<128, false>(tk, tv, p, limit, stall, stream);
  return launch_sum<64, false>(tk, tv, p, limit, stall, stream);
}

}  // namespace pa
