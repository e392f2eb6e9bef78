// k_window.cu -- causal attention over the paged cache behind a sliding window whose first tokens stay
// visible: the planning kernel and the general kernel's launch (k_tree_generic.cuh; on the tensor cores
// k_window_tc.cu).
//
// Math.  A token at position p sees key j when j <= p and (j > p - w or j < f): the window's w keys and
// the sequence's first f.  Without a window (w = 0) it sees all j <= p.
//
// Layout of the work.  An item is one (sequence, kv head) and up to rows_per_item query rows.  With a
// window, the blocks between the first tokens' and the first one that any of its rows reaches are left
// out: the item's keys are counted without that gap, so its key tiles are full of visible keys.  (A
// tile of 128 keys for the first tokens alone would cost a decoding token behind a window of 1024 an
// eighth of its time.)  A sequence's positions do not decrease, so an item's keys follow from its first
// and last token alone.
// The items' tiles are laid end to end, weighted, and cut into equal shares, one contiguous range
// per CTA; the pieces of a cut item are merged in key order (k_tree.cu).  Chunks of prompts and
// decoding tokens lie in the same list, so some SMs stream keys while others compute.
// Large batches of chunks go to the prefill kernel instead (k_prefill_tc.cu): whole items, the longest
// first, on as many pairs of SMs as end together with the decoding sequences on the others
// (k_window_decode.cu).  Batches of decoding tokens alone are not planned, only checked.
#include <algorithm>

#include "k_tree_generic.cuh"
#include "k_window.cuh"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCumShared = 2048;   // sequences whose prefix sums the planner keeps in shared memory

// In front of k_window_decode, which starts once every block has waited for the work ahead and waits for
// the end of this kernel before it writes.
__global__ void __launch_bounds__(256) k_window_check(const TreeParams p) {
  const VarlenMeta& m = p.m;
  pdl_wait();
  pdl_launch_dependents();
  const int at = blockIdx.x * 256 + threadIdx.x, threads = gridDim.x * 256;
  bool bad = blockIdx.x == 0 && bad_scales(p, threadIdx.x, 256);
  for (int s = at; s < m.num_seqs; s += threads) {
    int qs, q, n;
    bad |= !sequence(p, s, qs, q, n);
  }
  bad |= bad_reads(p, at >> 5, threads >> 5);
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) record_error(p.status, PA_EINVAL);
}

// The first of a sequence's tokens [a, b) at position `at` or later (b: none).  Mostly they are
// consecutive: then it is found at once.
__device__ __forceinline__ int token_from(const int32_t* pos, int a, int b, int64_t at) {
  const int64_t guess = a + max(at - pos[a], (int64_t)0);
  if (guess == a) return a;
  if (guess < b && pos[guess] == at && pos[guess - 1] < at) return (int)guess;
  while (a < b) {
    const int mid = a + (b - a) / 2;
    if (pos[mid] < at) a = mid + 1; else b = mid;
  }
  return a;
}

// Warp `me` of `warps`, for batches that go to the prefill kernel: marks the (sequence, kv head)s in whose V no
// value of 2^-9 or more is found.  That kernel holds V in f16, off by up to 2^-25 below 2^-14: 2^-16 of such a
// value, but all of a V of 1e-8, so items of marked ones are done again with V as it is.  8 values of each of 32
// rows at a time; mostly the first ones say so.  (A look by the prefill kernel's converters or producers, which
// have the values at hand, took 2 to 6 % of a call.)  Returns whether it marked one.
__device__ bool mark_small_values(const TreeParams& p, int me, int warps) {
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31;
  const int64_t units = (int64_t)m.num_seqs * m.num_kv_heads;
  bool marked = false;
  for (int64_t u = me; u < units; u += warps) {
    const int s = (int)(u / m.num_kv_heads), g = (int)(u % m.num_kv_heads);
    int qs, q, n;
    sequence(p, s, qs, q, n);
    if (q * m.group <= kWindowDecodeRows) continue;
    const Keys k = keys_from(p, m.window > 0 ? m.positions[qs] : 0);
    const int blocks = (int)(((int64_t)n + 15) / 16) - k.gap;
    const int32_t* row = m.block_tables + (int64_t)s * m.max_blocks;
    // 16 bytes of the first row of a block; the chunks of a block's row change with the lane
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v_blocks) + (int64_t)g * m.head_dim +
                             lane % (m.head_dim / 8) * 8;
    bool found = false;
    for (int b0 = 0; b0 < blocks && !found; b0 += 32) {
      const int b = b0 + lane, id = b < blocks ? row[b < k.front ? b : b + k.gap] : -1;
      uint32_t x = 0;
      if (id >= 0 && (int64_t)id < m.num_blocks) {
        const uint4 w = *reinterpret_cast<const uint4*>(v + (int64_t)id * 16 * m.num_kv_heads * m.head_dim);
        x = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                     __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
      }
      found = __any_sync(0xffffffffu, max(x & 0xffffu, x >> 16) >= 0x3b00u);  // (bf16 2^-9)
    }
    if (lane == 0) p.tc.plan[p.tc.small_off + kSmallBlocks + u] = !found;
    marked |= !found;
  }
  return marked;
}

// One block, for batches that go to the prefill kernel: its items, those of the most keys first (a counting
// sort, sixteen buckets to an octave), and how many pairs of CTAs take them: the number that ends both it
// and the decoding sequences beside it soonest.
__device__ void plan_prefill(const TreeParams& p, int items, int64_t* s_scratch) {
  const VarlenMeta& m = p.m;
  constexpr int kBuckets = 512;
  __shared__ int s_at[kBuckets];
  __shared__ unsigned long long s_tiles, s_keys;
  __shared__ unsigned int s_best;
  const int tid = threadIdx.x;
  int* s_warp = reinterpret_cast<int*>(s_scratch);
  auto bucket = [](int keys) {  // 0: the most (float bits from the exponent down to four of the fraction)
    return kBuckets - 1 - ((int)(__float_as_uint((float)keys) >> 19) - (127 << 4));
  };
  if (tid < kBuckets) s_at[tid] = 0;
  if (tid == 0) {
    s_tiles = s_keys = 0;
    s_best = ~0u;
  }
  __syncthreads();
  unsigned long long tiles = 0, keys = 0;
  for (int i = tid; i < items; i += kPlanThreads) {
    const int4 k = p.item_keys[i];
    if (p.seqs[2 * k.x + 1].z > kWindowDecodeRows) {
      tiles += k.z;
      atomicAdd(&s_at[bucket(k.w)], 1);
    } else {
      keys += k.w;
    }
  }
  if (tiles) atomicAdd(&s_tiles, tiles);
  if (keys) atomicAdd(&s_keys, keys);
  __syncthreads();
  int total;
  const int at = block_exclusive_scan(tid < kBuckets ? s_at[tid] : 0, s_warp, &total);
  if (tid < kBuckets) s_at[tid] = at;
  __syncthreads();
  int4* list = reinterpret_cast<int4*>(p.tc.plan + p.tc.items_off);
  for (int i = tid; i < items; i += kPlanThreads) {
    const int4 k = p.item_keys[i], w = p.seqs[2 * k.x + 1];
    if (w.z <= kWindowDecodeRows) continue;
    const int to = atomicAdd(&s_at[bucket(k.w)], 1);
    list[to] = make_int4(k.x, i - w.y, k.y, k.w);
    p.tc.plan[p.tc.redo_off + to] = 0;
  }
  // k pairs: a key tile of 256 rows takes a pair 1.1 us; decoding sequences stream at the memory's rate
  // on 80 SMs or more (the other pairs' SMs), and on all when the prefill items have ended
  if (tid < p.tc.pairs) {
    const int k = tid + 1, left = p.tc.num_sms - 2 * k;
    const float prefill = (float)s_tiles * m.num_kv_heads * 1.1f / k;
    const float stream = (float)s_keys * p.tc.decode_bytes_per_key / 6.7e6f;  // us on all SMs
    const float rate = min(1.f, left / 80.f);  // while the prefill items run
    const float time = prefill * rate >= stream ? prefill : prefill + (stream - prefill * rate);
    atomicMin(&s_best, ((unsigned)min(time, 1e6f) << 8) | (unsigned)(p.tc.pairs - k));
  }
  __syncthreads();
  if (tid == 0) {
    p.tc.plan[1] = total;
    p.tc.plan[3] = 0;
    p.tc.plan[5] = p.tc.pairs - (int)(s_best & 255u);
  }
}

// The work of an item of the key weights, in about hundredths of a microsecond (only the balance
// between the CTAs depends on it): its keys, and each row tile.
constexpr int kWeightItem = 150, kWeightRowTile = 100;

// One block: the plan of the key weights (k_weights_tc.cu).  It checks what it uses as an index and
// leaves the errors to block 0, which finds the same; a batch that is not valid has no items.
__device__ void plan_weights(const TreeParams& p, int64_t* s_warp, int64_t* s_cum, int* s_base) {
  const VarlenMeta& m = p.m;
  const int tid = threadIdx.x;
  const bool shared = m.num_seqs <= kCumShared;
  bool bad = false;
  int64_t items = 0;
  for (int s0 = 0; s0 < m.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int qs = 0, q = 0, n = 0, mine = 0;
    int4 first = make_int4(0, 0, 0, 0);
    if (s < m.num_seqs) {
      bad |= !sequence(p, s, qs, q, n);
      // (the others' weights are added where they decode)
      if (q > 0 && !(p.tc.plan && q * m.group <= kWindowDecodeRows)) {
        // the keys that counted tokens see: those of the first positions, and from lo to the last one
        const int skip = p.observed > 0 ? max(0, q - p.observed) : 0;
        const int low = m.positions[qs + skip], last = m.positions[qs + q - 1];
        bad |= low < 0 || last < low || last >= n;
        const int end = min(max(last, 0), n - 1) / kWeightKeys + 1;
        const int lo = m.window > 0 ? max(min(max(low, 0), n - 1) - m.window + 1, 0) / kWeightKeys : 0;
        const int front = m.window > 0 ? min((int)(((int64_t)p.first + kWeightKeys - 1) / kWeightKeys), end) : 0;
        const int gap = max(lo - front, 0);
        mine = max(end - gap, 0);
        first = make_int4(0, 0, front, gap);
        p.w.seqs[2 * s + 1] = make_int4(qs + skip, q - skip, n, 0);
      }
    }
    int64_t total;
    const int64_t at = items + block_sum_scan(mine, s_warp, &total);
    if (s < m.num_seqs) {
      p.w.seqs[2 * s] = make_int4((int)at, mine, first.z, first.w);
      if (shared) s_base[s] = (int)at;
    }
    items += total;
  }
  if (__syncthreads_or(bad)) items = 0;
  int64_t base = 0;
  for (int64_t i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int64_t i = i0 + tid;
    int64_t weight = 0;
    if (i < items) {
      int lo = 0, hi = m.num_seqs;  // the last sequence whose first item is at most i: it has items
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((shared ? s_base[mid] : p.w.seqs[2 * mid].x) <= i) lo = mid; else hi = mid;
      }
      const int4 r = p.w.seqs[2 * lo], t = p.w.seqs[2 * lo + 1];
      int tile = (int)(i - r.x);
      if (tile >= r.z) tile += r.w;
      const int64_t key0 = (int64_t)tile * kWeightKeys;
      // tokens that see one of the keys at least
      const int a = token_from(m.positions, t.x, t.x + t.y, key0) - t.x;
      int b = t.y;
      if (m.window > 0 && key0 >= p.first)
        b = token_from(m.positions, t.x, t.x + t.y, key0 + kWeightKeys - 1 + m.window) - t.x;
      // (an item between the tokens' positions, where these skip, may be seen by none)
      const int r0 = a / p.tile_tokens, r1 = max((b + p.tile_tokens - 1) / p.tile_tokens, r0 + 1);
      p.w.items[i] = make_int4(tile, r0, r1, 0);
      weight = kWeightItem + (int64_t)kWeightRowTile * (r1 - r0);
    }
    int64_t total;
    const int64_t at = base + block_sum_scan(weight, s_warp, &total);
    if (i < items) p.w.cum[i] = at;
    base += total;
  }
  if (tid == 0) p.w.cum[items] = base;
  __syncthreads();
  if (items == 0) {
    for (int s = tid; s < m.num_seqs; s += kPlanThreads) p.w.seqs[2 * s] = make_int4(0, 0, 0, 0);
    for (int c = tid; c <= p.w.grid; c += kPlanThreads) p.w.starts[c] = make_int4(m.num_seqs, 0, 0, 0);
    return;
  }
  for (int s = tid; shared && s <= m.num_seqs; s += kPlanThreads)
    s_cum[s] = (s < m.num_seqs ? p.w.cum[p.w.seqs[2 * s].x] : base) * m.num_kv_heads;
  __syncthreads();
  base *= m.num_kv_heads;
  for (int c = tid; c <= p.w.grid; c += kPlanThreads) {
    int4 st = make_int4(m.num_seqs, 0, 0, 0);
    if (c < p.w.grid) {
      auto before = [&](int s) {
        return shared ? s_cum[s]
                      : (s < m.num_seqs ? p.w.cum[p.w.seqs[2 * s].x] * m.num_kv_heads : base);
      };
      const int64_t x = base / p.w.grid * c + base % p.w.grid * c / p.w.grid;  // floor(base c / grid)
      int lo = 0, hi = m.num_seqs;  // the last sequence with no more weight before it
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before(mid) <= x) lo = mid; else hi = mid;
      }
      const int64_t at = before(lo), per_head = (before(lo + 1) - at) / m.num_kv_heads;
      const int4 r = p.w.seqs[2 * lo];
      const int kvh = (int)((x - at) / per_head);
      const int64_t rem = (x - at) % per_head, cum0 = p.w.cum[r.x];
      int it = 0, top = r.y;
      while (top - it > 1) {
        const int mid = (it + top) >> 1;
        if (p.w.cum[r.x + mid] - cum0 <= rem) it = mid; else top = mid;
      }
      const int4 w = p.w.items[r.x + it];
      const int64_t in = max(rem - (p.w.cum[r.x + it] - cum0) - kWeightItem, (int64_t)0);
      st = make_int4(lo, kvh, it, (int)min(w.y + in / kWeightRowTile, (int64_t)w.z - 1));
    }
    p.w.starts[c] = st;
  }
}

// Block 0 plans (block 1 the key weights, where they are asked for); the blocks behind check the
// sequences' positions and table entries.  Everything is read after the wait for the kernels ahead, and
// no output is written before this launch is done.  A plan that failed is one of empty shares and of
// sequences without tokens, so the kernels behind do nothing even where another stream has cleared the
// status word in between.
__global__ void __launch_bounds__(kPlanThreads) k_window_plan(const TreeParams p) {
  __shared__ int64_t s_warp[32];
  __shared__ int64_t s_cum[kCumShared + 1];
  __shared__ int s_base[kCumShared + 1];
  const VarlenMeta& m = p.m;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  const int planners = p.w.grid > 0 ? 2 : 1;
  if (blockIdx.x == 1 && planners == 2) {
    plan_weights(p, s_warp, s_cum, s_base);
    return;
  }
  if (blockIdx.x > 0) {
    const int warps = (gridDim.x - planners) * (kPlanThreads / 32);
    bad = bad_reads(p, (blockIdx.x - planners) * (kPlanThreads / 32) + warp, warps);
    if (p.tc.small_off) {
      const int block = blockIdx.x - planners, blocks = gridDim.x - planners;
      const int any = __syncthreads_or(mark_small_values(p, block * (kPlanThreads / 32) + warp, warps));
      if (tid < kSmallBlocks && tid % blocks == block) p.tc.plan[p.tc.small_off + tid] = any;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(p.status, PA_EINVAL);
    return;
  }

  bad = bad_scales(p, tid, kPlanThreads);
  const bool shared = m.num_seqs <= kCumShared;
  int64_t items = 0;
  for (int s0 = 0; s0 < m.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int qs = 0, q = 0, n = 0;
    if (s < m.num_seqs) bad |= !sequence(p, s, qs, q, n);
    const int rows = q * m.group, mine = (rows + p.rows_per_item - 1) / p.rows_per_item;
    int64_t total;
    const int64_t at = items + block_sum_scan(mine, s_warp, &total);
    if (s < m.num_seqs) {
      p.seqs[2 * s] = make_int4(qs, q, n, 0);
      p.seqs[2 * s + 1] = make_int4(mine, (int)at, rows, 0);
      if (shared) s_base[s] = (int)at;
    }
    items += total;
  }
  // (query_start_loc may be anything: a batch that is not valid has no items, however many it counts)
  if (__syncthreads_or(bad)) items = 0;

  // the items' keys and weights
  int64_t base = 0;
  for (int64_t i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int64_t i = i0 + tid;
    int64_t weight = 0;
    if (i < items) {
      int lo = 0, hi = m.num_seqs;  // the last sequence whose first item is at most i: it has items
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((shared ? s_base[mid] : p.seqs[2 * mid + 1].y) <= i) lo = mid; else hi = mid;
      }
      const int4 q = p.seqs[2 * lo], w = p.seqs[2 * lo + 1];
      const int row0 = (int)(i - w.y) * p.rows_per_item, rows = min(p.rows_per_item, w.z - row0);
      const int a = m.positions[q.x + row0 / m.group];
      const int b = m.positions[q.x + (row0 + rows - 1) / m.group];
      bad |= a < 0 || b < a || b >= q.z;
      const Keys k = keys_from(p, a);
      const int end = min(max(b, a), q.z - 1) + 1 - k.gap * m.block_size;
      const int tiles = max(1, (end + p.key_tile - 1) / p.key_tile);
      p.item_keys[i] = make_int4(lo, k.gap, tiles, max(end, 1));
      weight = (int64_t)tree_weight(p, rows) * tiles + kTreeItemWeight;
    }
    if (p.tc.plan) continue;  // (no shares)
    int64_t total;
    const int64_t at = base + block_sum_scan(weight, s_warp, &total);
    if (i < items) p.item_cum[i] = at;
    base += total;
  }
  if (tid == 0 && !p.tc.plan) p.item_cum[items] = base;
  bad = __syncthreads_or(bad);  // (and the items' records can be read)
  if (bad) {
    if (tid == 0) record_error(p.status, PA_EINVAL);
    for (int s = tid; s < m.num_seqs; s += kPlanThreads)
      p.seqs[2 * s] = p.seqs[2 * s + 1] = make_int4(0, 0, 0, 0);
  }
  if (p.tc.plan) {
    plan_prefill(p, bad ? 0 : (int)items, s_warp);
    return;
  }
  if (bad) {
    for (int c = tid; c <= p.grid; c += kPlanThreads) p.starts[c] = make_int4(m.num_seqs, 0, 0, 0);
    return;
  }
  for (int s = tid; s <= m.num_seqs; s += kPlanThreads) {
    const int64_t at = s < m.num_seqs ? p.item_cum[p.seqs[2 * s + 1].y] * m.num_kv_heads
                                      : base * m.num_kv_heads;
    if (shared) s_cum[s] = at; else p.cum[s] = at;
  }
  __syncthreads();
  // where each CTA's share begins
  base *= m.num_kv_heads;
  for (int c = tid; c <= p.grid; c += kPlanThreads) {
    int4 st = make_int4(m.num_seqs, 0, 0, 0);
    if (c < p.grid && base > 0) {
      const int64_t x = base / p.grid * c + base % p.grid * c / p.grid;  // floor(base c / grid)
      int lo = 0, hi = m.num_seqs;  // the last sequence with cum <= x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((shared ? s_cum[mid] : p.cum[mid]) <= x) lo = mid; else hi = mid;
      }
      const int64_t before = shared ? s_cum[lo] : p.cum[lo];
      const int64_t per_head = ((shared ? s_cum[lo + 1] : p.cum[lo + 1]) - before) / m.num_kv_heads;
      const int4 w = p.seqs[2 * lo + 1];
      const int kvh = (int)((x - before) / per_head);
      const int64_t r = (x - before) % per_head, cum0 = p.item_cum[w.y];
      int it = 0, top = w.x;  // the last item with cum <= r
      while (top - it > 1) {
        const int mid = (it + top) >> 1;
        if (p.item_cum[w.y + mid] - cum0 <= r) it = mid; else top = mid;
      }
      const int64_t in = max(r - (p.item_cum[w.y + it] - cum0) - kTreeItemWeight, (int64_t)0);
      const int tw = tree_weight(p, min(p.rows_per_item, w.z - it * p.rows_per_item));
      st = make_int4(lo, kvh, it, (int)min(in / tw, (int64_t)p.item_keys[w.y + it].z - 1));
    }
    p.starts[c] = st;
  }
}

}  // namespace

WindowLayout window_layout(int32_t num_seqs, int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                           int32_t head_dim, int64_t max_keys, int32_t rows_per_item, int32_t key_tile,
                           int32_t max_grid, bool weights) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  const int32_t group = num_heads / num_kv_heads;
  const TreeLayout t = tree_layout(num_seqs, num_tokens, group, num_kv_heads, head_dim, max_keys,
                                   rows_per_item, key_tile, max_grid);
  const int64_t items = (num_tokens * group + rows_per_item - 1) / rows_per_item + num_seqs;
  WindowLayout L;
  L.tree = t;
  L.items_off = t.bytes;
  L.item_cum_off = L.items_off + up(16 * items);
  L.tc_off = L.item_cum_off + up(8 * (items + 1));
  // header words, items, marks, list of marked items, marks of small values
  L.lse_off = L.tc_off + up(4 * (kPlanHeaderWords + 6 * items + kSmallBlocks + (int64_t)num_seqs * num_kv_heads));
  L.bytes = L.w_seqs_off = L.lse_off + (weights ? up(4 * num_tokens * num_heads) : 0);
  if (!weights) return L;
  const int64_t key_items = std::min<int64_t>(num_seqs, num_tokens) * ((max_keys + kWeightKeys - 1) / kWeightKeys);
  L.w_items_off = L.w_seqs_off + up(32 * (int64_t)num_seqs);
  L.w_cum_off = L.w_items_off + up(16 * key_items);
  L.w_starts_off = L.w_cum_off + up(8 * (key_items + 1));
  L.w_part_off = L.w_starts_off + up(16 * (kTreeTcGrid + 1));
  L.bytes = L.w_part_off + up(8 * (int64_t)kTreeTcGrid * kWeightKeys);
  return L;
}

cudaError_t launch_window_plan(const TreeParams& p, cudaStream_t stream) {
  // checks beside the planner: a warp per 256 table entries or 1024 tokens, at most 64 blocks
  const int64_t chunks = (int64_t)p.m.num_seqs * ((p.m.max_blocks + 255) / 256 +
                                                  (p.m.num_tokens + kCheckTokens - 1) / kCheckTokens);
  static_assert(kSmallBlocks == 64, "a word for each of the blocks");
  const int blocks = (int)std::min<int64_t>((chunks + 31) / 32, 64);
  return launch_pdl(k_window_plan, dim3((p.w.grid > 0 ? 2 : 1) + blocks), dim3(kPlanThreads), 0, stream, p);
}

cudaError_t launch_window_check(const TreeParams& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.m.num_seqs * ((p.m.max_blocks + 255) / 256 +
                                                 (p.m.num_tokens + kCheckTokens - 1) / kCheckTokens);
  const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>((units + 7) / 8, 64));
  return launch_pdl(k_window_check, dim3(blocks), dim3(256), 0, stream, p);
}

cudaError_t launch_window_generic(const TreeParams& p, pa_dtype kv, cudaStream_t stream) {
  return generic_types<true>(p, kv, stream);
}

}  // namespace pa
