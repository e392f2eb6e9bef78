// k_tree.cuh -- what the tree attention kernels share: how the work items of a batch are
// numbered and walked, which keys a node sees, and how a finished row is normalised.
#pragma once

#include <climits>

#include "pa_internal.cuh"

namespace pa {

// Exclusive prefix sum over a block of 1024 threads; *total receives the sum.
__device__ __forceinline__ int64_t block_sum_scan(int64_t v, int64_t* s_warp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  const int64_t before = warp ? s_warp[warp - 1] : 0;
  *total = s_warp[31];
  __syncthreads();
  return before + x - v;
}

__device__ __forceinline__ int64_t item_weight(const TreeParams& p, int tiles, int rows) {
  return (int64_t)tree_weight(p, rows) * tiles + kTreeItemWeight;
}

// One CTA's share of one item: key tiles [t0, t1).
struct TreeSegment {
  int s, kvh, row0, rows;  // rows row0 .. of the sequence's (node, head of the group) rows
  int item;                // row0 / rows_per_item
  int qs, nodes, n, kv0;
  int t0, t1;
  int slot;  // partial state it writes, or -1: the item is whole and goes to the output
  // window calls: keys are counted without the gap of `gap` blocks behind the first `front` blocks
  // (n and the key tiles, too; kv0 is 0)
  int front, gap;
};

// The segments of a CTA's share, in order.  (No division: this code is part of every role.)  WIN: the
// items have a record each, as their keys differ.
template <bool WIN>
struct TreeWalk {
  int4 at, end;  // (sequence, kv head, item, key tile) where the next segment begins, the share ends
  int slot;      // of a partial segment
  __device__ __forceinline__ TreeWalk(const TreeParams& p, int cta) {
    at = p.starts[cta];
    end = p.starts[cta + 1];
    slot = 2 * cta;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreeSegment& g) {
    if (at.x >= p.m.num_seqs) return false;
    int4 q = p.seqs[2 * at.x];
    while (q.y == 0) {  // sequences without nodes
      if (++at.x >= p.m.num_seqs) return false;
      q = p.seqs[2 * at.x];
    }
    const int4 w = p.seqs[2 * at.x + 1];  // (items, key tiles, rows), WIN: (items, first record, rows)
    const bool last = at.x == end.x && at.y == end.y && at.z == end.z;
    int tiles = w.y;
    if constexpr (WIN) {
      const int4 it = p.item_keys[w.y + at.z];
      tiles = it.z;
      g.front = p.front;
      g.gap = it.y;
    }
    const int t1 = last ? end.w : tiles;
    if (t1 <= at.w) return false;
    g.s = at.x;
    g.kvh = at.y;
    g.item = at.z;
    g.row0 = at.z * p.rows_per_item;
    g.rows = min(p.rows_per_item, w.z - g.row0);
    g.qs = q.x;
    g.nodes = q.y;
    g.n = WIN ? q.z - g.gap * p.m.block_size : q.z;
    g.kv0 = WIN ? 0 : q.w;
    g.t0 = at.w;
    g.t1 = t1;
    g.slot = at.w > 0 || t1 < tiles ? slot : -1;
    slot |= 1;  // a share's first segment has the even slot
    at.w = 0;
    if (last) {
      at.x = p.m.num_seqs;  // the share is used up
    } else if (++at.z == w.x) {
      at.z = 0;
      if (++at.y == p.m.num_kv_heads) {
        at.y = 0;
        ++at.x;
      }
    }
    return true;
  }
};

// Whether token tok (at logical position pos) of the segment's sequence sees key position key.
__device__ __forceinline__ bool tree_visible(const TreeParams& p, const TreeSegment& g, int tok,
                                             int pos, int key) {
  if (key >= g.n) return false;
  const int node = key - (g.n - g.nodes);
  if (node < 0) return p.m.window <= 0 || key > pos - p.m.window;
  const uint32_t word = (uint32_t)p.mask[(int64_t)tok * p.mask_words + (node >> 5)];
  if (!((word >> (node & 31)) & 1u)) return false;
  return p.m.window <= 0 || p.m.positions[g.qs + node] > pos - p.m.window;
}

// The same behind a window with first tokens; pos and key counted without the gap.
__device__ __forceinline__ bool window_visible(const TreeParams& p, int pos, int key) {
  return key <= pos && (p.m.window <= 0 || key > pos - p.m.window || key < p.first);
}

// The factor that normalises a row's output, given its running max (log2 units) and exp-sum;
// a sink (a virtual position with score sinks[h] and value zero) joins the sum, and the row's
// lse is written when asked for.  A row that sees nothing (its sum is 0) gets 0 and lse -inf; a
// sum that is NaN (a score was NaN or +inf) makes the factor and the lse NaN, so that a row
// spoiled by its inputs never looks like an empty one.
__device__ __forceinline__ float tree_finish(const TreeParams& p, int kvh, int h, int tok, float mx,
                                             float l, bool write_lse) {
  const VarlenMeta& m = p.m;
  float a = 1.f;
  const float sk = m.sinks ? m.sinks[h] * kLog2e : -INFINITY;
  if (sk > -INFINITY) {
    const float m2 = fmaxf(mx, sk);
    a = mx == -INFINITY ? 0.f : exp2f(mx - m2);
    l = l * a + exp2f(sk - m2);
    mx = m2;
  }
  if (m.lse && write_lse)
    m.lse[(int64_t)h * m.num_tokens + tok] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
  return l == 0.f ? 0.f : a * head_scale(m.v_scales, kvh, m.v_scale) / l;
}

}  // namespace pa
