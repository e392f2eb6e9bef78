// k_tree.cuh -- what the tree attention kernels share: how the work items of a batch are
// numbered and walked, which keys a node sees, and how a finished row is normalised.
#pragma once

#include <climits>

#include "pa_internal.cuh"

namespace pa {

// Items of one kv head of a sequence (plan record q: first token, nodes, seq_len, first key).
struct TreeGeometry {
  int rows, items, tiles;
  int full_w, rest_w;
  __device__ __forceinline__ TreeGeometry(const TreeParams& p, int4 q) {
    rows = q.y * p.m.group;
    items = (rows + p.rows_per_item - 1) / p.rows_per_item;
    tiles = (q.z - q.w + p.key_tile - 1) / p.key_tile;
    full_w = tree_weight(p, p.rows_per_item);
    rest_w = items ? tree_weight(p, rows - (items - 1) * p.rows_per_item) : 0;
  }
  __device__ __forceinline__ int rows_of(const TreeParams& p, int item) const {
    return min(p.rows_per_item, rows - item * p.rows_per_item);
  }
  // weight of one key tile of the first `i` items (i == items: of all of them)
  __device__ __forceinline__ int64_t weight_before(int i) const {
    return i < items ? (int64_t)i * full_w : (int64_t)(items - 1) * full_w + rest_w;
  }
};

// One CTA's share of one item: key tiles [t0, t1) of `tiles`.
struct TreeSegment {
  int s, kvh, row0, rows;  // rows row0 .. of the sequence's (node, head of the group) rows
  int qs, nodes, n, kv0;
  int t0, t1, tiles;
  int slot;  // partial state it writes, or -1: the item is whole and goes to the output
};

struct TreeWalk {
  int s, item, tile;        // where the next segment begins
  int es, eitem, etile;     // where the share ends
  int first_slot;
  bool first;
  __device__ __forceinline__ TreeWalk(const TreeParams& p, int cta) {
    const int4 a = p.starts[cta], e = p.starts[cta + 1];
    s = a.x;
    item = a.y;
    tile = a.z;
    es = e.x;
    eitem = e.y;
    etile = e.z;
    first_slot = 2 * cta;
    first = true;
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreeSegment& g) {
    if (s >= p.m.num_seqs) return false;
    int4 q = p.seqs[s];
    while (q.y == 0) {  // sequences without nodes
      if (++s >= p.m.num_seqs) return false;
      q = p.seqs[s];
    }
    const TreeGeometry ge(p, q);
    const bool last = s == es && item == eitem;
    const int t1 = last ? etile : ge.tiles;
    if (s > es || (s == es && item > eitem) || t1 <= tile) return false;
    g.s = s;
    g.kvh = item / ge.items;
    const int it = item % ge.items;
    g.row0 = it * p.rows_per_item;
    g.rows = ge.rows_of(p, it);
    g.qs = q.x;
    g.nodes = q.y;
    g.n = q.z;
    g.kv0 = q.w;
    g.t0 = tile;
    g.t1 = t1;
    g.tiles = ge.tiles;
    g.slot = tile > 0 || t1 < ge.tiles ? first_slot + (first ? 0 : 1) : -1;
    first = false;
    tile = 0;
    if (last) {
      s = p.m.num_seqs;  // the share is used up
    } else if (++item == ge.items * p.m.num_kv_heads) {
      item = 0;
      ++s;
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

// The factor that normalises a row's output, given its running max (log2 units) and exp-sum;
// a sink (a virtual position with score sinks[h] and value zero) joins the sum, and the row's
// lse is written when asked for.  A row that sees nothing gets 0 and lse -inf.
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
    m.lse[(int64_t)h * m.num_tokens + tok] = l > 0.f ? (mx + log2f(l)) * kLn2 : -INFINITY;
  return l > 0.f ? a * head_scale(m.v_scales, kvh, m.v_scale) / l : 0.f;
}

}  // namespace pa
