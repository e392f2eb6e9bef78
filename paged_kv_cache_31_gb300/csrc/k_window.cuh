// k_window.cuh -- what the kernels of the attention behind a window with first tokens share: which blocks
// of its table a sequence reads, and the checks of a batch's metadata.
#pragma once

#include "pa_internal.cuh"

namespace pa {

constexpr int kCheckTokens = 1024;  // of one sequence, checked by a warp

// Blocks of a sequence's table that its tokens read: [0, front) and [front + gap, its end).
struct Keys {
  int front, gap;
};
__device__ __forceinline__ Keys keys_from(const TreeParams& p, int lowest) {
  const VarlenMeta& m = p.m;
  const int lo = m.window > 0 ? max(max(lowest, 0) - m.window + 1, 0) / m.block_size : 0;
  return Keys{p.front, max(lo - p.front, 0)};
}

// First token, tokens and length of sequence s; false (and no tokens) when they cannot be used.
__device__ __forceinline__ bool sequence(const TreeParams& p, int s, int& qs, int& q, int& n) {
  const VarlenMeta& m = p.m;
  qs = m.query_start_loc[s];
  const int qe = m.query_start_loc[s + 1];
  q = n = 0;
  bool ok = qs >= 0 && qe >= qs && (int64_t)qe <= m.num_tokens && (s > 0 || qs == 0) &&
            (s < m.num_seqs - 1 || (int64_t)qe == m.num_tokens);
  if (qs >= 0 && qe > qs && (int64_t)qe <= m.num_tokens) {
    q = qe - qs;
    n = m.seq_lens[s];
    if (n < 1 || ((int64_t)n + m.block_size - 1) / m.block_size > m.max_blocks ||
        (p.key_weights && (int64_t)n > p.weights_len)) {
      ok = false;
      q = 0;
    }
  }
  return ok;
}

// Warp `me` of `warps`: the sequences' table entries that are read, and their positions; true when one
// is bad.  (Sequences that cannot be used are found by sequence().)
__device__ __forceinline__ bool bad_reads(const TreeParams& p, int me, int warps) {
  const VarlenMeta& m = p.m;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  const int per = (m.max_blocks + 255) / 256;  // chunks of a table row
  const int64_t chunks = (int64_t)m.num_seqs * per;
  for (int64_t c = me; c < chunks; c += warps) {
    const int s = (int)(c / per), e0 = (int)(c % per) * 256;
    const int qs = m.query_start_loc[s], n = m.seq_lens[s];
    if (m.query_start_loc[s + 1] <= qs || n < 1 || qs < 0 || qs >= m.num_tokens) continue;
    const int64_t need = ((int64_t)n + m.block_size - 1) / m.block_size;
    const int lim = (int)min(need, (int64_t)m.max_blocks);
    if (e0 >= lim) continue;
    const Keys k = keys_from(p, m.window > 0 ? m.positions[qs] : 0);
    const int32_t* row = m.block_tables + (int64_t)s * m.max_blocks;
    int id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int e = e0 + lane + 32 * u;
      id[u] = e < lim && (e < k.front || e >= k.front + k.gap) ? row[e] : 0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) bad |= id[u] < 0 || (int64_t)id[u] >= m.num_blocks;
  }
  const int parts = (int)((m.num_tokens + kCheckTokens - 1) / kCheckTokens);
  const int64_t units = (int64_t)m.num_seqs * parts;
  for (int64_t c = me; c < units; c += warps) {
    const int s = (int)(c / parts);
    const int64_t t0 = (int64_t)m.query_start_loc[s] + c % parts * kCheckTokens;
    const int64_t end = min(min((int64_t)m.query_start_loc[s + 1], t0 + kCheckTokens), m.num_tokens);
    if (t0 < 0 || t0 >= end) continue;
    const int n = m.seq_lens[s];
    const bool more = t0 + kCheckTokens < m.query_start_loc[s + 1] && t0 + kCheckTokens < m.num_tokens;
    for (int64_t t = t0 + lane; t < end; t += 32) {
      const int pos = m.positions[t];
      const int after = t + 1 < end || more ? m.positions[t + 1] : pos;
      bad |= pos < 0 || pos >= n || after < pos;
    }
  }
  return bad;
}

// Per-head scales (each array may be missing).
__device__ __forceinline__ bool bad_scales(const TreeParams& p, int tid, int threads) {
  bool bad = false;
  for (int g = tid; g < p.m.num_kv_heads; g += threads) {
    const float a = p.m.k_scales ? p.m.k_scales[g] : 1.f, b = p.m.v_scales ? p.m.v_scales[g] : 1.f;
    bad |= !(a > 0.f && a <= 3.402823466e38f) || !(b > 0.f && b <= 3.402823466e38f);
  }
  return bad;
}

}  // namespace pa
