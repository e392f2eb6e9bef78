// pa_api_bounded.cu -- the C ABI's calls for caches of bounded size: attention behind a window with
// first tokens, the attention weights that keys receive, and the eviction of keys.  Argument checks,
// path selection and launches only.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pa_internal.cuh"

using namespace pa;

namespace {

// Rows of one row tile of the tensor-core kernel: whole tokens, at most 128 rows.
int32_t tile_rows(int32_t group) { return 128 / group * group; }

bool tc_sizes(int32_t group, int32_t head_dim) {
  return group <= 128 && (head_dim == 64 || head_dim == 128);
}

// Whether a batch is one of decoding tokens, or of a few tokens of one sequence (k_window_decode.cu).
bool decodes(int32_t num_seqs, int64_t num_tokens, int32_t num_kv_heads, int32_t group) {
  return (num_tokens <= num_seqs || (num_seqs == 1 && num_tokens * group <= 64)) &&
         (int64_t)num_seqs * num_kv_heads < (1 << 24);
}

// Scores of a (sequence, kv head) that the workspace has room for: all keys of a token's heads, up to
// 256 MB for the batch or, where that is more, 2048 (8 KB: 512 keys of 4 heads) for each.
int64_t score_room(int32_t num_seqs, int32_t num_kv_heads, int32_t group, int64_t keys) {
  const int64_t all = std::min(group, 16) * ((keys + 511) / 512 * 512);
  return std::min(all, std::max<int64_t>((1 << 26) / ((int64_t)num_seqs * num_kv_heads), 2048)) / 512 * 512;
}

size_t workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                      int32_t head_dim, int32_t max_blocks, int32_t block_size, bool weights) {
  if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      num_heads % num_kv_heads != 0 || head_dim <= 0 || max_blocks < 0 || block_size <= 0)
    return 0;
  const int64_t keys = (int64_t)max_blocks * block_size;
  int64_t bytes = window_layout(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, keys,
                                kTreeGenericRows, kTreeGenericKeys, kTreeGenericGrid, weights)
                      .bytes;
  const int32_t group = num_heads / num_kv_heads;
  // the tensor-core kernel may run, with items of one row tile or of two (one: more items, more CTAs)
  for (int tiles = 1; tiles <= 2 && tc_sizes(group, head_dim); ++tiles)
    bytes = std::max(bytes, window_layout(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, keys,
                                          tiles * tile_rows(group), kTreeTcKeys, kTreeTcGrid, weights)
                                .bytes);
  if (weights && num_seqs > 0 && decodes(num_seqs, num_tokens, num_kv_heads, group))
    bytes = std::max(bytes, 4 * (int64_t)num_seqs * num_kv_heads *
                                score_room(num_seqs, num_kv_heads, group, keys));
  return (size_t)bytes;
}

// How a batch of decoding tokens goes: CTAs of a cluster for each (sequence, kv head), their shape, and
// whether the longest sequences come first.  keys: the most that a token can see (of the table's width
// and the window; the lengths are on the device).
struct DecodeForm {
  int32_t cluster, shape;  // 1: narrow CTAs, 2: broad ones
  bool ordered;
};
// More CTAs to a unit read its keys sooner, but each costs some 4 us of latencies (metadata, first keys,
// joins) in which it reads nothing.  Measured (us in a graph, bf16, 8 kv heads of 4 heads, lengths up to
// the given one; CTAs to a unit): 1 sequence of 2048 1: 27.8, 4: 12.4, 8: 9.4; of 16384 8: 28.8, 16: 20.7;
// 4 of 4096 2: 29.4, 4: 18.0, 8: 13.6; 8 of 1024 1: 16.6, 4: 10.4, 8: 16.0; 16 of 8192 1: 95, 2: 76, 4: 76,
// 8: 85; 24 of 4096 1: 58, 2: 54, 4: 63; 48 of 16384 1: 319, 2: 288, 4: 312; 64 of 4096 1: 105, 2: 126.
// Clusters of 16 only over e4m3 pools and long contexts (1 sequence of 65536 8: 53.5, 16: 45.5; of 2048
// 8.4 / 9.7), broad CTAs (bf16, twice the warps) where there are a few units: 1 of 16384 28.8 -> 20.3, but
// 2 of 8192 20.2 / 25.3, as clusters of 8 broad CTAs find fewer places.
// Narrow CTAs (half the warps, four to an SM) where units are short or many: 64 sequences of 256 14.0
// against 17.7, 128 of 1024 65.8 / 76.2, e4m3 64 of 1024 19.8 / 24.4; but 64 of 4096 129 / 105.
// Longest first where not all units are resident: 64 of 4096, ragged, 118 -> 98.
DecodeForm decode_form(int64_t units, int32_t num_seqs, int64_t keys, int64_t key_bytes, bool fp8, int32_t sms) {
  DecodeForm f{1, 0, false};
  while (f.cluster < 16) {
    const int64_t ctas = units * 2 * f.cluster, each = keys / (2 * f.cluster);
    const int64_t least = ctas <= sms ? 64 : ctas <= 2 * sms ? 256 : ctas <= 6 * sms ? 2048 : INT64_MAX;
    if (each < least || (f.cluster == 8 && (!fp8 || ctas > sms || keys < 16384))) break;
    f.cluster *= 2;
  }
  if (units > 2 * sms && (units >= 6 * sms || keys * key_bytes <= 384 * 1024)) f.shape = 1;
  if (!fp8 && f.cluster == 8 && units * 16 <= sms) f.shape = 2;
  f.ordered = f.cluster == 1 && units > (f.shape == 1 ? 4 : 2) * sms && num_seqs <= 256;
  return f;
}

struct Call {
  const void *q, *k_blocks, *v_blocks;
  void* out;
  const int32_t *query_start_loc, *seq_lens, *positions, *block_tables;
  int32_t num_seqs;
  int64_t num_tokens;
  int32_t num_heads, num_kv_heads, head_dim, block_size;
  int64_t num_blocks;
  int32_t max_blocks;
  pa_dtype q_dtype, kv_dtype;
  float scale;
  int32_t window, first;
  const float* sinks;
  float* lse;
  float k_scale, v_scale;
  const float *k_scales, *v_scales;
  bool weighs;
  float* key_weights;
  int64_t weights_len;
  int32_t observed;
  void* workspace;
  size_t workspace_bytes;
  cudaStream_t stream;
};

pa_status attend(const Call& c) {
  bool empty = false;  // no token: nothing to do, whatever the sequences
  const int32_t check_seqs = c.num_tokens == 0 && c.num_seqs > 0 ? 0 : c.num_seqs;
  const pa_status chk = varlen_check(c.q, c.k_blocks, c.v_blocks, c.out, c.query_start_loc, c.seq_lens,
                                     c.positions, c.block_tables, check_seqs, c.num_tokens, c.num_heads,
                                     c.num_kv_heads, c.head_dim, c.block_size, c.num_blocks,
                                     c.max_blocks, c.q_dtype, c.kv_dtype, c.k_scale, c.v_scale, 0u,
                                     &empty);
  if (chk != PA_OK) return chk;
  if ((c.k_scales && c.k_scale != 1.f) || (c.v_scales && c.v_scale != 1.f) || c.window < 0 ||
      c.first < 0 || c.observed < 0 || c.weights_len < 0)
    return PA_EINVAL;
  if (empty) return PA_OK;
  if (c.num_seqs == 0 || !std::isfinite(c.scale) || (c.weighs && !c.key_weights)) return PA_EINVAL;
  const int32_t group = c.num_heads / c.num_kv_heads;
  const int64_t max_keys = (int64_t)c.max_blocks * c.block_size;
  // token * group rows of one sequence, and positions, are counted in 32 bits
  if (c.num_tokens * group > INT32_MAX / 2 || max_keys > INT32_MAX - 1024) return PA_EUNSUPPORTED;
  if (!c.workspace || !aligned(c.workspace, 256)) return PA_EINVAL;
  if (c.workspace_bytes < workspace_size(c.num_seqs, c.num_tokens, c.num_heads, c.num_kv_heads,
                                         c.head_dim, c.max_blocks, c.block_size, c.weighs))
    return PA_EINVAL;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;

  TreeParams p;
  std::memset(&p, 0, sizeof p);
  p.q = c.q;
  p.k_blocks = c.k_blocks;
  p.v_blocks = c.v_blocks;
  p.out = c.out;
  VarlenMeta& m = p.m;
  m.query_start_loc = c.query_start_loc;
  m.seq_lens = c.seq_lens;
  m.positions = c.positions;
  m.block_tables = c.block_tables;
  m.num_seqs = c.num_seqs;
  m.num_tokens = c.num_tokens;
  m.num_heads = c.num_heads;
  m.num_kv_heads = c.num_kv_heads;
  m.group = group;
  m.head_dim = c.head_dim;
  m.block_size = c.block_size;
  m.num_blocks = c.num_blocks;
  m.max_blocks = c.max_blocks;
  m.window = c.window;
  m.sinks = c.sinks;
  m.lse = c.lse;
  m.v_scale = c.v_scale;
  m.k_scales = c.k_scales;
  m.v_scales = c.v_scales;
  p.first = c.window > 0 ? (int32_t)std::min<int64_t>(c.first, max_keys) : 0;
  p.front = (int32_t)(((int64_t)p.first + c.block_size - 1) / c.block_size);
  p.scale = c.scale * c.k_scale;
  p.status = d->status;
  p.q_bf16 = c.q_dtype == PA_BF16;
  p.key_weights = c.key_weights;
  p.weights_len = c.weights_len;
  p.observed = c.observed;
  const bool fp8 = c.kv_dtype == PA_FP8_E4M3;
  // the tensor-core kernel: its types and sizes, tensors aligned for TMA, and a positive scale (its
  // row maxima are taken before the scale)
  const bool tc = c.q_dtype == PA_BF16 && c.block_size == 16 && tc_sizes(group, c.head_dim) &&
                  (fp8 ? c.head_dim == 128 : c.kv_dtype == PA_BF16) && aligned(c.q, 16) &&
                  aligned(c.out, 16) && aligned(c.k_blocks, 16) && aligned(c.v_blocks, 16) &&
                  p.scale > 0.f && c.num_blocks > 0 && tc_enabled();
  // a batch of decoding tokens, or a few tokens of one sequence
  const int64_t units = (int64_t)c.num_seqs * c.num_kv_heads;
  if (tc && decodes(c.num_seqs, c.num_tokens, c.num_kv_heads, group)) {
    const int64_t keys = c.window > 0 ? std::min<int64_t>((int64_t)c.window + p.first, max_keys) : max_keys;
    const DecodeForm f = decode_form(units, c.num_seqs, keys, 2 * c.head_dim * esize(c.kv_dtype), fp8, d->sms);
    p.cluster = f.cluster;
    p.shape = f.shape;
    p.ordered = f.ordered;
    p.w.part = static_cast<float*>(c.workspace);
    p.w.room = (int32_t)(score_room(c.num_seqs, c.num_kv_heads, group, max_keys) / p.cluster);
    CUtensorMap tk, tv;
    const bool ok =
        fp8 ? pool_map_fp8(&tk, c.k_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim, true) &&
                  pool_map_fp8(&tv, c.v_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim, true)
            : pool_map_rows(&tk, c.k_blocks, c.num_blocks, c.num_kv_heads, c.head_dim) &&
                  pool_map_rows(&tv, c.v_blocks, c.num_blocks, c.num_kv_heads, c.head_dim);
    if (!ok) return PA_ECUDA;
    uint64_t limit;
    uint32_t stall;
    stall_hook(limit, stall);
    if (launch_window_check(p, c.stream) != cudaSuccess) return PA_ECUDA;
    return from_cuda(launch_window_decode(tk, tv, p, fp8, limit, stall, c.stream));
  }
  WindowLayout L;
  if (tc) {
    p.tile_rows = tile_rows(group);
    p.tile_tokens = p.tile_rows / group;
    p.key_tile = kTreeTcKeys;
    // items of one row tile when no sequence can have more rows, else of two
    p.rows_per_item = c.num_tokens * group > p.tile_rows ? 2 * p.tile_rows : p.tile_rows;
    L = window_layout(c.num_seqs, c.num_tokens, c.num_heads, c.num_kv_heads, c.head_dim, max_keys,
                      p.rows_per_item, p.key_tile, kTreeTcGrid, c.weighs);
    L.tree.grid = std::min(L.tree.grid, d->sms);
  } else {
    p.tile_rows = p.rows_per_item = kTreeGenericRows;
    p.key_tile = kTreeGenericKeys;
    L = window_layout(c.num_seqs, c.num_tokens, c.num_heads, c.num_kv_heads, c.head_dim, max_keys,
                      p.rows_per_item, p.key_tile, kTreeGenericGrid, c.weighs);
  }
  if ((uint64_t)L.bytes > c.workspace_bytes) return PA_EINVAL;  // (workspace_size() covers every layout)
  p.grid = L.tree.grid;
  uint8_t* ws = static_cast<uint8_t*>(c.workspace);
  p.seqs = reinterpret_cast<int4*>(ws);
  p.cum = reinterpret_cast<int64_t*>(ws + L.tree.cum_off);
  p.starts = reinterpret_cast<int4*>(ws + L.tree.starts_off);
  p.part_ml = reinterpret_cast<float2*>(ws + L.tree.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + L.tree.o_off);
  p.item_keys = reinterpret_cast<int4*>(ws + L.items_off);
  p.item_cum = reinterpret_cast<int64_t*>(ws + L.item_cum_off);
  if (c.weighs && !m.lse) m.lse = reinterpret_cast<float*>(ws + L.lse_off);
  if (c.weighs && tc) {
    p.w.seqs = reinterpret_cast<int4*>(ws + L.w_seqs_off);
    p.w.items = reinterpret_cast<int4*>(ws + L.w_items_off);
    p.w.cum = reinterpret_cast<int64_t*>(ws + L.w_cum_off);
    p.w.starts = reinterpret_cast<int4*>(ws + L.w_starts_off);
    p.w.part = reinterpret_cast<float*>(ws + L.w_part_off);
    p.w.grid = std::min(kTreeTcGrid, d->sms);
  }
  CUtensorMap tq, tk, tv;
  if (tc) {
    const bool ok =
        query_map(&tq, c.q, c.num_tokens, c.num_heads, c.head_dim, group, p.tile_tokens) &&
        (fp8 ? pool_map_fp8(&tk, c.k_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim, true) &&
                   pool_map_fp8(&tv, c.v_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim, true)
             : pool_map_rows(&tk, c.k_blocks, c.num_blocks, c.num_kv_heads, c.head_dim) &&
                   pool_map_rows(&tv, c.v_blocks, c.num_blocks, c.num_kv_heads, c.head_dim));
    if (!ok) return PA_ECUDA;
  }
  // many items of prompt chunks: the prefill kernel takes them (its pairs of CTAs do a fifth to a half
  // more a second, but an item's keys are not cut, so there have to be more items than pairs)
  const int64_t key_bytes = 2 * (int64_t)c.head_dim * esize(c.kv_dtype);
  const bool prefill = tc && c.head_dim == 128 && 128 % group == 0 &&
                       c.num_tokens * group / 256 * c.num_kv_heads >= 2 * d->sms && units < (1 << 24);
  if (prefill) {
    p.tc.plan = reinterpret_cast<int32_t*>(ws + L.tc_off);
    const int64_t items = (c.num_tokens * group + 255) / 256 + c.num_seqs;
    p.tc.items_off = kPlanHeaderWords;
    p.tc.redo_off = p.tc.items_off + 4 * items;
    p.tc.redo_list_off = p.tc.redo_off + items;
    p.tc.small_off = fp8 ? 0 : p.tc.redo_list_off + items;
    p.tc.num_sms = d->sms;
    p.tc.pairs = d->sms / 2;
    p.tc.decode_bytes_per_key = (float)(key_bytes * c.num_kv_heads);
  }
  if (launch_window_plan(p, c.stream) != cudaSuccess) return PA_ECUDA;
  uint64_t limit;
  uint32_t stall;
  stall_hook(limit, stall);
  if (prefill) {
    CUtensorMap pk, pv;
    const bool ok = fp8 ? pool_map_fp8(&pk, c.k_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim) &&
                              pool_map_fp8_half(&pv, c.v_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim)
                        : pool_map(&pk, c.k_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim) &&
                              pool_map(&pv, c.v_blocks, c.num_blocks, 16, c.num_kv_heads, c.head_dim);
    if (!ok) return PA_ECUDA;
    TcParams tp;
    std::memset(&tp, 0, sizeof tp);
    tp.out = c.out;
    tp.m = m;
    tp.plan = p.tc.plan;
    tp.tc_off = p.tc.items_off;
    tp.status = d->status;
    tp.scale_log2 = p.scale * kLog2e;
    tp.wait_limit_ns = limit;
    tp.debug_stall = stall;
    tp.win = 1;
    tp.kv_fp8 = fp8;
    tp.first = p.first;
    tp.redo_flags = p.tc.plan + p.tc.redo_off;
    tp.redo_list = p.tc.plan + p.tc.redo_list_off;
    tp.redo_count = p.tc.plan + 3;
    if (launch_tc_prefill(tq, pk, pv, tp, 2 * p.tc.pairs, c.stream) != cudaSuccess) return PA_ECUDA;
    if (c.num_seqs > 1) {  // (one sequence has more rows than a decoding one)
      TreeParams dp = p;  // the decoding sequences
      dp.after_tc = 1;
      dp.w.room = 0;
      const int64_t keys = c.window > 0 ? std::min<int64_t>((int64_t)c.window + p.first, max_keys) : max_keys;
      const DecodeForm f = decode_form(units, c.num_seqs, keys, key_bytes, fp8, d->sms);
      dp.cluster = f.cluster;
      dp.shape = f.shape;
      dp.ordered = f.ordered;
      if (launch_window_decode(tk, tv, dp, fp8, limit, stall, c.stream) != cudaSuccess) return PA_ECUDA;
    }
  }
  if (tc && !(prefill && fp8)) {  // (f16 holds every e4m3 value: no items to do again)
    if (launch_window_tc(tq, tk, tv, p, fp8, limit, stall, c.stream) != cudaSuccess) return PA_ECUDA;
  } else if (!tc && launch_window_generic(p, c.kv_dtype, c.stream) != cudaSuccess) {
    return PA_ECUDA;
  }
  if (!prefill && launch_tree_merge(p, c.stream) != cudaSuccess) return PA_ECUDA;
  if (!c.weighs) return PA_OK;
  if (p.w.grid > 0) return from_cuda(launch_weights_tc(tq, tk, p, fp8, limit, stall, c.stream));
  return from_cuda(launch_key_weights_generic(p, c.kv_dtype, c.stream));
}

}  // namespace

extern "C" {

size_t pa_window_attention_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                          int32_t num_kv_heads, int32_t head_dim,
                                          int32_t max_blocks_per_seq, int32_t block_size) {
  return workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                        block_size, false);
}

pa_status pa_window_attention(const void* q, const void* k_blocks, const void* v_blocks, void* out,
                              const int32_t* query_start_loc, const int32_t* seq_lens,
                              const int32_t* positions, const int32_t* block_tables, int32_t num_seqs,
                              int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int64_t num_blocks,
                              int32_t max_blocks_per_seq, pa_dtype q_dtype, pa_dtype kv_dtype,
                              float scale, int32_t sliding_window, int32_t first_tokens,
                              const float* sinks, float* lse, float k_scale, float v_scale,
                              const float* k_scales, const float* v_scales, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  return attend(Call{q, k_blocks, v_blocks, out, query_start_loc, seq_lens, positions, block_tables,
                     num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                     max_blocks_per_seq, q_dtype, kv_dtype, scale, sliding_window, first_tokens, sinks,
                     lse, k_scale, v_scale, k_scales, v_scales, false, nullptr, 0, 0, workspace,
                     workspace_bytes, stream});
}

size_t pa_attention_key_weights_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                               int32_t num_kv_heads, int32_t head_dim,
                                               int32_t max_blocks_per_seq, int32_t block_size) {
  return workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                        block_size, true);
}

pa_status pa_attention_key_weights(const void* q, const void* k_blocks, const void* v_blocks, void* out,
                                   const int32_t* query_start_loc, const int32_t* seq_lens,
                                   const int32_t* positions, const int32_t* block_tables,
                                   float* key_weights, int64_t weights_len, int32_t observed_tokens,
                                   int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   int64_t num_blocks, int32_t max_blocks_per_seq, pa_dtype q_dtype,
                                   pa_dtype kv_dtype, float scale, int32_t sliding_window,
                                   int32_t first_tokens, const float* sinks, float* lse, float k_scale,
                                   float v_scale, const float* k_scales, const float* v_scales,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return attend(Call{q, k_blocks, v_blocks, out, query_start_loc, seq_lens, positions, block_tables,
                     num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
                     max_blocks_per_seq, q_dtype, kv_dtype, scale, sliding_window, first_tokens, sinks,
                     lse, k_scale, v_scale, k_scales, v_scales, true, key_weights, weights_len,
                     observed_tokens, workspace, workspace_bytes, stream});
}

size_t pa_evict_keys_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t max_blocks_per_seq,
                                    int32_t block_size) {
  if (num_seqs < 0 || num_kv_heads <= 0 || max_blocks_per_seq < 0 || block_size <= 0) return 0;
  return (size_t)evict_workspace(num_seqs, num_kv_heads, (int64_t)max_blocks_per_seq * block_size);
}

pa_status pa_evict_keys(void* k_blocks, void* v_blocks, const int32_t* block_tables,
                        const int32_t* seq_lens, const int32_t* new_lens, float* key_weights,
                        int64_t weights_len, int32_t keep_first, int32_t keep_recent, int32_t num_seqs,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks,
                        int32_t max_blocks_per_seq, pa_dtype kv_dtype, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0) return PA_ESHAPE;
  if (!pool_dtype_ok(kv_dtype)) return PA_EUNSUPPORTED;
  if (num_seqs < 0 || num_blocks < 0 || max_blocks_per_seq < 0 || keep_first < 0 || keep_recent < 0 ||
      weights_len < 0)
    return PA_EINVAL;
  const int64_t max_keys = (int64_t)max_blocks_per_seq * block_size;
  const int64_t most = key_weights ? std::min(max_keys, weights_len) : max_keys;
  if (num_blocks * block_size > INT32_MAX) return PA_EUNSUPPORTED;  // slots are int32
  if (num_seqs > 65535 || num_kv_heads > 65535 || max_keys > INT32_MAX - 1024 || most > kEvictMostKeys ||
      (int64_t)head_dim * esize(kv_dtype) > (1 << 20))
    return PA_EUNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  // (arrays without an element have no address: tables of no column, pools of no block)
  if ((num_blocks > 0 && (!k_blocks || !v_blocks)) || (max_blocks_per_seq > 0 && !block_tables) || !seq_lens ||
      !new_lens)
    return PA_EINVAL;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < pa_evict_keys_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq, block_size))
    return PA_EINVAL;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;
  EvictParams p{};
  p.k_blocks = k_blocks;
  p.v_blocks = v_blocks;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.key_weights = key_weights;
  p.weights_len = weights_len;
  p.num_seqs = num_seqs;
  p.keep_first = keep_first;
  p.keep_recent = keep_recent;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.block_shift = (block_size & (block_size - 1)) == 0 ? __builtin_ctz(block_size) : -1;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.row_bytes = (int64_t)head_dim * esize(kv_dtype);
  p.verdict = static_cast<int32_t*>(workspace);
  p.moves = p.verdict + kEvictVerdict / 4;
  p.moves_len = most;
  p.status = d->status;
  return from_cuda(launch_evict(p, d->sms, stream));
}

}  // extern "C"
