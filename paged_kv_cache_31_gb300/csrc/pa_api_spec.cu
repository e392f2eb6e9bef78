// pa_api_spec.cu -- the C ABI's calls for speculative decoding over the paged cache: rotary
// caching, tree attention, moving accepted rows, and the page bookkeeping.  Argument checks,
// path selection and launches only.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "pa_internal.cuh"

using namespace pa;

extern "C" {

pa_status pa_rope_frequencies(int32_t rotary_dim, double base, const pa_rope_scaling* scaling,
                              double* inv_freq, float* attn_factor) {
  if (rotary_dim <= 0 || rotary_dim % 2 != 0) return PA_ESHAPE;
  if (!inv_freq || !(base > 1.0) || !std::isfinite(base)) return PA_EINVAL;
  const double pi2 = 6.283185307179586476925;
  const int32_t kind = scaling ? scaling->kind : PA_ROPE_PLAIN;
  if (kind < PA_ROPE_PLAIN || kind > PA_ROPE_BANDS) return PA_EUNSUPPORTED;
  const double s = scaling ? scaling->factor : 1.0;
  const double trained = scaling ? scaling->original_max_position : 0.0;
  if (kind != PA_ROPE_PLAIN && !(s >= 1.0 && std::isfinite(s))) return PA_EINVAL;
  if (kind >= PA_ROPE_YARN && !(trained > 0.0 && std::isfinite(trained))) return PA_EINVAL;
  double low = 0.0, high = 0.0;
  if (kind == PA_ROPE_NTK) {
    if (rotary_dim == 2) return PA_EUNSUPPORTED;  // one pair: no base to change
    base *= std::pow(s, (double)rotary_dim / (rotary_dim - 2));
  } else if (kind == PA_ROPE_YARN) {
    // the pair that turns n times over the trained length
    if (!(scaling->beta_fast > scaling->beta_slow && scaling->beta_slow > 0.0)) return PA_EINVAL;
    auto pair = [&](double n) { return rotary_dim * std::log(trained / (n * pi2)) / (2.0 * std::log(base)); };
    low = std::max(std::floor(pair(scaling->beta_fast)), 0.0);
    high = std::min(std::ceil(pair(scaling->beta_slow)), rotary_dim - 1.0);
  } else if (kind == PA_ROPE_BANDS) {
    if (!(scaling->high_freq_factor > scaling->low_freq_factor && scaling->low_freq_factor > 0.0))
      return PA_EINVAL;
  }
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 1.0;  // how much of the plain frequency stays
    if (kind == PA_ROPE_LINEAR) {
      keep = 0.0;
    } else if (kind == PA_ROPE_YARN) {
      keep = 1.0 - std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
    } else if (kind == PA_ROPE_BANDS) {
      const double turns = trained * f / pi2;  // over the trained length
      keep = (turns - scaling->low_freq_factor) /
             (scaling->high_freq_factor - scaling->low_freq_factor);
      keep = std::min(1.0, std::max(0.0, keep));
    }
    inv_freq[i] = f * keep + f / s * (1.0 - keep);
    if (kind == PA_ROPE_NTK || kind == PA_ROPE_PLAIN) inv_freq[i] = f;
  }
  if (attn_factor) *attn_factor = kind == PA_ROPE_YARN ? (float)(0.1 * std::log(s) + 1.0) : 1.f;
  return PA_OK;
}

pa_status pa_rope_and_cache(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                            const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            void* k_blocks, void* v_blocks, const int32_t* positions,
                            const int32_t* slot_mapping, const double* inv_freq,
                            int32_t rotary_dim, int32_t interleaved, float attn_factor,
                            int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, int64_t num_blocks,
                            pa_dtype src_dtype, pa_dtype kv_dtype, float k_scale, float v_scale,
                            const float* k_scales, const float* v_scales, cudaStream_t stream) {
  if (num_heads < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || rotary_dim <= 0 ||
      rotary_dim % 2 != 0 || rotary_dim > head_dim || (q && num_heads == 0))
    return PA_ESHAPE;
  if (!dtype_ok(src_dtype) || !pool_dtype_ok(kv_dtype)) return PA_EUNSUPPORTED;
  if (rotary_dim > 256 || (interleaved && head_dim % 2 != 0)) return PA_EUNSUPPORTED;
  if (!scale_ok(k_scale) || !scale_ok(v_scale) || !std::isfinite(attn_factor)) return PA_EINVAL;
  if ((k_scales && k_scale != 1.f) || (v_scales && v_scale != 1.f)) return PA_EINVAL;
  if (num_tokens < 0 || num_blocks < 0) return PA_EINVAL;
  if (num_tokens > INT32_MAX / 2) return PA_EUNSUPPORTED;
  if (num_blocks * block_size > INT32_MAX) return PA_EUNSUPPORTED;  // slots are int32
  const int64_t row = ((int64_t)num_heads + 2 * (int64_t)num_kv_heads) * head_dim;
  if (row > (1 << 24)) return PA_EUNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !k_blocks || !v_blocks || !positions || !slot_mapping || !inv_freq ||
      (q == nullptr) != (q_out == nullptr))
    return PA_EINVAL;
  const int64_t kv_row = (int64_t)num_kv_heads * head_dim;
  if (k_stride < kv_row || v_stride < kv_row) return PA_EINVAL;
  if (q && (q_stride < (int64_t)num_heads * head_dim || q_out_stride < (int64_t)num_heads * head_dim))
    return PA_EINVAL;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;
  if (launch_validate_scales(k_scales, v_scales, num_kv_heads, d->status, stream) != cudaSuccess)
    return PA_ECUDA;
  RopeParams p;
  std::memset(&p, 0, sizeof p);
  p.q = q;
  p.q_out = q_out;
  p.k = k;
  p.v = v;
  p.k_blocks = k_blocks;
  p.v_blocks = v_blocks;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slot_mapping;
  p.inv_freq = inv_freq;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved;
  p.attn_factor = attn_factor;
  p.num_tokens = num_tokens;
  p.num_slots = num_blocks * block_size;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.status = d->status;
  return from_cuda(launch_rope_and_cache(p, src_dtype, kv_dtype, d->sms, stream));
}

// Rows of one row tile of the tensor-core kernel: whole nodes, at most 128 rows.
static int32_t tree_tile_rows(int32_t group) { return 128 / group * group; }

// Layout of a call on the tensor-core kernel: items of one row tile when no sequence can have
// more rows (mask_words bounds a tree), else of two.
static TreeLayout tree_tc_layout(int32_t num_seqs, int64_t num_tokens, int32_t group,
                                 int32_t num_kv_heads, int32_t head_dim, int64_t max_keys,
                                 int32_t rows_per_item) {
  return tree_layout(num_seqs, num_tokens, group, num_kv_heads, head_dim, max_keys, rows_per_item,
                     kTreeTcKeys, kTreeTcGrid);
}

// CTAs of a cluster for each (sequence, kv head, item of `wide` row tiles) of a small call, which
// then is one launch; 0: the call takes the planned shares (three launches).  Both are right for
// any batch.  The largest clusters that are all resident at once (a second wave costs more than a
// larger cluster gives), no larger than the key tiles that a table can hold.  The slowest CTA's key
// tiles decide: they may be as many as a CTA's even share of the batch (taken as 0.7 of what the
// tables can hold: few sequences are as long as the longest) and the nine that the two other
// launches are worth.  The lengths are on the device, so the width of the table stands for them: one
// sequence of 8 kv heads leaves the clusters behind a table for about 12 000 positions, 8 at 5 000,
// 16 at 2 500, any call with more than kTreeSmallEntries entries, however short its sequences are (8
// nodes over 700 positions: 9.3 / 15.9 us in a graph).  Measured (us, clusters / shares, bf16, 32 rows a kv head): 8 units of 5 tiles
// 8.7 / 15.3, of 63 tiles 16.9 / 21.4; 128 units of 16 tiles 30.7 / 38.3, of 64 tiles 93 / 100.
static int32_t tree_cluster(int32_t num_seqs, int32_t num_kv_heads, int32_t items, int32_t wide,
                            int64_t max_keys, int32_t max_blocks, int32_t sms, bool fp8,
                            int32_t head_dim) {
  const int64_t units = (int64_t)num_seqs * num_kv_heads * items;
  const int64_t tiles = (max_keys + kTreeTcKeys - 1) / kTreeTcKeys;
  int device = 0;
  if (units > sms || (int64_t)num_seqs * max_blocks > kTreeSmallEntries ||
      cudaGetDevice(&device) != cudaSuccess)
    return 0;
  int32_t c = 8;
  while (c > 1 && (c / 2 >= tiles || units * c > sms ||
                   units > tree_clusters_resident(device, fp8, head_dim, c)))
    c /= 2;
  const int64_t most = (tiles + c - 1) / c * wide, share = units * wide * tiles / sms;
  return most <= share * 7 / 10 + kTreeSmallTiles ? c : 0;
}

// Types and sizes that the tensor-core kernel takes: bf16 q over bf16 or e4m3 pools of 16-position
// blocks, a group that fits a row tile.
static bool tree_tc_takes(int32_t group, int32_t head_dim, int32_t block_size, pa_dtype q_dtype,
                          pa_dtype kv_dtype) {
  return q_dtype == PA_BF16 && block_size == 16 && group <= 128 &&
         (kv_dtype == PA_FP8_E4M3 ? head_dim == 128
                                  : kv_dtype == PA_BF16 && (head_dim == 64 || head_dim == 128));
}

// How a call on the tensor-core kernel goes: clusters, of items of one row tile (more of them, on
// more SMs) or else of two, or (cluster 0) the planned shares.
struct TreeForm {
  int32_t row_tiles;       // of an item, at most
  int32_t items, cluster;  // items of a (sequence, kv head), at most; CTAs to each
};
static TreeForm tree_tc_form(int32_t num_seqs, int64_t num_tokens, int32_t mask_words, int32_t group,
                             int32_t num_kv_heads, int32_t head_dim, int32_t max_blocks, bool fp8,
                             int32_t sms) {
  const int64_t most = std::min<int64_t>(32 * (int64_t)mask_words, num_tokens) * group;
  const int32_t tile = tree_tile_rows(group), wide = most > tile ? 2 : 1;
  TreeForm f{0, 0, 0};
  while (f.row_tiles < wide && !f.cluster) {
    ++f.row_tiles;
    f.items = (int32_t)((most + f.row_tiles * tile - 1) / (f.row_tiles * tile));
    f.cluster = tree_cluster(num_seqs, num_kv_heads, f.items, f.row_tiles, (int64_t)max_blocks * 16,
                             max_blocks, sms, fp8, head_dim);
  }
  return f;
}

pa_status pa_tree_attention_form(int32_t num_seqs, int64_t num_tokens, int32_t mask_words,
                                 int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t max_blocks_per_seq, int32_t block_size, pa_dtype q_dtype,
                                 pa_dtype kv_dtype, int32_t* row_tiles, int32_t* cluster) {
  if (num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_heads % num_kv_heads != 0)
    return PA_ESHAPE;
  if (!dtype_ok(q_dtype) || !pool_dtype_ok(kv_dtype) || head_dim > 256 ||
      mask_words > kTreeMaxMaskWords || num_tokens > INT32_MAX / 2 ||
      num_tokens * (num_heads / num_kv_heads) > INT32_MAX / 2 ||
      (int64_t)max_blocks_per_seq * block_size > INT32_MAX - 1024)
    return PA_EUNSUPPORTED;
  if (num_seqs <= 0 || num_tokens <= 0 || mask_words <= 0 || max_blocks_per_seq < 0 || !row_tiles ||
      !cluster)
    return PA_EINVAL;
  *row_tiles = *cluster = 0;
  const int32_t group = num_heads / num_kv_heads;
  if (!tree_tc_takes(group, head_dim, block_size, q_dtype, kv_dtype) || !tc_enabled()) return PA_OK;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;
  const TreeForm f = tree_tc_form(num_seqs, num_tokens, mask_words, group, num_kv_heads, head_dim,
                                  max_blocks_per_seq, kv_dtype == PA_FP8_E4M3, d->sms);
  *row_tiles = f.row_tiles;
  *cluster = f.cluster;
  return PA_OK;
}

size_t pa_tree_attention_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t max_blocks_per_seq, int32_t block_size) {
  if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      num_heads % num_kv_heads != 0 || head_dim <= 0 || max_blocks_per_seq < 0 || block_size <= 0)
    return 0;
  const TreeLayout L = tree_layout(num_seqs, num_tokens, num_heads / num_kv_heads, num_kv_heads,
                                   head_dim, (int64_t)max_blocks_per_seq * block_size,
                                   kTreeGenericRows, kTreeGenericKeys, kTreeGenericGrid);
  int64_t bytes = L.bytes;
  const int32_t group = num_heads / num_kv_heads;
  if (group <= 128 && (head_dim == 64 || head_dim == 128))  // the tensor-core kernel may run
    for (int tiles = 1; tiles <= 2; ++tiles)
      bytes = std::max(bytes, tree_tc_layout(num_seqs, num_tokens, group, num_kv_heads, head_dim,
                                             (int64_t)max_blocks_per_seq * block_size,
                                             tiles * tree_tile_rows(group))
                                  .bytes);
  return (size_t)bytes;
}

pa_status pa_tree_attention(const void* q, const void* k_blocks, const void* v_blocks, void* out,
                            const int32_t* query_start_loc, const int32_t* seq_lens,
                            const int32_t* positions, const int32_t* tree_mask,
                            const int32_t* block_tables, int32_t num_seqs, int64_t num_tokens,
                            int32_t mask_words, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, int64_t num_blocks,
                            int32_t max_blocks_per_seq, pa_dtype q_dtype, pa_dtype kv_dtype,
                            float scale, int32_t sliding_window, const float* sinks, float* lse,
                            float k_scale, float v_scale, const float* k_scales,
                            const float* v_scales, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  bool empty = false;  // no token: nothing to do, whatever the sequences
  const int32_t check_seqs = num_tokens == 0 && num_seqs > 0 ? 0 : num_seqs;
  const pa_status chk = varlen_check(q, k_blocks, v_blocks, out, query_start_loc, seq_lens,
                                     positions, block_tables, check_seqs, num_tokens, num_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks,
                                     max_blocks_per_seq, q_dtype, kv_dtype, k_scale, v_scale, 0u,
                                     &empty);
  if (chk != PA_OK) return chk;
  if (mask_words < 0 || (k_scales && k_scale != 1.f) || (v_scales && v_scale != 1.f))
    return PA_EINVAL;
  if (mask_words > kTreeMaxMaskWords) return PA_EUNSUPPORTED;
  if (empty) return PA_OK;
  if (num_seqs == 0 || (num_tokens > 0 && (mask_words == 0 || !tree_mask))) return PA_EINVAL;
  if (!std::isfinite(scale)) return PA_EINVAL;
  // node * group rows of one sequence, and table entries, are counted in 32 bits
  if (num_tokens * (num_heads / num_kv_heads) > INT32_MAX / 2 ||
      (int64_t)max_blocks_per_seq * block_size > INT32_MAX - 1024)
    return PA_EUNSUPPORTED;
  if (!workspace || !aligned(workspace, 256)) return PA_EINVAL;
  const size_t need =
      pa_tree_attention_workspace_size(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                                       max_blocks_per_seq, block_size);
  if (workspace_bytes < need) return PA_EINVAL;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;

  TreeParams p;
  std::memset(&p, 0, sizeof p);
  p.q = q;
  p.k_blocks = k_blocks;
  p.v_blocks = v_blocks;
  p.out = out;
  VarlenMeta& m = p.m;
  m.query_start_loc = query_start_loc;
  m.seq_lens = seq_lens;
  m.positions = positions;
  m.block_tables = block_tables;
  m.num_seqs = num_seqs;
  m.num_tokens = num_tokens;
  m.num_heads = num_heads;
  m.num_kv_heads = num_kv_heads;
  m.group = num_heads / num_kv_heads;
  m.head_dim = head_dim;
  m.block_size = block_size;
  m.num_blocks = num_blocks;
  m.max_blocks = max_blocks_per_seq;
  m.window = sliding_window > 0 ? sliding_window : 0;
  m.sinks = sinks;
  m.lse = lse;
  m.v_scale = v_scale;
  m.k_scales = k_scales;
  m.v_scales = v_scales;
  p.mask = tree_mask;
  p.mask_words = mask_words;
  p.scale = scale * k_scale;
  p.status = d->status;
  p.q_bf16 = q_dtype == PA_BF16;
  const int64_t max_keys = (int64_t)max_blocks_per_seq * block_size;
  const bool fp8 = kv_dtype == PA_FP8_E4M3;
  // the tensor-core kernel: its types and sizes, tensors aligned for TMA, and a positive scale (its
  // row maxima are taken before the scale)
  const bool tc = tree_tc_takes(m.group, head_dim, block_size, q_dtype, kv_dtype) &&
                  aligned(q, 16) && aligned(out, 16) && aligned(k_blocks, 16) &&
                  aligned(v_blocks, 16) && p.scale > 0.f && num_blocks > 0 && tc_enabled();
  TreeLayout L;
  if (tc) {
    p.tile_rows = tree_tile_rows(m.group);
    p.tile_tokens = p.tile_rows / m.group;
    p.key_tile = kTreeTcKeys;
    const TreeForm f = tree_tc_form(num_seqs, num_tokens, mask_words, m.group, num_kv_heads, head_dim,
                                    max_blocks_per_seq, fp8, d->sms);
    p.rows_per_item = f.row_tiles * p.tile_rows;
    p.items = f.items;
    p.cluster = f.cluster;
    L = tree_tc_layout(num_seqs, num_tokens, m.group, num_kv_heads, head_dim, max_keys,
                       p.rows_per_item);
    L.grid = p.cluster ? num_seqs * num_kv_heads * p.items * p.cluster
                       : std::min(L.grid, d->sms);  // (no more than the workspace has room for)
  } else {
    p.tile_rows = p.rows_per_item = kTreeGenericRows;
    p.key_tile = kTreeGenericKeys;
    L = tree_layout(num_seqs, num_tokens, m.group, num_kv_heads, head_dim, max_keys,
                    p.rows_per_item, p.key_tile, kTreeGenericGrid);
  }
  p.grid = L.grid;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.seqs = reinterpret_cast<int4*>(ws);
  p.cum = reinterpret_cast<int64_t*>(ws + L.cum_off);
  p.starts = reinterpret_cast<int4*>(ws + L.starts_off);
  p.part_ml = reinterpret_cast<float2*>(ws + L.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + L.o_off);
  CUtensorMap tq, tk, tv;
  if (tc) {
    const bool ok =
        query_map(&tq, q, num_tokens, num_heads, head_dim, m.group, p.tile_tokens) &&
        // (the head beside it is read much later, or by another SM: fetched together, 48 x 16 nodes
        // read 515 MB for 346 MB and took 107.8 us instead of 104.6)
        (fp8 ? pool_map_fp8(&tk, k_blocks, num_blocks, 16, num_kv_heads, head_dim, true) &&
                   pool_map_fp8(&tv, v_blocks, num_blocks, 16, num_kv_heads, head_dim, true)
             : pool_map_rows(&tk, k_blocks, num_blocks, num_kv_heads, head_dim) &&
                   pool_map_rows(&tv, v_blocks, num_blocks, num_kv_heads, head_dim));
    if (!ok) return PA_ECUDA;
  }
  if (!p.cluster && launch_tree_plan(p, stream) != cudaSuccess) return PA_ECUDA;
  if (tc) {
    uint64_t limit;
    uint32_t stall;
    stall_hook(limit, stall);
    if (launch_tree_tc(tq, tk, tv, p, fp8, limit, stall, stream) != cudaSuccess) return PA_ECUDA;
    if (p.cluster) return PA_OK;
  } else if (launch_tree_generic(p, kv_dtype, stream) != cudaSuccess) {
    return PA_ECUDA;
  }
  return from_cuda(launch_tree_merge(p, stream));
}

pa_status pa_tree_commit(void* k_blocks, void* v_blocks, const int32_t* block_tables,
                         const int32_t* context_lens, const int32_t* accepted,
                         const int32_t* num_accepted, int32_t num_seqs, int32_t max_accepted,
                         int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                         int64_t num_blocks, int32_t max_blocks_per_seq, pa_dtype kv_dtype,
                         cudaStream_t stream) {
  if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0) return PA_ESHAPE;
  if (!pool_dtype_ok(kv_dtype)) return PA_EUNSUPPORTED;
  if (num_seqs < 0 || max_accepted < 0 || num_blocks < 0 || max_blocks_per_seq < 0)
    return PA_EINVAL;
  const int64_t row_bytes = (int64_t)num_kv_heads * head_dim * esize(kv_dtype);
  if (row_bytes > (1 << 22)) return PA_EUNSUPPORTED;
  if (num_seqs == 0 || max_accepted == 0) return PA_OK;
  if (!k_blocks || !v_blocks || !block_tables || !context_lens || !accepted || !num_accepted)
    return PA_EINVAL;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;
  return from_cuda(launch_tree_commit(k_blocks, v_blocks, block_tables, context_lens, accepted,
                                      num_accepted, num_seqs, max_accepted, max_blocks_per_seq,
                                      row_bytes, block_size, num_blocks, d->status, stream));
}

pa_status pa_copy_blocks(void* k_blocks, void* v_blocks, const int32_t* block_pairs,
                         int64_t num_pairs, int32_t num_kv_heads, int32_t head_dim,
                         int32_t block_size, int64_t num_blocks, pa_dtype kv_dtype,
                         cudaStream_t stream) {
  if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0) return PA_ESHAPE;
  if (!pool_dtype_ok(kv_dtype)) return PA_EUNSUPPORTED;
  if (num_pairs < 0 || num_blocks < 0) return PA_EINVAL;
  if (num_pairs == 0) return PA_OK;
  if (!k_blocks || !block_pairs || !aligned(block_pairs, 8)) return PA_EINVAL;
  const int64_t block_bytes = (int64_t)block_size * num_kv_heads * head_dim * esize(kv_dtype);
  // (a list longer than kFusedPairs is checked with one bit per block)
  if (num_pairs > INT32_MAX / 2 || block_bytes > (1ll << 31) ||
      (num_pairs > kFusedPairs && num_blocks > kMaxTrackedBlocks))
    return PA_EUNSUPPORTED;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;
  return from_cuda(launch_copy_blocks(k_blocks, v_blocks, block_pairs, num_pairs, block_bytes,
                                      num_blocks, d->status, d->sms, stream));
}

static pa_status pages_call(int what, PagesParams& p, const int32_t* rows, const int32_t* other,
                            cudaStream_t stream) {
  if (p.block_size <= 0) return PA_ESHAPE;
  if (p.count < 0 || p.num_rows < 0 || p.max_blocks < 0 || p.num_blocks < 0) return PA_EINVAL;
  if (p.count == 0) return PA_OK;
  if (p.count > p.num_rows) return PA_EINVAL;  // the written rows cannot be distinct
  if (p.num_rows > kMaxPageRows || p.num_blocks > kMaxTrackedBlocks ||
      (int64_t)p.num_rows * p.max_blocks > INT32_MAX)
    return PA_EUNSUPPORTED;
  if (!p.block_tables || !p.seq_lens || !rows || (what != PAGES_FREE && !other) ||
      (what == PAGES_FORK && !p.block_pairs) || !p.ref_counts || !p.free_list || !p.free_count)
    return PA_EINVAL;
  const DeviceState* d = device_state();
  if (!d) return PA_ECUDA;
  p.rows = rows;
  p.other = other;
  p.status = d->status;
  return from_cuda(launch_pages(what, p, stream));
}

pa_status pa_fork_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* parents,
                            const int32_t* children, int32_t num_forks, int32_t num_rows,
                            int32_t max_blocks_per_seq, int32_t block_size, int32_t* ref_counts,
                            int32_t* free_list, int32_t* free_count, int64_t num_blocks,
                            int32_t* block_pairs, cudaStream_t stream) {
  PagesParams p{};
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.block_pairs = block_pairs;
  p.ref_counts = ref_counts;
  p.free_list = free_list;
  p.free_count = free_count;
  p.count = num_forks;
  p.num_rows = num_rows;
  p.max_blocks = max_blocks_per_seq;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  return pages_call(PAGES_FORK, p, parents, children, stream);
}

pa_status pa_grow_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* sequences,
                            const int32_t* new_lens, int32_t num_sequences, int32_t num_rows,
                            int32_t max_blocks_per_seq, int32_t block_size, int32_t* ref_counts,
                            int32_t* free_list, int32_t* free_count, int64_t num_blocks,
                            cudaStream_t stream) {
  PagesParams p{};
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.ref_counts = ref_counts;
  p.free_list = free_list;
  p.free_count = free_count;
  p.count = num_sequences;
  p.num_rows = num_rows;
  p.max_blocks = max_blocks_per_seq;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  return pages_call(PAGES_GROW, p, sequences, new_lens, stream);
}

pa_status pa_free_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* sequences,
                            int32_t num_sequences, int32_t num_rows, int32_t max_blocks_per_seq,
                            int32_t block_size, int32_t* ref_counts, int32_t* free_list,
                            int32_t* free_count, int64_t num_blocks, cudaStream_t stream) {
  PagesParams p{};
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.ref_counts = ref_counts;
  p.free_list = free_list;
  p.free_count = free_count;
  p.count = num_sequences;
  p.num_rows = num_rows;
  p.max_blocks = max_blocks_per_seq;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  return pages_call(PAGES_FREE, p, sequences, nullptr, stream);
}

pa_status pa_trim_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* sequences,
                            const int32_t* new_lens, int32_t num_sequences, int32_t num_rows,
                            int32_t max_blocks_per_seq, int32_t block_size, int32_t* ref_counts,
                            int32_t* free_list, int32_t* free_count, int64_t num_blocks,
                            cudaStream_t stream) {
  PagesParams p{};
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.ref_counts = ref_counts;
  p.free_list = free_list;
  p.free_count = free_count;
  p.count = num_sequences;
  p.num_rows = num_rows;
  p.max_blocks = max_blocks_per_seq;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  if (num_sequences > 0 && !new_lens) return PA_EINVAL;
  return pages_call(PAGES_FREE, p, sequences, new_lens, stream);
}

}  // extern "C"
