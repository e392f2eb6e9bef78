// k_tree.cu -- attention of a tree of drafted tokens over the paged cache: the planning kernel,
// the general kernel (any types, head size and block size) and the merge of split items.
//
// Math.  Sequence s has n nodes (its query tokens), cached as its last n positions behind a
// context of c = seq_len - n positions.  Node t attends to the context and to the nodes whose
// bit is set in its mask row (its ancestors and itself, in a tree).  A key's logical position is
// j for context position j and positions[node] for a node; with a sliding window w a key is
// visible when its logical position is greater than positions[t] - w.  The visible scores go
// through one softmax, online over key tiles: m' = max(m, .), l = 2^(m - m') l + sum p,
// O = 2^(m - m') O + P V.
//
// Why split: a drafted step has few query rows and long contexts, so (sequence, kv head) items
// alone do not fill the GPU evenly.  All items' key tiles are laid end to end and every CTA
// takes an equal, contiguous share; the pieces of an item are merged afterwards in key order.
// How a batch is cut depends on its lengths alone, so equal inputs give equal bits.  (Small calls
// on the tensor cores need none of this: k_tree_tc.cu's clusters.)  Measured beside an attention
// kernel of 118 us (64 sequences, 151 cuts of up to 128 rows): the plan 4.7 us, the merge 10 us.
#include <algorithm>

#include "k_tree.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPlanThreads = 1024;
constexpr int kCumShared = 2048;  // sequences whose prefix weights the planner keeps in smem

__device__ __forceinline__ int64_t block_sum_scan(int64_t v, int64_t* s_warp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, w, o);
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

// Block 0 plans; blocks 1 .. check the table entries of the sequences, one warp per 256 entries.
// Everything is read after the wait for the kernels ahead, and nothing is written by the
// attention kernel before this whole launch is done, so an error leaves the outputs untouched.  (The
// status word may be cleared by another stream before the kernels behind read it.  Their indices hold
// all the same: a plan that failed is one of empty shares, and block ids are looked at again where
// they are used, by the copies' tensor maps or the general kernel.)
__global__ void __launch_bounds__(kPlanThreads) k_tree_plan(const TreeParams p) {
  __shared__ int64_t s_warp[32];
  __shared__ int64_t s_cum[kCumShared + 1];
  __shared__ int s_first[kPlanThreads], s_nodes[kPlanThreads], s_low[kPlanThreads];
  const VarlenMeta& m = p.m;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  if (blockIdx.x > 0) {
    const int warps = (gridDim.x - 1) * (kPlanThreads / 32);
    const int me = (blockIdx.x - 1) * (kPlanThreads / 32) + warp;
    const int per = (m.max_blocks + 255) / 256;  // chunks of a table row
    const int64_t chunks = (int64_t)m.num_seqs * per;
    for (int64_t c = me; c < chunks; c += warps) {
      const int s = (int)(c / per), e0 = (int)(c % per) * 256;
      const int n = m.seq_lens[s];
      if (m.query_start_loc[s + 1] <= m.query_start_loc[s] || n < 1) continue;
      const int64_t need = ((int64_t)n + m.block_size - 1) / m.block_size;
      const int lim = (int)min(need, (int64_t)m.max_blocks);
      const int32_t* row = m.block_tables + (int64_t)s * m.max_blocks;
      int id[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int e = e0 + lane + 32 * u;
        id[u] = e < lim ? row[e] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) bad |= id[u] < 0 || (int64_t)id[u] >= m.num_blocks;
    }
    if (__any_sync(kFull, bad) && lane == 0) record_error(p.status, PA_EINVAL);
    return;
  }

  // per-head scales (each array may be missing)
  for (int g = tid; g < m.num_kv_heads; g += kPlanThreads) {
    const float a = m.k_scales ? m.k_scales[g] : 1.f, b = m.v_scales ? m.v_scales[g] : 1.f;
    bad |= !(a > 0.f && a <= 3.402823466e38f) || !(b > 0.f && b <= 3.402823466e38f);
  }
  int64_t base = 0;
  for (int s0 = 0; s0 < m.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int qs = 0, nodes = 0, n = 0;
    if (s < m.num_seqs) {
      qs = m.query_start_loc[s];
      const int qe = m.query_start_loc[s + 1];
      bad |= qs < 0 || qe < qs || (int64_t)qe > m.num_tokens || (s == 0 && qs != 0) ||
             (s == m.num_seqs - 1 && (int64_t)qe != m.num_tokens);
      if (qs >= 0 && qe > qs && (int64_t)qe <= m.num_tokens) {
        nodes = qe - qs;
        n = m.seq_lens[s];
        if (n < nodes || nodes > 32 * (int64_t)p.mask_words ||
            ((int64_t)n + m.block_size - 1) / m.block_size > m.max_blocks) {
          bad = true;
          nodes = 0;
        }
      }
    }
    // with a window: the lowest position of each sequence's nodes decides the first key it reads
    if (m.window > 0) {
      s_first[tid] = qs;
      s_nodes[tid] = nodes;
      __syncthreads();
      const int here = min(kPlanThreads, m.num_seqs - s0);
      for (int i = warp; i < here; i += kPlanThreads / 32) {
        int lo = INT_MAX;
        for (int t = lane; t < s_nodes[i]; t += 32) lo = min(lo, m.positions[s_first[i] + t]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lo = min(lo, __shfl_xor_sync(kFull, lo, o));
        if (lane == 0) s_low[i] = lo;
      }
      __syncthreads();
    }
    int64_t weight = 0;
    if (nodes > 0) {
      int kv0 = 0;
      if (m.window > 0) {
        bad |= s_low[tid] < 0;
        kv0 = min(max(s_low[tid] - m.window + 1, 0), n - nodes);
      }
      kv0 -= kv0 % m.block_size;
      const int tiles = (n - kv0 + p.key_tile - 1) / p.key_tile;
      const int rows = nodes * m.group, items = (rows + p.rows_per_item - 1) / p.rows_per_item;
      p.seqs[2 * s] = make_int4(qs, nodes, n, kv0);
      p.seqs[2 * s + 1] = make_int4(items, tiles, rows, 0);
      weight = item_weight(p, tiles, p.rows_per_item) * (items - 1) +
               item_weight(p, tiles, rows - (items - 1) * p.rows_per_item);
      weight *= m.num_kv_heads;
    } else if (s < m.num_seqs) {
      p.seqs[2 * s] = p.seqs[2 * s + 1] = make_int4(0, 0, 0, 0);
    }
    int64_t total;
    const int64_t at = base + block_sum_scan(weight, s_warp, &total);
    if (s < m.num_seqs) {
      p.cum[s] = at;
      if (s < kCumShared) s_cum[s] = at;
    }
    base += total;
  }
  if (tid == 0) {
    p.cum[m.num_seqs] = base;
    if (m.num_seqs <= kCumShared) s_cum[m.num_seqs] = base;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (tid == 0) record_error(p.status, PA_EINVAL);
    for (int c = tid; c <= p.grid; c += kPlanThreads) p.starts[c] = make_int4(m.num_seqs, 0, 0, 0);
    return;
  }
  // where each CTA's share begins
  const bool shared = m.num_seqs <= kCumShared;
  for (int c = tid; c <= p.grid; c += kPlanThreads) {
    int4 st = make_int4(m.num_seqs, 0, 0, 0);
    if (c < p.grid && base > 0) {
      const int64_t x = base / p.grid * c + base % p.grid * c / p.grid;  // floor(base c / grid)
      int lo = 0, hi = m.num_seqs;  // the last sequence with cum <= x
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((shared ? s_cum[mid] : p.cum[mid]) <= x) lo = mid; else hi = mid;
      }
      const int64_t rem = x - (shared ? s_cum[lo] : p.cum[lo]);
      const int4 w = p.seqs[2 * lo + 1];
      const int last_rows = w.z - (w.x - 1) * p.rows_per_item;
      const int64_t full = item_weight(p, w.y, p.rows_per_item);
      const int64_t per_head = full * (w.x - 1) + item_weight(p, w.y, last_rows);
      const int kvh = (int)(rem / per_head);
      const int64_t r = rem % per_head;
      const int it = (int)min(r / full, (int64_t)w.x - 1);
      const int64_t in = max(r - it * full - kTreeItemWeight, (int64_t)0);
      const int tw = tree_weight(p, it == w.x - 1 ? last_rows : p.rows_per_item);
      st = make_int4(lo, kvh, it, (int)min(in / tw, (int64_t)w.y - 1));
    }
    p.starts[c] = st;
  }
}

// ---- the general kernel -----------------------------------------------------------------------
// 32 query rows x 32 keys per step in fp32 on the FMA pipes: thread (rg = tid / 16, c = tid % 16)
// computes the scores of rows 4 rg .. 4 rg + 3 and keys c and c + 16, and dims 4c + 64i .. of the
// same rows' outputs.  It is bound by shared-memory reads (a 16-byte read takes as long as 16 of
// a warp's FMAs): 9 of them for the 64 FMAs per thread of four dims of Q K^T and one key of P V at
// head size 128, against 18 when a thread had one row, eight keys and a quarter of the dims
// (16 x 16 nodes x 4 heads over 2000 fp32 positions: 563 -> 299 us).  The arithmetic is packed, two
// fp32 to an instruction, and the loops written out by eight: 275 us, 31 TFLOP/s.
// Rows of the tiles are padded by four floats, so 16-byte reads of different rows hit different
// banks.

constexpr int kBM = kTreeGenericRows, kBN = kTreeGenericKeys;

template <typename TKV>
__device__ __forceinline__ float4 load4(const TKV* p) {
  if constexpr (sizeof(TKV) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else if constexpr (sizeof(TKV) == 2) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  } else {
    uint32_t lo, hi;
    e4m3x4_to_f16(*reinterpret_cast<const uint32_t*>(p), lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(a.x, a.y, b.x, b.y);
  }
}

// Up to four of the n values that a row has left at p.
template <typename T>
__device__ __forceinline__ float4 row4(const T* p, int n, bool vec) {
  if (vec) return load4<T>(p);
  float x[4] = {};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) x[e] = to_f32(p[e]);
  return make_float4(x[0], x[1], x[2], x[3]);
}

constexpr int kLDP = kBM + 4;  // row length of the transposed weights

template <int DP>
constexpr size_t generic_smem() {
  return (size_t)((kBM + 2 * kBN) * (DP + 4) + kBN * kLDP) * 4;
}

// DP: head size padded to 64, 128 or 256; vec: rows can be read four elements at a time
template <typename TQ, typename TKV, int DP>
__global__ void __launch_bounds__(128) k_tree_generic(const TreeParams p, const bool vec) {
  constexpr int LD = DP + 4;
  constexpr int kDI = DP / 64;  // float4s of a thread's output row
  // when a tile is read, a thread's four columns are the same in all its rows, kStep apart
  constexpr int kCols = DP / 4, kStep = 128 / kCols;
  extern __shared__ __align__(16) float s_mem[];
  float* sq = s_mem;
  float* sk = sq + kBM * LD;
  float* sv = sk + kBN * LD;
  float* sp = sv + kBN * LD;      // [key][row]
  __shared__ int64_t s_row[kBN];  // pool rows (position, kv head) of the tile's keys, or -1
  __shared__ int s_skip;
  const VarlenMeta& m = p.m;
  const int tid = threadIdx.x, rg = 4 * (tid >> 4), c = tid & 15;
  const int col = tid % kCols * 4;
  const int D = m.head_dim, G = m.group;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) s_skip = status_set(p.status) ? 1 : 0;
  __syncthreads();
  if (s_skip) return;
  const TQ* q = static_cast<const TQ*>(p.q);
  const TKV* kb = static_cast<const TKV*>(p.k_blocks);
  const TKV* vb = static_cast<const TKV*>(p.v_blocks);

  TreeWalk walk(p, blockIdx.x);
  TreeSegment sg;
  while (walk.next(p, sg)) {
    const int rows = sg.rows;
    int tok[4], pos[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      tok[k] = sg.qs + (rg + k < rows ? (sg.row0 + rg + k) / G : 0);
      pos[k] = m.window > 0 ? m.positions[tok[k]] : 0;
    }
    const float sl = head_scale(m.k_scales, sg.kvh, p.scale) * kLog2e;
    __syncthreads();  // the buffers of the segment before are free
    for (int r0 = tid / kCols; r0 < kBM; r0 += 4 * kStep) {
      float4 a[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int rr = r0 + u * kStep, R = sg.row0 + rr;
        a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rr < rows && col < D)
          a[u] = row4<TQ>(q + ((int64_t)(sg.qs + R / G) * m.num_heads + sg.kvh * G + R % G) * D + col,
                          D - col, vec);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<float4*>(sq + (r0 + u * kStep) * LD + col) = a[u];
    }
    float mx[4], l[4];
    ulonglong2 o[4][kDI];  // packed pairs of fp32
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mx[k] = -INFINITY;
      l[k] = 0.f;
#pragma unroll
      for (int i = 0; i < kDI; ++i) o[k][i] = make_ulonglong2(0, 0);
    }
    const int32_t* trow = m.block_tables + (int64_t)sg.s * m.max_blocks;
    for (int j = sg.t0; j < sg.t1; ++j) {
      const int key0 = sg.kv0 + j * kBN;
      if (tid < kBN) {
        const int key = key0 + tid, id = key < sg.n ? trow[key / m.block_size] : -1;
        s_row[tid] = id >= 0 && (int64_t)id < m.num_blocks
                         ? ((int64_t)id * m.block_size + key % m.block_size) * m.num_kv_heads + sg.kvh
                         : -1;
      }
      __syncthreads();  // (the tile before has been used, too)
      for (int k0 = tid / kCols; k0 < kBN; k0 += 4 * kStep) {
        float4 a[4], b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // (four rows in flight)
          a[u] = b[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          const int64_t at = s_row[k0 + u * kStep] * D + col;
          if (at < 0 || col >= D) continue;
          a[u] = row4<TKV>(kb + at, D - col, vec);
          b[u] = row4<TKV>(vb + at, D - col, vec);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int kk = k0 + u * kStep;
          *reinterpret_cast<float4*>(sk + kk * LD + col) = a[u];
          *reinterpret_cast<float4*>(sv + kk * LD + col) = b[u];
        }
      }
      __syncthreads();
      uint64_t x2[4][2] = {};  // sums over even and over odd dims, two to a packed instruction
#pragma unroll 8
      for (int d4 = 0; d4 < DP; d4 += 4) {
        ulonglong2 b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          b[i] = *reinterpret_cast<const ulonglong2*>(sk + (c + 16 * i) * LD + d4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(sq + (rg + k) * LD + d4);
#pragma unroll
          for (int i = 0; i < 2; ++i) x2[k][i] = f2_fma(a.y, b[i].y, f2_fma(a.x, b[i].x, x2[k][i]));
        }
      }
      float x[4][2];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float even, odd;
          f2_unpack(x2[k][i], even, odd);
          x[k][i] = even + odd;
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          x[k][i] = rg + k < rows && tree_visible(p, sg, tok[k], pos[k], key0 + c + 16 * i)
                        ? x[k][i] * sl
                        : -INFINITY;
        float mt = fmaxf(x[k][0], x[k][1]);
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, s));
        const float mn = fmaxf(mx[k], mt), b0 = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(mx[k] - b0);
        x[k][0] = exp2f(x[k][0] - b0);
        x[k][1] = exp2f(x[k][1] - b0);
        mx[k] = mn;
        l[k] = l[k] * alpha + (x[k][0] + x[k][1]);  // this thread's keys; summed at the end
#pragma unroll
        for (int i = 0; i < kDI; ++i) {
          o[k][i].x = f2_mul(o[k][i].x, f2_pack(alpha, alpha));
          o[k][i].y = f2_mul(o[k][i].y, f2_pack(alpha, alpha));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float4*>(sp + (c + 16 * i) * kLDP + rg) =
            make_float4(x[0][i], x[1][i], x[2][i], x[3][i]);
      __syncwarp();  // a row's weights come from its own warp
#pragma unroll 8
      for (int kk = 0; kk < kBN; ++kk) {
        const float4 w4 = *reinterpret_cast<const float4*>(sp + kk * kLDP + rg);
        const uint64_t w[4] = {f2_pack(w4.x, w4.x), f2_pack(w4.y, w4.y), f2_pack(w4.z, w4.z),
                               f2_pack(w4.w, w4.w)};
#pragma unroll
        for (int i = 0; i < kDI; ++i) {
          const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(sv + kk * LD + 4 * c + 64 * i);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[k][i].x = f2_fma(w[k], b.x, o[k][i].x);
            o[k][i].y = f2_fma(w[k], b.y, o[k][i].y);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) l[k] += __shfl_xor_sync(kFull, l[k], s);
      const int r = rg + k;
      if (r >= rows) continue;  // (the same for all sixteen threads of a row)
      const bool part = sg.slot >= 0;
      const int64_t at = (int64_t)sg.slot * p.rows_per_item + r;
      const int R = sg.row0 + r, h = sg.kvh * G + R % G;
      float f = 1.f;
      if (!part)
        f = tree_finish(p, sg.kvh, h, tok[k], mx[k], l[k], c == 0);
      else if (c == 0)
        p.part_ml[at] = make_float2(mx[k], l[k]);
      TQ* out = static_cast<TQ*>(p.out) + ((int64_t)tok[k] * m.num_heads + h) * D;
#pragma unroll
      for (int i = 0; i < kDI; ++i) {
        float v[4];
        f2_unpack(o[k][i].x, v[0], v[1]);
        f2_unpack(o[k][i].y, v[2], v[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = 4 * c + 64 * i + e;
          if (d >= D) continue;
          if (part)
            p.part_o[at * D + d] = v[e];
          else
            out[d] = from_f32<TQ>(v[e] * f);
        }
      }
    }
  }
}

// ---- merge ------------------------------------------------------------------------------------
// Block (b, y): the item that the boundary between CTA b and b + 1 cuts, when that is the item's
// first cut; a warp for R rows.  out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over
// the item's pieces in key order: CTA b's piece (its first segment when the item begins its share,
// else its last), then those of the CTAs behind it whose shares begin inside the item.  Bound by
// the latency of its loads: 32 pieces' states are read at once, a lane each, and the outputs of
// two pieces for all of the warp's rows.  A warp takes one row, or as many more as keep the whole
// grid resident at once (151 cuts of 128 rows: 12.5 us with one row, in two waves of CTAs).
// VEC: rows of whole float4s (head sizes that are multiples of 4); DK: 128-dim parts of a row
template <typename TQ, bool VEC, int DK, int R>
__global__ void __launch_bounds__(256) k_tree_merge(const TreeParams p) {
  constexpr int E = 4 * DK;  // a lane's values of a row
  const VarlenMeta& m = p.m;
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  // The plan is read before the wait: the attention kernel let this one start only after the
  // planning kernel's end.  (A plan that failed has empty shares: nothing is cut.)
  const int4 cut = __ldcg(&p.starts[b + 1]), from = __ldcg(&p.starts[b]);
  const bool in = cut.x >= 0 && cut.x < m.num_seqs;
  const int4 q = in ? __ldcg(&p.seqs[2 * cut.x]) : make_int4(0, 0, 0, 0);
  pdl_wait();
  pdl_launch_dependents();
  if (__syncthreads_or(status_set(p.status))) return;  // (one answer for the whole CTA)
  if (!in || cut.w == 0) return;
  const bool same = from.x == cut.x && from.y == cut.y && from.z == cut.z;
  if (same && from.w > 0) return;  // a later cut of the item
  const int kvh = cut.y, row0 = cut.z * p.rows_per_item;
  const int rows = min(p.rows_per_item, q.y * m.group - row0);
  const int row = (blockIdx.y * 8 + (threadIdx.x >> 5)) * R;
  if (row >= rows) return;
  const int D = m.head_dim, G = m.group;
  float M[R], L[R], acc[R][E];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    M[k] = -INFINITY;
    L[k] = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[k][i] = 0.f;
  }
  for (int c0 = b;; c0 += 32) {  // pieces of CTAs c0 .. c0 + 31, one per lane
    const int c = c0 + lane;
    bool in = c == b;
    int slot = same ? 2 * b : 2 * b + 1;
    if (c > b && c < p.grid) {
      const int4 s0 = p.starts[c], s1 = p.starts[c + 1];
      in = s0.x == cut.x && s0.y == cut.y && s0.z == cut.z;
      // (a CTA whose share is empty left nothing)
      slot = in && (s1.x != s0.x || s1.y != s0.y || s1.z != s0.z || s1.w != s0.w) ? 2 * c : -1;
    }
    const int n = __popc(__ballot_sync(kFull, in));  // contiguous from lane 0
    const bool have = in && slot >= 0;
    float w[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float2 ml = have && row + k < rows
                            ? p.part_ml[(int64_t)slot * p.rows_per_item + row + k]
                            : make_float2(-INFINITY, 0.f);
      float mx = ml.x;  // (over the lanes of the n pieces: their group of a power of two)
      for (int o = 1; o < n; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      mx = __shfl_sync(kFull, mx, 0);
      const float mn = fmaxf(M[k], mx), base = mn == -INFINITY ? 0.f : mn;
      const float a = exp2f(M[k] - base);
      w[k] = have ? exp2f(ml.x - base) : 0.f;
      float l = w[k] * ml.y;
      for (int o = 1; o < n; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
      l = __shfl_sync(kFull, l, 0);
      M[k] = mn;
      L[k] = L[k] * a + l;
#pragma unroll
      for (int i = 0; i < E; ++i) acc[k][i] *= a;
    }
    for (int j0 = 0; j0 < n; j0 += 2) {
      float x[2][R][E];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int sj = __shfl_sync(kFull, have ? slot : -1, min(j0 + u, 31));
        const bool ok = j0 + u < n && sj >= 0;
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const float* src = p.part_o + ((int64_t)sj * p.rows_per_item + row + k) * D;
          const bool get = ok && row + k < rows;
#pragma unroll
          for (int i = 0; i < DK; ++i) {
            if constexpr (VEC) {
              const int d = 128 * i + 4 * lane;
              const float4 v = get && d < D ? *reinterpret_cast<const float4*>(src + d)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
              x[u][k][4 * i] = v.x;
              x[u][k][4 * i + 1] = v.y;
              x[u][k][4 * i + 2] = v.z;
              x[u][k][4 * i + 3] = v.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int d = 128 * i + 32 * e + lane;
                x[u][k][4 * i + e] = get && d < D ? src[d] : 0.f;
              }
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < R; ++k) {
          const float wj = __shfl_sync(kFull, w[k], min(j0 + u, 31));
#pragma unroll
          for (int i = 0; i < E; ++i) acc[k][i] += (j0 + u < n ? wj : 0.f) * x[u][k][i];
        }
    }
    if (n < 32) break;
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (row + k >= rows) break;
    const int r = row0 + row + k;
    const int tok = q.x + r / G, h = kvh * G + r % G;
    const float inv = tree_finish(p, kvh, h, tok, M[k], L[k], lane == 0);
    TQ* out = static_cast<TQ*>(p.out) + ((int64_t)tok * m.num_heads + h) * D;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int d = VEC ? 128 * (i >> 2) + 4 * lane + (i & 3) : 128 * (i >> 2) + 32 * (i & 3) + lane;
      if (d < D) out[d] = from_f32<TQ>(acc[k][i] * inv);
    }
  }
}

template <typename TQ, bool VEC, int R>
cudaError_t merge_rows(const TreeParams& p, int64_t rows, cudaStream_t stream) {
  const dim3 grid((unsigned)(p.grid - 1), (unsigned)((rows + 8 * R - 1) / (8 * R)));
  if (p.m.head_dim <= 128)
    return launch_pdl(k_tree_merge<TQ, VEC, 1, R>, grid, dim3(256), 0, stream, p);
  return launch_pdl(k_tree_merge<TQ, VEC, 2, R>, grid, dim3(256), 0, stream, p);
}
template <typename TQ, bool VEC>
cudaError_t merge_as(const TreeParams& p, cudaStream_t stream) {
  const int64_t rows = std::min<int64_t>(p.rows_per_item, p.m.num_tokens * p.m.group);
  const int64_t warps = (p.grid - 1) * ((rows + 7) / 8 * 8), resident = 48 * (int64_t)num_sms();
  if (warps <= resident) return merge_rows<TQ, VEC, 1>(p, rows, stream);
  if (warps <= 2 * resident) return merge_rows<TQ, VEC, 2>(p, rows, stream);
  return merge_rows<TQ, VEC, 4>(p, rows, stream);
}

template <typename TQ, typename TKV, int DP>
cudaError_t generic_as(const TreeParams& p, bool vec, cudaStream_t stream) {
  auto kern = k_tree_generic<TQ, TKV, DP>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)generic_smem<DP>());
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.grid), dim3(128), generic_smem<DP>(), stream, p, vec);
}

template <typename TQ, typename TKV>
cudaError_t generic_dims(const TreeParams& p, cudaStream_t stream) {
  const int D = p.m.head_dim;
  const bool vec = D % 4 == 0 && aligned(p.q, 4 * sizeof(TQ)) && aligned(p.k_blocks, 4 * sizeof(TKV)) &&
                   aligned(p.v_blocks, 4 * sizeof(TKV));
  if (D <= 64) return generic_as<TQ, TKV, 64>(p, vec, stream);
  if (D <= 128) return generic_as<TQ, TKV, 128>(p, vec, stream);
  return generic_as<TQ, TKV, 256>(p, vec, stream);
}

}  // namespace

TreeLayout tree_layout(int32_t num_seqs, int64_t num_tokens, int32_t group, int32_t num_kv_heads,
                       int32_t head_dim, int64_t max_keys, int32_t rows_per_item,
                       int32_t key_tile, int32_t max_grid) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  TreeLayout L;
  // no more CTAs than there can be (item, key tile) pairs
  const int64_t items = (num_tokens * group / rows_per_item + num_seqs) * num_kv_heads;
  const int64_t tiles = max_keys / key_tile + 2;
  L.grid = (int32_t)std::max<int64_t>(1, std::min<int64_t>(max_grid, std::min<int64_t>(items, max_grid) * tiles));
  L.cum_off = up(32 * (int64_t)num_seqs);
  L.starts_off = L.cum_off + up(8 * ((int64_t)num_seqs + 1));
  L.ml_off = L.starts_off + up(16 * ((int64_t)L.grid + 1));
  L.o_off = L.ml_off + up(2 * (int64_t)L.grid * rows_per_item * 8);
  L.bytes = L.o_off + up(2 * (int64_t)L.grid * rows_per_item * head_dim * 4);
  return L;
}

cudaError_t launch_tree_plan(const TreeParams& p, cudaStream_t stream) {
  // table checks beside the planner: a warp per 256 entries, at most 64 blocks
  const int64_t chunks = (int64_t)p.m.num_seqs * ((p.m.max_blocks + 255) / 256);
  const int blocks = (int)std::min<int64_t>((chunks + 31) / 32, 64);
  return launch_pdl(k_tree_plan, dim3(1 + blocks), dim3(kPlanThreads), 0, stream, p);
}

cudaError_t launch_tree_generic(const TreeParams& p, pa_dtype kv, cudaStream_t stream) {
  if (p.q_bf16) {
    if (kv == PA_BF16) return generic_dims<__nv_bfloat16, __nv_bfloat16>(p, stream);
    if (kv == PA_F32) return generic_dims<__nv_bfloat16, float>(p, stream);
    return generic_dims<__nv_bfloat16, e4m3_t>(p, stream);
  }
  if (kv == PA_BF16) return generic_dims<float, __nv_bfloat16>(p, stream);
  if (kv == PA_F32) return generic_dims<float, float>(p, stream);
  return generic_dims<float, e4m3_t>(p, stream);
}

cudaError_t launch_tree_merge(const TreeParams& p, cudaStream_t stream) {
  if (p.grid < 2) return cudaSuccess;
  if (p.m.head_dim % 4 == 0)
    return p.q_bf16 ? merge_as<__nv_bfloat16, true>(p, stream) : merge_as<float, true>(p, stream);
  return p.q_bf16 ? merge_as<__nv_bfloat16, false>(p, stream) : merge_as<float, false>(p, stream);
}

}  // namespace pa
