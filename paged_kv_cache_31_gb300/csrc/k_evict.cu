// k_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Of a sequence's n keys a kv head keeps `new`: the first f, the last r and, of those between, the m =
// new - f - r with the largest weights (ties: the lowest index).  The places [f, new - r) hold m keys,
// too: those of the m that lie there stay, the others fill the places that became free, in ascending
// order, and the last r rows move up behind them.  So a cache that is cut by a few keys moves its
// recent rows and a few others, not everything behind the first evicted key.
//
// k_evict_select (one CTA per (sequence, kv head)): the m-th largest weight by histograms over 11, 11 and
// 10 bits of its order-preserving integer form (the first covers exponent and two bits of the fraction, so
// its bins seldom collide; bisection by two bits a step took 2.6 times as many instructions, which bound
// it); then two bitmaps, of the larger keys and of the equal ones, whose prefix sums number the places and
// the keys that fill them.
//
// k_evict_move: pure data movement, bound by memory.  A sequence's moves in list order (the fillers,
// then the recent rows, ascending) never write a row that a later one reads, so a CTA that moves its
// part of every row - a slice of K's or of V's bytes, or the weights - needs only to read a batch of
// rows before it writes the batch.  Slices are independent: no order between CTAs.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBins = 2048;

// Larger weights have larger keys; both zeros the same, NaN the largest.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (!(w == w)) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Plan {
  int n, to, first, recent, middle;  // `to` keys are kept
};
__device__ __forceinline__ Plan evict_plan(const EvictParams& p, int s) {
  Plan e;
  e.n = p.seq_lens[s];
  e.to = p.new_lens[s];
  e.first = min(p.keep_first, e.to);
  e.recent = min(p.keep_recent, e.to - e.first);
  e.middle = e.to - e.first - e.recent;
  return e;
}
// Whether the sequence's numbers can be used as indices.
__device__ __forceinline__ bool evict_bad(const EvictParams& p, const Plan& e) {
  return e.n < 0 || e.to < 0 || ((int64_t)e.n + p.block_size - 1) / p.block_size > p.max_blocks ||
         (p.key_weights && e.n > p.weights_len);
}
__device__ __forceinline__ int64_t moves_at(const EvictParams& p, int64_t unit) {
  return unit * (2 * p.moves_len + 2);
}

// Lists of a unit (sequence, kv head) in the workspace: the number of fillers, then from which index
// each comes, then (from moves_len on) where it goes.
// E > 0: a thread keeps the (ordered forms of the) weights of up to E keys in registers; 0: they are read
// again in every pass.
template <int NT, int E>
__global__ void __launch_bounds__(NT) k_evict_select(const EvictParams p) {
  extern __shared__ uint32_t s_bits[];  // larger keys, then equal ones, 32 to a word
  __shared__ int s_hist[kBins];
  __shared__ int3 s_found;  // bin, keys in larger ones, keys in it
  __shared__ int s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int s = blockIdx.y, g = blockIdx.x;
  const int64_t unit = (int64_t)s * p.num_kv_heads + g;
  int32_t* list = p.moves + moves_at(p, unit);
  const Plan e = evict_plan(p, s);
  bool bad = evict_bad(p, e);
  const float* w = p.key_weights ? p.key_weights + unit * p.weights_len + e.first : nullptr;
  const int count = e.n - e.recent - e.first;  // keys between the first and the recent ones
  uint32_t own[E > 0 ? E : 1];
  if constexpr (E > 0) {
    const bool any = !bad && e.to < e.n && w;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int i = tid + k * NT;
      own[k] = any && i < count ? order_key(__ldg(w + i)) : 0u;
    }
  }
  if (g == 0 && !bad && e.to < e.n) {  // the blocks that the sequence's rows lie in
    const int need = (e.n + p.block_size - 1) / p.block_size;
    for (int i = tid; i < need; i += NT) {
      const int id = p.block_tables[(int64_t)s * p.max_blocks + i];
      bad |= id < 0 || (int64_t)id >= p.num_blocks;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) record_error(p.status, PA_EINVAL);
  if (bad || e.to >= e.n || e.middle == 0) {
    if (tid == 0) list[0] = 0;
    return;
  }
  const int words = (count + 31) / 32;
  auto key = [&](int i) { return w ? order_key(__ldg(w + i)) : 0u; };
  // the middle-th largest key, 11, 11 and 10 bits at a time: the bin that holds it among the keys that
  // agree with the bits found so far
  uint32_t at = 0;
  int need = e.middle;
#pragma unroll 1
  for (int pass = 0; w && pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    for (int i = tid; i < kBins; i += NT) s_hist[i] = 0;
    __syncthreads();
    auto count_key = [&](uint32_t k) {  // (0: a key that is not there)
      if (k != 0 && (pass == 0 || k >> (shift + bits) == at >> (shift + bits)))
        atomicAdd(&s_hist[(k >> shift) & ((1 << bits) - 1)], 1);
    };
    if constexpr (E > 0) {
#pragma unroll
      for (int k = 0; k < E; ++k) count_key(own[k]);
    } else {
#pragma unroll 4
      for (int i = tid; i < count; i += NT) count_key(key(i));
    }
    __syncthreads();
    constexpr int kPer = kBins / NT;  // bins of a thread, from the highest down
    int sum = 0, total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) sum += s_hist[kBins - 1 - (tid * kPer + k)];
    int before = block_exclusive_scan(sum, s_warp, &total);
    if (before < need && need <= before + sum) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int bin = kBins - 1 - (tid * kPer + k), n = s_hist[bin];
        if (before < need && need <= before + n) s_found = make_int3(bin, before, n);
        before += n;
      }
    }
    __syncthreads();
    at |= (uint32_t)s_found.x << shift;
    need -= s_found.y;
    if (need == s_found.z) break;  // all of the bin's keys are taken
    __syncthreads();
  }
  uint32_t* more = s_bits;
  uint32_t* same = s_bits + words;
  auto mark = [&](int i0, uint32_t k) {
    const bool in = i0 + lane < count;
    const uint32_t a = __ballot_sync(kFull, in && k > at);
    const uint32_t b = __ballot_sync(kFull, in && k == at);
    if (lane == 0) {
      more[i0 >> 5] = a;
      same[i0 >> 5] = b;
    }
  };
  if constexpr (E > 0) {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (warp * 32 + k * NT < count) mark(warp * 32 + k * NT, own[k]);
  } else {
    for (int i0 = warp * 32; i0 < count; i0 += NT) mark(i0, i0 + lane < count ? key(i0 + lane) : 0u);
  }
  __syncthreads();
  // a thread's words are consecutive, so prefix sums over threads number the keys in order
  const int per = (words + NT - 1) / NT, w0 = min(words, tid * per), w1 = min(words, w0 + per);
  int larger = 0, equal = 0;
  for (int i = w0; i < w1; ++i) {
    larger += __popc(more[i]);
    equal += __popc(same[i]);
  }
  int total_larger, total;
  block_exclusive_scan(larger, s_warp, &total_larger);
  int ties = e.middle - total_larger - block_exclusive_scan(equal, s_warp, &total);  // left for this thread
  int holes = 0, fillers = 0;
  const int stay = e.middle;  // kept keys in front of this index of the middle stay where they are
  for (int i = w0; i < w1; ++i) {
    uint32_t b = same[i], kept = more[i];
    if (ties >= __popc(b)) {
      kept |= b;
    } else {
      for (int k = 0; k < ties; ++k) {
        kept |= b & (0u - b);
        b &= b - 1;
      }
    }
    ties = max(0, ties - __popc(same[i]));
    const int in = stay - 32 * i;  // bits below it stay
    const uint32_t front = in >= 32 ? kFull : in <= 0 ? 0u : (1u << in) - 1u;
    more[i] = kept & ~front;  // fillers
    same[i] = ~kept & front;  // holes
    fillers += __popc(more[i]);
    holes += __popc(same[i]);
  }
  const int f0 = block_exclusive_scan(fillers, s_warp, &total);
  int h0 = block_exclusive_scan(holes, s_warp, &total);
  if (tid == 0) list[0] = total;
  int32_t* from = list + 2 + f0;
  int32_t* to = list + 2 + p.moves_len + h0;
  for (int i = w0; i < w1; ++i) {
    for (uint32_t b = more[i]; b; b &= b - 1) *from++ = e.first + 32 * i + __ffs(b) - 1;
    for (uint32_t b = same[i]; b; b &= b - 1) *to++ = e.first + 32 * i + __ffs(b) - 1;
  }
}

// Move the weights of a unit, and zero those of the keys behind its new end.
__device__ __forceinline__ void move_weights(const EvictParams& p, const Plan& e, int64_t unit,
                                             const int32_t* list, int fillers) {
  float* w = p.key_weights + unit * p.weights_len;
  const int moves = fillers + e.recent;
  for (int b = 0; b < moves; b += 4 * blockDim.x) {
    float v[4];
    int to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = b + u * blockDim.x + threadIdx.x;
      to[u] = -1;
      if (i < moves) {
        const int k = i - fillers;
        v[u] = w[k < 0 ? list[2 + i] : e.n - e.recent + k];
        to[u] = k < 0 ? list[2 + p.moves_len + i] : e.to - e.recent + k;
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (to[u] >= 0) w[to[u]] = v[u];
    __syncthreads();
  }
  for (int i = e.to + threadIdx.x; i < e.n; i += blockDim.x) w[i] = 0.f;
}

// blockIdx.x: a slice of `width` accesses of K's rows, then of V's, then (given weights) the weights.
// Rows are read one batch ahead of the batch that is written, and the places of the batch after that are
// looked up meanwhile, so reads are in flight all the time.
template <typename T>
__global__ void __launch_bounds__(256) k_evict_move(const EvictParams p, int slices, int width,
                                                    int row_words) {
  constexpr int U = 2;  // rows of a thread's batch
  const int s = blockIdx.z, g = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  if (__syncthreads_or(status_set(p.status))) return;
  const Plan e = evict_plan(p, s);
  // (the status word may have been cleared by another stream in between)
  if (evict_bad(p, e) || e.to >= e.n) return;
  const int64_t unit = (int64_t)s * p.num_kv_heads + g;
  const int32_t* list = p.moves + moves_at(p, unit);
  const int fillers = __ldcg(list);
  if (blockIdx.x == 2 * slices) {
    move_weights(p, e, unit, list, fillers);
    return;
  }
  T* pool = static_cast<T*>(blockIdx.x < slices ? p.k_blocks : p.v_blocks);
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  const int moves = fillers + e.recent;
  const int x = (blockIdx.x % slices) * width + threadIdx.x % width, lane = threadIdx.x / width;
  const int step = blockDim.x / width;
  const bool in = x < row_words && lane < step;
  struct Places {
    int from[U], to[U];  // slots, or -1
  };
  auto slot = [&](int i) -> int {  // of index i, or -1
    int b, o;
    if (p.block_shift >= 0) {
      b = i >> p.block_shift;
      o = i & (p.block_size - 1);
    } else {
      b = i / p.block_size;
      o = i - b * p.block_size;
    }
    const int id = table[b];
    if (id < 0 || (int64_t)id >= p.num_blocks) return -1;
    return id * p.block_size + o;
  };
  T* mine = pool + (int64_t)g * row_words + x;
  const int64_t stride = (int64_t)p.num_kv_heads * row_words;
  auto places = [&](int b, Places& at) {
    int i0[U], i1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * step + lane, k = i - fillers;
      i0[u] = i1[u] = -1;
      if (in && i < moves) {
        // (the lists are read before their length is known)
        const int a = i < p.moves_len ? __ldcg(list + 2 + i) : 0;
        const int b = i < p.moves_len ? __ldcg(list + 2 + p.moves_len + i) : 0;
        i0[u] = k < 0 ? a : e.n - e.recent + k;
        i1[u] = k < 0 ? b : e.to - e.recent + k;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at.from[u] = i0[u] >= 0 ? slot(i0[u]) : -1;
      at.to[u] = i1[u] >= 0 && at.from[u] >= 0 ? slot(i1[u]) : -1;
    }
  };
  auto read = [&](const Places& at, T (&v)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at.to[u] >= 0) v[u] = mine[at.from[u] * stride];
  };
  auto write = [&](const Places& at, const T (&v)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at.to[u] >= 0) mine[at.to[u] * stride] = v[u];
  };
  const int batch = U * step;
  Places a, b;
  T va[U], vb[U];
  places(0, a);
  read(a, va);
  places(batch, b);
  for (int i = 0; i < moves; i += 2 * batch) {
    read(b, vb);
    Places c;
    places(i + 2 * batch, c);
    __syncthreads();  // batch i has been read by all
    write(a, va);
    a = c;
    read(a, va);
    places(i + 3 * batch, c);
    __syncthreads();
    write(b, vb);
    b = c;
  }
}

template <typename T>
cudaError_t move_as(const EvictParams& p, cudaStream_t stream) {
  const int row_words = (int)(p.row_bytes / sizeof(T));
  // whole rows to a CTA, up to 256 accesses
  const int width = std::min(row_words, 256), slices = (row_words + width - 1) / width;
  const dim3 grid(2 * slices + (p.key_weights ? 1 : 0), p.num_kv_heads, p.num_seqs);
  return launch_pdl(k_evict_move<T>, grid, dim3(256), 0, stream, p, slices, width, row_words);
}

template <int NT, int E>
cudaError_t select_as(const EvictParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)((p.moves_len + 31) / 32) * 8;
  auto kern = k_evict_select<NT, E>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.num_kv_heads, p.num_seqs), dim3(NT), smem, stream, p);
}

}  // namespace

int64_t evict_workspace(int32_t num_seqs, int32_t num_kv_heads, int64_t max_keys) {
  return (int64_t)num_seqs * num_kv_heads * (2 * max_keys + 2) * 4;
}

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
  const int64_t keys = p.moves_len;  // at most
  const cudaError_t e = keys <= 2048   ? select_as<256, 8>(p, stream)
                        : keys <= 8192 ? select_as<1024, 8>(p, stream)
                                       : select_as<1024, 0>(p, stream);
  if (e != cudaSuccess) return e;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.k_blocks) | reinterpret_cast<uintptr_t>(p.v_blocks) |
                       (uintptr_t)p.row_bytes;
  if (at % 16 == 0) return move_as<uint4>(p, stream);
  if (at % 4 == 0) return move_as<uint32_t>(p, stream);
  return move_as<uint8_t>(p, stream);
}

}  // namespace pa
