// k_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Of a sequence's n keys a kv head keeps `new`: the first f, the last r and, of those between, the m =
// new - f - r with the largest weights (ties: the lowest index).  The places [f, new - r) hold m keys,
// too: those of the m that lie there stay, the others fill the places that became free, in ascending
// order, and the last r rows move up behind them.  So a cache that is cut by a few keys moves its
// recent rows and a few others, not everything behind the first evicted key.
//
// k_evict_select (one CTA per (sequence, kv head)): the m-th largest weight by bisection over the
// bits of its order-preserving integer form, two bits a step (16 steps over weights that stay in L1,
// counts by warp reductions; no histogram whose bins collide, as the exponents of weights do); then two
// bitmaps, of the larger keys and of the equal ones, whose prefix sums number the places and the keys
// that fill them.
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
template <int NT>
__global__ void __launch_bounds__(NT) k_evict_select(const EvictParams p) {
  extern __shared__ uint32_t s_bits[];  // larger keys, then equal ones, 32 to a word
  __shared__ int s_cnt[2][3][32];
  __shared__ int s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = NT / 32;
  const int s = blockIdx.y, g = blockIdx.x;
  const int64_t unit = (int64_t)s * p.num_kv_heads + g;
  int32_t* list = p.moves + moves_at(p, unit);
  const Plan e = evict_plan(p, s);
  bool bad = evict_bad(p, e);
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
  const float* w = p.key_weights ? p.key_weights + unit * p.weights_len + e.first : nullptr;
  const int count = e.n - e.recent - e.first;  // keys between the first and the recent ones
  const int words = (count + 31) / 32;
  auto key = [&](int i) { return w ? order_key(__ldg(w + i)) : 0u; };
  // the middle-th largest key: the largest value that at least `middle` keys reach
  uint32_t at = 0;
  for (int step = 0; w && step < 16; ++step) {
    const int shift = 30 - 2 * step;
    const uint32_t c1 = at + (1u << shift), c2 = at + (2u << shift), c3 = at + (3u << shift);
    int n1 = 0, n2 = 0, n3 = 0;
#pragma unroll 8
    for (int i = tid; i < count; i += NT) {
      const uint32_t k = key(i);
      n1 += k >= c1;
      n2 += k >= c2;
      n3 += k >= c3;
    }
    n1 = __reduce_add_sync(kFull, n1);
    n2 = __reduce_add_sync(kFull, n2);
    n3 = __reduce_add_sync(kFull, n3);
    int(&cnt)[3][32] = s_cnt[step & 1];
    if (lane == 0) {
      cnt[0][warp] = n1;
      cnt[1][warp] = n2;
      cnt[2][warp] = n3;
    }
    __syncthreads();
    n1 = __reduce_add_sync(kFull, lane < kWarps ? cnt[0][lane] : 0);
    n2 = __reduce_add_sync(kFull, lane < kWarps ? cnt[1][lane] : 0);
    n3 = __reduce_add_sync(kFull, lane < kWarps ? cnt[2][lane] : 0);
    at = n3 >= e.middle ? c3 : n2 >= e.middle ? c2 : n1 >= e.middle ? c1 : at;
  }
  uint32_t* more = s_bits;
  uint32_t* same = s_bits + words;
  for (int i0 = warp * 32; i0 < count; i0 += NT) {
    const int i = i0 + lane;
    const uint32_t k = i < count ? key(i) : 0u;
    const uint32_t a = __ballot_sync(kFull, i < count && k > at);
    const uint32_t b = __ballot_sync(kFull, i < count && k == at);
    if (lane == 0) {
      more[i0 >> 5] = a;
      same[i0 >> 5] = b;
    }
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
template <typename T>
__global__ void __launch_bounds__(256) k_evict_move(const EvictParams p, int slices, int width,
                                                    int row_words) {
  const int s = blockIdx.z, g = blockIdx.y;
  __shared__ int s_skip;
  if (threadIdx.x == 0) s_skip = status_set(p.status) ? 1 : 0;
  __syncthreads();
  if (s_skip) return;
  const Plan e = evict_plan(p, s);
  // (the status word may have been cleared by another stream in between)
  if (evict_bad(p, e) || e.to >= e.n) return;
  const int64_t unit = (int64_t)s * p.num_kv_heads + g;
  const int32_t* list = p.moves + moves_at(p, unit);
  const int fillers = list[0];
  if (blockIdx.x == 2 * slices) {
    move_weights(p, e, unit, list, fillers);
    return;
  }
  T* pool = static_cast<T*>(blockIdx.x < slices ? p.k_blocks : p.v_blocks);
  const int x0 = (blockIdx.x % slices) * width;
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  auto row = [&](int i) -> int64_t {  // of index i, or -1
    const int id = table[i / p.block_size];
    if (id < 0 || (int64_t)id >= p.num_blocks) return -1;
    return (((int64_t)id * p.block_size + i % p.block_size) * p.num_kv_heads + g) * row_words;
  };
  const int moves = fillers + e.recent;
  const int x = x0 + threadIdx.x % width, lane = threadIdx.x / width, step = blockDim.x / width;
  const bool in = x < row_words && lane < step;
  constexpr int U = 8;  // rows in flight per thread
  for (int b = 0; b < moves; b += U * step) {
    T v[U];
    int64_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * step + lane;
      to[u] = -1;
      if (in && i < moves) {
        const int k = i - fillers;
        const int64_t src = row(k < 0 ? list[2 + i] : e.n - e.recent + k);
        const int64_t dst = row(k < 0 ? list[2 + p.moves_len + i] : e.to - e.recent + k);
        if (src >= 0 && dst >= 0) {
          v[u] = pool[src + x];
          to[u] = dst + x;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0) pool[to[u]] = v[u];
    __syncthreads();
  }
}

template <typename T>
cudaError_t move_as(const EvictParams& p, cudaStream_t stream) {
  const int row_words = (int)(p.row_bytes / sizeof(T));
  // whole rows to a CTA, up to 256 accesses
  const int width = std::min(row_words, 256), slices = (row_words + width - 1) / width;
  const dim3 grid(2 * slices + (p.key_weights ? 1 : 0), p.num_kv_heads, p.num_seqs);
  k_evict_move<T><<<grid, 256, 0, stream>>>(p, slices, width, row_words);
  return cudaGetLastError();
}

template <int NT>
cudaError_t select_as(const EvictParams& p, cudaStream_t stream) {
  const size_t smem = (size_t)((p.moves_len + 31) / 32) * 8;
  auto kern = k_evict_select<NT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(p.num_kv_heads, p.num_seqs), NT, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int64_t evict_workspace(int32_t num_seqs, int32_t num_kv_heads, int64_t max_keys) {
  return (int64_t)num_seqs * num_kv_heads * (2 * max_keys + 2) * 4;
}

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
  const cudaError_t e = p.moves_len > 4096 ? select_as<1024>(p, stream) : select_as<256>(p, stream);
  if (e != cudaSuccess) return e;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.k_blocks) | reinterpret_cast<uintptr_t>(p.v_blocks) |
                       (uintptr_t)p.row_bytes;
  if (at % 16 == 0) return move_as<uint4>(p, stream);
  if (at % 4 == 0) return move_as<uint32_t>(p, stream);
  return move_as<uint8_t>(p, stream);
}

}  // namespace pa
