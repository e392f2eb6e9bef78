// k_evict.cu -- eviction from the paged cache by accumulated attention weight.
//
// Of a sequence's n keys a kv head keeps `new`: the first f, the last r and, of those between, the m =
// new - f - r with the largest weights (ties: the lowest index).  The places [f, new - r) hold m keys,
// too: those of the m that lie there stay, the others fill the places that became free, in ascending
// order, and the last r rows move up behind them.  So a cache that is cut by a few keys moves its
// recent rows and a few others, not everything behind the first evicted key.
//
// k_evict_check looks at all metadata.  Beside it k_evict, a CTA (or a small cluster) for each (sequence,
// kv head), already selects; it waits for the check before it writes, and bounds its own indices.  All go by
// the check's answer, which lies in the workspace: the status word may change under the call (another stream
// records an error, or clears one), and half of a cache that is cut in place could not be repaired.
//
// Selection.  The m-th largest weight by histograms over 11, 11 and 10 bits of its order-preserving integer
// form (the first covers exponent and two bits of the fraction, so its bins seldom collide), or, as soon
// as a bin holds 128 keys at most, by comparing each of these with all; then two
// bitmaps, of the larger keys and of the equal ones, whose prefix sums number the places and the keys that
// fill them.  (Bisection, two bits a step, took 2.6 times as many instructions and bound the selection.)
//
// Moves.  Pure data movement, bound by memory.  A sequence's moves in list order (the fillers, then the
// recent rows, ascending) never write a row that a later one reads, so a CTA that moves its part of every
// row needs only to have read a batch of rows before it writes the batch; it reads several batches ahead,
// asynchronously, into shared memory.  The CTAs of a cluster take parts of the rows (of K's and V's
// together), each for itself: there is no order between them but that the weights are moved when all have
// read them.
//
// What bounds it: memory, with rows of 256 bytes read and written in places of their own at 0.81 of the copy rate
// (half of 64 prompts of 2048 to 8192 keys, 758 MB with the weights, 138 us, of which the first 16 select), of
// 128 bytes at 0.77 (256 sequences cut by 2 %, e4m3, 571 MB, 109 us); one sequence a chain of latencies (metadata,
// weights, histogram, places, rows: 9.7 us).  The form for more than 8192 keys reads the weights again in each pass,
// one CTA to an SM: 16 prompts of 16384 keys cut to half 154 us for 85; tables and weights of 16384 columns alone
// make the 256 sequences take it, and 217 us.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBins = 2048;   // of the histogram
constexpr int kMoves = 1024;  // whose places are looked up at a time
constexpr int kNearKeys = 8192;  // of a sequence up to which the list lies in shared memory

// Larger weights have larger keys (none is 0); both zeros the same, NaN the largest.
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
// Whether the sequence's numbers cannot be used as indices.
__device__ __forceinline__ bool evict_bad(const EvictParams& p, const Plan& e) {
  return e.n < 0 || e.to < 0 || ((int64_t)e.n + p.block_size - 1) / p.block_size > p.max_blocks ||
         (p.key_weights && e.n > p.weights_len);
}

// A warp per 256 table entries of a sequence.  Each block's answer goes to verdict[block]; the first block's
// says as well whether an error was recorded before the call.
__global__ void __launch_bounds__(256) k_evict_check(const EvictParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warps = gridDim.x * 8;
  const int per = (p.max_blocks + 255) / 256 + 1;  // (one at least)
  const int64_t chunks = (int64_t)p.num_seqs * per;
  bool bad = false;
  const bool before = blockIdx.x == 0 && threadIdx.x == 0 && status_set(p.status);
  for (int64_t c = blockIdx.x * 8 + (threadIdx.x >> 5); c < chunks; c += warps) {
    const int s = (int)(c / per), e0 = (int)(c % per) * 256;
    const Plan e = evict_plan(p, s);
    if (evict_bad(p, e)) {
      bad = true;
      continue;
    }
    if (e.to >= e.n) continue;
    const int need = (e.n + p.block_size - 1) / p.block_size;
    const int32_t* row = p.block_tables + (int64_t)s * p.max_blocks;
    int id[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) id[u] = e0 + lane + 32 * u < need ? row[e0 + lane + 32 * u] : 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) bad |= id[u] < 0 || (int64_t)id[u] >= p.num_blocks;
  }
  if (__any_sync(kFull, bad) && lane == 0) record_error(p.status, PA_EINVAL);
  const int stop = __syncthreads_or(bad || before);
  if (threadIdx.x == 0) p.verdict[blockIdx.x] = stop;
}

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A word from global to the thread's own place in shared memory (4 bytes or more: asynchronously).
template <typename T>
__device__ __forceinline__ void copy_async(T* dst, const T* src) {
  if constexpr (sizeof(T) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else if constexpr (sizeof(T) == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    *dst = *src;
}

// CTAs of an SM, and batches of rows (a word of each thread) on their way or landed: what shared memory holds.
// (256 sequences of 1030 to 1060 keys, e4m3: 3 batches 133 us, 4 125, 5 118, 6 116, 7 114, 10 119; half of 64 prompts
// by 512 threads: 3 159, 4 153, 6, three CTAs still, 152, 8 147; through registers, two rows a thread in two
// batches, 128 and 148.)
constexpr int per_sm(int nt) { return nt == 1024 ? 1 : nt == 512 ? 2 : 5; }
constexpr int stages(int nt) { return nt == 1024 ? 4 : nt == 512 ? 8 : 7; }

// E > 0: sequences of at most NT * E keys; a thread keeps the ordered forms of E weights in registers, and
// the list of fillers (from, to) lies in shared memory.  E = 0: weights are read again in every pass, and
// the list lies in the workspace, written by the cluster's first CTA.
template <typename T, int NT, int E>
__global__ void __launch_bounds__(NT, per_sm(NT))
    k_evict(const EvictParams p, int cluster, int row_words, int part_words, int ordered, int ring_at) {
  extern __shared__ __align__(16) uint8_t s_mem[];
  __shared__ __align__(16) int s_work[kBins];  // histogram; then the moves' places, kMoves int2
  static_assert(kMoves * 8 <= kBins * 4, "places");
  __shared__ int s_warp[32];
  __shared__ int3 s_found;  // bin, keys in larger ones, keys in it
  __shared__ int s_left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, g = blockIdx.x / cluster;
  int s = blockIdx.y;
  if (ordered) {  // the longest sequences come first, to a 64th of the most keys; those that are not cut last
    const int n = tid < p.num_seqs ? p.seq_lens[tid] : 0;
    const bool cut = tid < p.num_seqs && p.new_lens[tid] < n;
    const int bin = !cut ? 64 : 63 - (int)(min((int64_t)max(n, 0), p.moves_len) * 63 / max(p.moves_len, (int64_t)1));
    int total;
    if (tid <= 64) s_work[tid] = 0;
    __syncthreads();
    if (tid < p.num_seqs) atomicAdd(&s_work[bin], 1);
    __syncthreads();
    const int here = tid <= 64 ? s_work[tid] : 0, before = block_exclusive_scan(here, s_warp, &total);
    if (before <= s && s < before + here) s_found = make_int3(tid, s - before, 0);
    __syncthreads();
    const int mine = tid < p.num_seqs && bin == s_found.x, at = block_exclusive_scan(mine, s_warp, &total);
    if (mine && at == s_found.y) s_left = tid;
    __syncthreads();
    s = s_left;
    __syncthreads();  // (the words are used again)
  }
  const int64_t unit = (int64_t)s * p.num_kv_heads + g;
  const Plan e = evict_plan(p, s);
  if (evict_bad(p, e) || e.to >= e.n) {
    pdl_wait();
    pdl_launch_dependents();
    return;
  }
  // the list: from, then to, each up to half of the keys
  uint16_t* near_list = reinterpret_cast<uint16_t*>(s_mem);
  constexpr int kNear = NT * E / 2;
  int32_t* far_list = p.moves + unit * p.moves_len;
  const int far_to = (int)(p.moves_len / 2);
  uint32_t* more = reinterpret_cast<uint32_t*>(s_mem + 4 * kNear);  // bitmaps: larger keys, then equal ones
  int fillers = 0;

  // ---- selection
  if (e.middle > 0) {
    const float* w = p.key_weights ? p.key_weights + unit * p.weights_len + e.first : nullptr;
    const int count = e.n - e.recent - e.first;  // keys between the first and the recent ones
    const int words = (count + 31) / 32;
    uint32_t* same = more + words;
    uint32_t own[E > 0 ? E : 1];
    auto key = [&](int i) { return w ? order_key(w[i]) : 0u; };
    if constexpr (E > 0) {
#pragma unroll
      for (int k = 0; k < E; ++k) own[k] = tid + k * NT < count ? key(tid + k * NT) : 0u;
    }
    auto each_key = [&](auto f) {  // (0: a key that is not there)
      if constexpr (E > 0) {
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (own[k] != 0) f(own[k]);
      } else {
#pragma unroll 4
        for (int i = tid; i < count; i += NT) f(key(i));
      }
    };
    // the middle-th largest key: the bin that holds it among the keys that agree with the bits found so far
    uint32_t at = 0;
    int need = e.middle;
#pragma unroll 1
    for (int pass = 0; w && pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      for (int i = tid; i < kBins; i += NT) s_work[i] = 0;
      if (tid == 0) s_left = 0;
      __syncthreads();
      each_key([&](uint32_t k) {
        if (pass == 0 || k >> (shift + bits) == at >> (shift + bits))
          atomicAdd(&s_work[(k >> shift) & ((1 << bits) - 1)], 1);
      });
      __syncthreads();
      constexpr int kPer = kBins / NT;  // bins of a thread, from the highest down
      int sum = 0, total;
#pragma unroll
      for (int k = 0; k < kPer; ++k) sum += s_work[kBins - 1 - (tid * kPer + k)];
      int before = block_exclusive_scan(sum, s_warp, &total);
      if (before < need && need <= before + sum) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int bin = kBins - 1 - (tid * kPer + k), n = s_work[bin];
          if (before < need && need <= before + n) s_found = make_int3(bin, before, n);
          before += n;
        }
      }
      __syncthreads();
      at |= (uint32_t)s_found.x << shift;
      need -= s_found.y;
      const int in = s_found.z;
      if (need == in) break;  // all of the bin's keys are taken
      if (in <= min(NT, 128)) {
        // few are left: each is compared with all others
        each_key([&](uint32_t k) {
          if (k >> shift == at >> shift) s_work[atomicAdd(&s_left, 1)] = (int)k;
        });
        __syncthreads();
        if (tid < in) {
          const uint32_t mine = (uint32_t)s_work[tid];
          int larger = 0, equal = 0;
#pragma unroll 4
          for (int i = 0; i < in; ++i) {
            larger += (uint32_t)s_work[i] > mine;
            equal += (uint32_t)s_work[i] == mine;
          }
          if (larger < need && need <= larger + equal) s_found.x = (int)mine;
        }
        __syncthreads();
        at = (uint32_t)s_found.x;
        break;
      }
      __syncthreads();
    }
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
    int all_larger, total;
    block_exclusive_scan(larger, s_warp, &all_larger);
    int ties = e.middle - all_larger - block_exclusive_scan(equal, s_warp, &total);  // left for this thread
    int holes = 0, mine = 0;
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
      const int in = e.middle - 32 * i;  // bits below it are places that stay
      const uint32_t front = in >= 32 ? kFull : in <= 0 ? 0u : (1u << in) - 1u;
      more[i] = kept & ~front;  // fillers
      same[i] = ~kept & front;  // holes
      mine += __popc(more[i]);
      holes += __popc(same[i]);
    }
    int f0 = block_exclusive_scan(mine, s_warp, &fillers);
    int h0 = block_exclusive_scan(holes, s_warp, &total);
    if constexpr (E > 0) {
      // a warp to a word, a lane to a key (a thread that wrote its word's list key by key took 2 us)
      int2* starts = reinterpret_cast<int2*>(s_work);
      static_assert(NT * E / 32 * 8 <= kBins * 4, "starts");
      for (int i = w0; i < w1; ++i) {
        starts[i] = make_int2(f0, h0);
        f0 += __popc(more[i]);
        h0 += __popc(same[i]);
      }
      __syncthreads();
      const uint32_t below = (1u << lane) - 1u;
      for (int i = warp; i < words; i += NT / 32) {
        const uint32_t b = more[i], c = same[i];
        const int2 at = starts[i];
        const uint16_t key = (uint16_t)(e.first + 32 * i + lane);
        if (b >> lane & 1u) near_list[at.x + __popc(b & below)] = key;
        if (c >> lane & 1u) near_list[kNear + at.y + __popc(c & below)] = key;
      }
    } else if (rank == 0) {
      for (int i = w0; i < w1; ++i) {
        const int at0 = e.first + 32 * i - 1;
        for (uint32_t b = more[i]; b; b &= b - 1, ++f0) far_list[f0] = at0 + __ffs(b);
        for (uint32_t b = same[i]; b; b &= b - 1, ++h0) far_list[far_to + h0] = at0 + __ffs(b);
      }
    }
    __syncthreads();
  }
  if (cluster > 1) {  // every CTA has read the weights, the list is there
    cluster_arrive();
    cluster_wait();
  }

  // ---- moves, once the whole batch has been checked
  pdl_wait();
  pdl_launch_dependents();
  if (__syncthreads_or(tid < p.checkers && __ldcg(p.verdict + tid) != 0)) return;
  auto from = [&](int i) {  // of move i
    const int k = i - fillers;
    if (k >= 0) return e.n - e.recent + k;
    if constexpr (E > 0) return (int)near_list[i]; else return __ldcg(far_list + i);
  };
  auto to = [&](int i) {
    const int k = i - fillers;
    if (k >= 0) return e.to - e.recent + k;
    if constexpr (E > 0) return (int)near_list[kNear + i]; else return __ldcg(far_list + far_to + i);
  };
  const int moves = fillers + e.recent;
  if (p.key_weights && rank == cluster - 1) {
    float* w = p.key_weights + unit * p.weights_len;
    for (int b = 0; b < moves; b += 4 * NT) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = b + u * NT + tid;
        if (i < moves) v[u] = w[from(i)];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = b + u * NT + tid;
        if (i < moves) w[to(i)] = v[u];
      }
      __syncthreads();
    }
    for (int i = e.to + tid; i < e.n; i += NT) w[i] = 0.f;
  }
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
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
  constexpr int D = stages(NT);
  T* ring = reinterpret_cast<T*>(s_mem + ring_at);  // [stage][thread]: what the thread itself reads and writes
  int2* places = reinterpret_cast<int2*>(s_work);  // slots (from, to); to -1: nothing is moved
  const int64_t stride = (int64_t)p.num_kv_heads * row_words;
  // this CTA's words of a row of K and of V laid end to end, up to NT at a time
  const int x_end = min(2 * row_words, (rank + 1) * part_words);
  for (int x0 = rank * part_words; x0 < x_end; x0 += NT) {
    const int width = min(NT, x_end - x0), step = NT / width;  // rows of a batch
    const int x = x0 + tid % width, row = tid / width;
    T* mine = x < row_words ? static_cast<T*>(p.k_blocks) + (int64_t)g * row_words + x
                            : static_cast<T*>(p.v_blocks) + (int64_t)g * row_words + (x - row_words);
    for (int base = 0; base < moves; base += kMoves) {
      const int here = min(kMoves, moves - base), batches = (here + step - 1) / step;
      __syncthreads();  // the places before (or the histogram) have been used
      for (int i = tid; i < here; i += NT) {
        int2 a;
        a.x = slot(from(base + i));
        a.y = a.x >= 0 ? slot(to(base + i)) : -1;
        places[i] = a;
      }
      __syncthreads();
      auto place = [&](int batch) {
        const int i = batch * step + row;
        return row < step && i < here ? places[i] : make_int2(-1, -1);
      };
      auto read = [&](int batch) {
        const int2 a = place(batch);
        if (a.y >= 0) copy_async(ring + batch % D * NT + tid, mine + a.x * stride);
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int i = 0; i < D - 1; ++i) read(i);
      for (int i = 0; i < batches; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory");
        __syncthreads();  // batch i has been read by all
        const int2 a = place(i);
        if (a.y >= 0) mine[a.y * stride] = ring[i % D * NT + tid];
        read(i + D - 1);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  }
}

template <typename T, int NT, int E>
cudaError_t evict_as(const EvictParams& p, int cluster, int num_sms, cudaStream_t stream) {
  const int row_words = (int)(p.row_bytes / sizeof(T));
  const int part = (2 * row_words + cluster - 1) / cluster;
  const int ring_at = (int)((2 * NT * E + (p.moves_len + 31) / 32 * 8 + 15) / 16 * 16);
  const int smem = ring_at + stages(NT) * NT * (int)sizeof(T);
  auto kern = k_evict<T, NT, E>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster * p.num_kv_heads, p.num_seqs);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // longest first where the last of few waves of CTAs is not filled, so that it is of short sequences (half of 64
  // prompts of 2048 to 8192, 512 units for 304 places, 156 -> 145 us; of 80 203 -> 197; of 128, 3.4 waves, 286
  // and 290; of 24 of 9000 to 30000 290 -> 228; 256 sequences of equal length 1.5 us more)
  const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads, resident = num_sms * per_sm(NT);
  const int ordered = cluster == 1 && units > resident && 2 * units < 5 * resident && p.num_seqs <= NT;
  return cudaLaunchKernelEx(&cfg, kern, p, cluster, row_words, part, ordered, ring_at);
}

template <typename T>
cudaError_t evict_keys(const EvictParams& p, int cluster, int num_sms, cudaStream_t stream) {
  const int64_t keys = p.moves_len;  // at most
  if (keys <= 2048) return evict_as<T, 256, 8>(p, cluster, num_sms, stream);
  if (keys <= kNearKeys) return evict_as<T, 512, kNearKeys / 512>(p, cluster, num_sms, stream);
  return evict_as<T, 1024, 0>(p, cluster, num_sms, stream);
}

}  // namespace

int64_t evict_workspace(int32_t num_seqs, int32_t num_kv_heads, int64_t max_keys) {
  return kEvictVerdict + (max_keys > kNearKeys ? (int64_t)num_seqs * num_kv_heads * max_keys * 4 : 0);
}

cudaError_t launch_evict(EvictParams p, int num_sms, cudaStream_t stream) {
  const int64_t chunks = (int64_t)p.num_seqs * ((p.max_blocks + 255) / 256 + 1);
  p.checkers = (int)std::min<int64_t>((chunks + 7) / 8, 64);
  static_assert(kEvictVerdict >= 64 * 4, "verdicts");
  const cudaError_t e = launch_pdl(k_evict_check, dim3(p.checkers), dim3(256), 0, stream, p);
  if (e != cudaSuccess) return e;
  // few units: each to as many CTAs as are resident at once, which all select
  const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads;
  int cluster = 8;
  while (cluster > 1 && units * cluster > 2 * num_sms) cluster /= 2;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.k_blocks) | reinterpret_cast<uintptr_t>(p.v_blocks) |
                       (uintptr_t)p.row_bytes;
  if (at % 16 == 0) return evict_keys<uint4>(p, cluster, num_sms, stream);
  if (at % 4 == 0) return evict_keys<uint32_t>(p, cluster, num_sms, stream);
  return evict_keys<uint8_t>(p, cluster, num_sms, stream);
}

}  // namespace pa
