// k_pages.cu -- pages of the K/V cache: copying blocks, moving the accepted rows of a drafted
// tree together, and the bookkeeping of forked, grown and freed sequences.
//
// Copies (k_copy_blocks, k_tree_commit).  Pure data movement, bound by memory: a block of a
// pool is contiguous (block_size * num_kv_heads * head_dim elements), a position's row is
// num_kv_heads * head_dim of them.  16-byte accesses, several in flight per thread.  Measured
// (captured graph): 4096 pairs of 32-KB blocks in both pools 76.7 us, 7.0 TB/s, 1.05 of the copy
// bandwidth; 7 pairs 1.8 us; the accepted rows of 1 tree of 24 nodes 3.3 us, of 256 of 64 5.5 us.
//
// Bookkeeping (k_pages).  A few hundred to some 10^5 integers: bound by the latency of its
// dependent loads, not by bandwidth, so one cluster of eight CTAs does a whole call in one
// launch.  Its phases are separated by cluster barriers: everything is checked, and the reference
// counts are changed, before anything else is written; an error then takes the changes of the
// counts back, so it leaves every array as it was.  No workspace is needed: the set of blocks
// whose last reference goes away is a bitmap spread over the CTAs' shared memory.  The blocks a
// call takes or gives back are numbered by prefix sums, never by the order in which atomics
// arrive, so equal inputs give equal tables and free lists.  Only the reference counts are
// changed by atomics (integer additions, whose order does not matter).  Measured (captured graph,
// fork + grow + free): 4 children of a parent 17.5 us, 256 of 16 parents 43 us; a call's six or so
// dependent loads and two or three cluster barriers are its 5.7 us, the 256 forks' (and their end's)
// 10^5 table entries and the counts of their blocks the rest, 18 us each.  Sixteen CTAs to the
// cluster measured 25.7 and 47.0 us where eight had 24.3 and 50.7 (dearer barriers, more loads in
// flight): not worth a cluster that needs a launch attribute.
//
// Lists too long for every CTA to check are checked by a kernel in front, which records what it finds
// in the device's status word.  Another stream may read and clear that word in between, so the kernel
// behind it does not rest its own bounds on it: it leaves out the entries that lie outside.
//
// These kernels write block tables and lengths that a planning kernel behind them may read
// before it waits for them (pa_varlen_forward's, launched with programmatic dependent launch),
// so none of them releases its dependents early.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {
namespace {

// ---- thread-block cluster ---------------------------------------------------------------------

constexpr int kCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Address, in the cluster's shared window, of p's counterpart in CTA `rank`.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_or(uint32_t addr, uint32_t bits) {
  uint32_t old;
  asm volatile("atom.shared::cluster.or.b32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(addr), "r"(bits)
               : "memory");
  return old;
}
__device__ __forceinline__ uint32_t peer_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A set of block ids, `words` 32-bit words of it in each CTA of the cluster.
struct BlockSet {
  uint32_t* mine;
  uint32_t words;
  __device__ __forceinline__ void clear() const {
    for (uint32_t i = threadIdx.x; i < words; i += blockDim.x) mine[i] = 0;
  }
  __device__ __forceinline__ uint32_t addr(uint32_t id) const {
    const uint32_t w = id >> 5;
    return peer_addr(mine + w % words, w / words);
  }
  __device__ __forceinline__ bool insert(uint32_t id) const {  // false: it was in the set
    return !((peer_or(addr(id), 1u << (id & 31)) >> (id & 31)) & 1u);
  }
  __device__ __forceinline__ bool has(uint32_t id) const {
    return (peer_load(addr(id)) >> (id & 31)) & 1u;
  }
};
inline uint32_t set_words(int64_t num_blocks) {
  return (uint32_t)std::max<int64_t>(1, (num_blocks + 32 * kCluster - 1) / (32 * kCluster));
}

// ---- copying blocks ---------------------------------------------------------------------------

__device__ __forceinline__ bool pair_bad(int2 pr, int64_t num_blocks) {
  return (pr.x != -1 || pr.y != -1) && (pr.x < 0 || (int64_t)pr.x >= num_blocks || pr.y < 0 ||
                                        (int64_t)pr.y >= num_blocks);
}

// Lists longer than kFusedPairs: ids inside the pool, destinations distinct, and no
// destination among the sources.
__global__ void __launch_bounds__(1024)
    k_check_pairs(const int2* __restrict__ pairs, int64_t n, int64_t num_blocks, uint32_t words,
                  int* status) {
  extern __shared__ uint32_t s_bits[];
  const BlockSet dst{s_bits, words};
  pdl_wait();
  dst.clear();
  cluster_sync();
  bool bad = false;
  const int64_t first = (int64_t)cluster_rank() * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)kCluster * blockDim.x;
  for (int64_t i = first; i < n; i += step) {
    const int2 pr = pairs[i];
    const bool b = pair_bad(pr, num_blocks);
    if (!b && pr.y >= 0) bad |= !dst.insert((uint32_t)pr.y);
    bad |= b;
  }
  cluster_sync();
  for (int64_t i = first; i < n; i += step) {
    const int2 pr = pairs[i];
    if (pr.x >= 0 && (int64_t)pr.x < num_blocks) bad |= dst.has((uint32_t)pr.x);
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) record_error(status, PA_EINVAL);
  cluster_sync();  // no CTA leaves while another may read its part of the set
}

// One CTA copies `chunk` units of one block of one pool (blockIdx.y: K, V), U units in flight
// per thread.  CHECKED: lists of up to kFusedPairs, which every CTA checks whole (a thread per
// pair against all destinations).
template <typename VEC, int U, bool CHECKED>
__global__ void __launch_bounds__(256)
    k_copy_blocks(VEC* k_blocks, VEC* v_blocks, const int2* __restrict__ pairs, int num_pairs,
                  int64_t units, int chunks, int64_t num_blocks, int* status) {
  __shared__ int s_skip;
  __shared__ int s_dst[kFusedPairs];
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) s_skip = status_set(status) ? 1 : 0;
  int2 mine = make_int2(-1, -1);
  if constexpr (CHECKED) {
    if ((int)threadIdx.x < num_pairs) mine = pairs[threadIdx.x];
    s_dst[threadIdx.x] = mine.y;
  }
  __syncthreads();
  if (s_skip) return;
  if constexpr (CHECKED) {
    bool bad = pair_bad(mine, num_blocks);
    if (mine.y >= 0)
      for (int i = 0; i < num_pairs; ++i) {
        const int d = s_dst[i];
        bad |= d == mine.x || (d == mine.y && i != (int)threadIdx.x);
      }
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(status, PA_EINVAL);
      return;
    }
  }
  const int pi = blockIdx.x / chunks;
  const int64_t at = (int64_t)(blockIdx.x % chunks) * (256 * U) + threadIdx.x;
  const int2 pr = pairs[pi];
  if (pr.x < 0 || (!CHECKED && pair_bad(pr, num_blocks))) return;
  VEC* pool = blockIdx.y ? v_blocks : k_blocks;
  const VEC* src = pool + pr.x * units;
  VEC* dst = pool + pr.y * units;
  VEC r[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (at + 256 * u < units) r[u] = src[at + 256 * u];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (at + 256 * u < units) dst[at + 256 * u] = r[u];
}

template <typename VEC, int U>
cudaError_t copy_as(void* kb, void* vb, const int32_t* pairs, int64_t n, int64_t block_bytes,
                    int64_t num_blocks, int* status, cudaStream_t stream) {
  const int64_t units = block_bytes / (int64_t)sizeof(VEC);
  const int64_t chunks = (units + 256 * U - 1) / (256 * U);
  if (n * chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(n * chunks), vb ? 2 : 1);
  const int2* pr = reinterpret_cast<const int2*>(pairs);
  if (n <= kFusedPairs)
    return launch_pdl(k_copy_blocks<VEC, U, true>, grid, dim3(256), 0, stream, (VEC*)kb, (VEC*)vb,
                      pr, (int)n, units, (int)chunks, num_blocks, status);
  return launch_pdl(k_copy_blocks<VEC, U, false>, grid, dim3(256), 0, stream, (VEC*)kb, (VEC*)vb,
                    pr, (int)n, units, (int)chunks, num_blocks, status);
}

// ---- moving accepted rows together ------------------------------------------------------------

// Entry e = (s, i) of the accepted lists: false when the call has to be refused.  from, to: the
// positions of the pool (block id * block_size + place) that it moves, when it has a node.
__device__ __forceinline__ bool accepted_ok(const int32_t* tables, const int32_t* ctx,
                                            const int32_t* accepted, const int32_t* num_accepted,
                                            int s, int i, int max_accepted, int max_blocks,
                                            int block_size, int64_t num_blocks, int64_t& from,
                                            int64_t& to) {
  const int na = num_accepted[s], c = ctx[s];
  if (na < 0 || na > max_accepted || c < 0) return false;
  if (i >= na) return true;
  const int32_t* list = accepted + (int64_t)s * max_accepted;
  const int a = list[i], before = i ? list[i - 1] : -1;
  if (a <= before || a < i) return false;  // (a < i: some entry in front does not increase)
  const int64_t p = (int64_t)c + a, q = (int64_t)c + i;
  const int64_t pb = p / block_size, qb = q / block_size;
  if (pb >= max_blocks) return false;  // (q <= p, as a >= i)
  const int32_t* row = tables + (int64_t)s * max_blocks;
  const int32_t x = row[pb], y = row[qb];
  from = (int64_t)x * block_size + (p - pb * block_size);
  to = (int64_t)y * block_size + (q - qb * block_size);
  return x >= 0 && (int64_t)x < num_blocks && y >= 0 && (int64_t)y < num_blocks;
}

constexpr int kFusedAccepted = 256;  // lists up to this many entries: every CTA checks them all

__global__ void __launch_bounds__(256)
    k_check_accepted(const int32_t* tables, const int32_t* ctx, const int32_t* accepted,
                     const int32_t* num_accepted, int num_seqs, int max_accepted, int max_blocks,
                     int block_size, int64_t num_blocks, int* status) {
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  int64_t from, to;
  const int64_t n = (int64_t)num_seqs * max_accepted;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256)
    bad |= !accepted_ok(tables, ctx, accepted, num_accepted, (int)(e / max_accepted),
                        (int)(e % max_accepted), max_accepted, max_blocks, block_size, num_blocks,
                        from, to);
  if (__syncthreads_or(bad) && threadIdx.x == 0) record_error(status, PA_EINVAL);
}

// Position ctx + i of sequence blockIdx.x gets the rows of position ctx + accepted[i].  A
// thread owns one 16-byte column of K or V (units 0 .. row - 1, then V's) and takes the rows in
// order, kRows at a time: accepted[i] >= i (the list increases), so a row it reads is never one
// that an earlier group has written.
template <typename VEC, bool CHECKED>
__global__ void __launch_bounds__(256)
    k_tree_commit(VEC* k_blocks, VEC* v_blocks, const int32_t* __restrict__ tables,
                  const int32_t* __restrict__ ctx, const int32_t* __restrict__ accepted,
                  const int32_t* __restrict__ num_accepted, int num_seqs, int max_accepted,
                  int max_blocks, int block_size, int64_t num_blocks, int64_t row, int* status) {
  constexpr int kRows = 8;
  __shared__ int s_skip;
  __shared__ int64_t s_from[kRows], s_to[kRows];
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) s_skip = status_set(status) ? 1 : 0;
  __syncthreads();
  if (s_skip) return;
  int64_t from, to;
  if constexpr (CHECKED) {
    bool bad = false;
    for (int e = threadIdx.x; e < num_seqs * max_accepted; e += 256)
      bad |= !accepted_ok(tables, ctx, accepted, num_accepted, e / max_accepted, e % max_accepted,
                          max_accepted, max_blocks, block_size, num_blocks, from, to);
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(status, PA_EINVAL);
      return;
    }
  }
  const int s = blockIdx.x, na = min(num_accepted[s], max_accepted);
  const int64_t u = (int64_t)blockIdx.y * 256 + threadIdx.x;
  VEC* pool = u < row ? k_blocks + u : v_blocks + (u - row);
  for (int i0 = 0; i0 < na; i0 += kRows) {
    const int m = min(kRows, na - i0);
    __syncthreads();  // the group before has been read
    if ((int)threadIdx.x < m) {
      const bool ok = accepted_ok(tables, ctx, accepted, num_accepted, s, i0 + threadIdx.x,
                                  max_accepted, max_blocks, block_size, num_blocks, from, to);
      s_from[threadIdx.x] = ok ? from * row : 0;  // (not ok: nothing is moved)
      s_to[threadIdx.x] = ok ? to * row : 0;
    }
    __syncthreads();
    if (u >= 2 * row) continue;
    VEC r[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < m && s_from[i] != s_to[i]) r[i] = pool[s_from[i]];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (i < m && s_from[i] != s_to[i]) pool[s_to[i]] = r[i];
  }
}

template <typename VEC>
cudaError_t commit_as(void* kb, void* vb, const int32_t* tables, const int32_t* ctx,
                      const int32_t* accepted, const int32_t* num_accepted, int S, int max_accepted,
                      int max_blocks, int64_t row_bytes, int block_size, int64_t num_blocks,
                      int* status, cudaStream_t stream) {
  const int64_t row = row_bytes / (int64_t)sizeof(VEC);
  const int64_t parts = (2 * row + 255) / 256;
  if (parts > 65535) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)S, (unsigned)parts);
  if ((int64_t)S * max_accepted <= kFusedAccepted)
    return launch_pdl(k_tree_commit<VEC, true>, grid, dim3(256), 0, stream, (VEC*)kb, (VEC*)vb,
                      tables, ctx, accepted, num_accepted, S, max_accepted, max_blocks, block_size,
                      num_blocks, row, status);
  const int64_t n = (int64_t)S * max_accepted;
  const cudaError_t e =
      launch_pdl(k_check_accepted, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1024)),
                 dim3(256), 0, stream, tables, ctx, accepted, num_accepted, S, max_accepted,
                 max_blocks, block_size, num_blocks, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_commit<VEC, false>, grid, dim3(256), 0, stream, (VEC*)kb, (VEC*)vb,
                    tables, ctx, accepted, num_accepted, S, max_accepted, max_blocks, block_size,
                    num_blocks, row, status);
}

// ---- bookkeeping ------------------------------------------------------------------------------

constexpr int kPagesThreads = 1024;
constexpr int kWarps = kPagesThreads / 32;
constexpr int kChunk = 256;  // table entries a warp takes at a time, eight per lane

struct PagesShared {
  int bad;                     // some CTA found an error (told to all)
  int totals[kCluster];        // free: blocks freed by each CTA (told to all)
  int scan[32];
  int off[kPagesThreads + 1];  // chunk offsets of this round's items
  int entries[kPagesThreads];  // table entries of the item that are walked
  int len[kPagesThreads];      // length of the row that is read
  int from[kPagesThreads];     // table row that is read
  int to[kPagesThreads];       // fork: table row that is written; else the first entry walked
  int taken[kPagesThreads];    // fork, grow: blocks taken before the item
  int refs[kPagesThreads];     // fork: the round's forks of this parent, at its first fork (else 0)
  uint32_t rows[kMaxPageRows / 32];
};

// WHAT: PAGES_FORK, PAGES_GROW or PAGES_FREE.  Items (forks, or sequences) go in rounds of up to
// 1024; a round's table entries are cut into chunks of 256, dealt to all warps of the cluster.
// What a CTA learns that all have to know is written into every CTA's shared memory before a
// cluster barrier, so no CTA reads another's and none has to wait for the others to leave.
// Reference counts are the scattered accesses (a sector each), which is what a large call takes
// its time for; a parent's are read and raised once per round, whatever its number of forks.
template <int WHAT>
__global__ void __launch_bounds__(kPagesThreads) k_pages(const PagesParams p, uint32_t words) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  PagesShared& sh = *reinterpret_cast<PagesShared*>(s_raw);
  const BlockSet gone{reinterpret_cast<uint32_t*>(s_raw + sizeof(PagesShared)), words};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  const int b = p.block_size;
  const bool single = p.count <= kPagesThreads;  // one round: it stays in shared memory
  if (tid == 0) sh.bad = 0;
  if (WHAT == PAGES_FREE) gone.clear();
  if (rank == 0)
    for (int i = tid; i < (p.num_rows + 31) / 32; i += kPagesThreads) sh.rows[i] = 0;
  cluster_arrive();  // (waited for before the first access to another CTA's shared memory)
  pdl_wait();
  const int have_free = *p.free_count;
  bool bad = have_free < 0 || (int64_t)have_free > p.num_blocks;
  // (one thread of the cluster reads the status word: another stream's call may set it meanwhile)
  if (rank == 0 && tid == 0) bad |= status_set(p.status);

  auto blocks_of = [&](int n) { return (int)(((int64_t)n + b - 1) / b); };
  auto in_pool = [&](int id) { return id >= 0 && (int64_t)id < p.num_blocks; };
  // Items r0 .. r0 + K - 1 into shared memory; returns the chunks to walk.  `taken` counts on
  // from `base` (blocks taken in earlier rounds), which is advanced.
  auto load_round = [&](int r0, int& base, bool group = false) {
    const int K = min(kPagesThreads, p.count - r0);
    int entries = 0, take = 0, row = -1, to = 0, n = 0;
    if (tid < K) {
      row = p.rows[r0 + tid];
      if (WHAT != PAGES_FREE || p.other) to = p.other[r0 + tid];
      if (row >= 0 && row < p.num_rows) {
        n = p.seq_lens[row];
        if (n < 0 || blocks_of(n) > p.max_blocks) {
          bad = true;
        } else if (WHAT == PAGES_FORK) {
          entries = blocks_of(n);
          take = n % b != 0;
        } else if (WHAT == PAGES_GROW) {
          const int want = to;
          if (want < n || blocks_of(want) > p.max_blocks) {
            bad = true;
          } else {
            entries = take = blocks_of(want) - blocks_of(n);
            to = blocks_of(n);
          }
        } else if (to < 0 || to > n) {
          bad = true;
        } else {
          entries = blocks_of(n) - blocks_of(to);
          to = blocks_of(to);
        }
      } else {
        bad = true;
      }
    }
    int chunks, took = 0, before = 0;
    const int off = block_exclusive_scan((entries + kChunk - 1) / kChunk, sh.scan, &chunks);
    if (WHAT != PAGES_FREE) before = block_exclusive_scan(take, sh.scan, &took);
    sh.off[tid] = off;
    sh.entries[tid] = entries;
    sh.len[tid] = n;
    sh.from[tid] = row;
    sh.to[tid] = to;
    sh.taken[tid] = base + before;
    if (tid == 0) sh.off[kPagesThreads] = chunks;
    base += took;
    __syncthreads();
    if (WHAT == PAGES_FORK && group) {  // forks of this parent in the round, told to the first of them
      int same = 0;
      bool first = true;
      if (tid < K)
        for (int i = 0; i < K; ++i) {
          const bool e = sh.from[i] == row;
          same += e;
          first = first && !(e && i < tid);
        }
      sh.refs[tid] = first ? same : 0;
      __syncthreads();
    }
    return chunks;
  };
  // f(item, first entry, entries) for this warp's chunks of the round
  auto walk = [&](int chunks, int K, auto&& f) {
    for (int j = rank * kWarps + warp; j < chunks; j += kCluster * kWarps) {
      int lo = 0, hi = K;  // the item that owns chunk j: the last with off <= j
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.off[mid] <= j) lo = mid; else hi = mid;
      }
      f(lo, (j - sh.off[lo]) * kChunk, sh.entries[lo]);
    }
    __syncthreads();  // the next round reuses the arrays
  };
  // Adds sign (-1: takes back) times the call's change to the reference counts of the table
  // entries it holds on to (fork: all but a partly filled last one) or lets go; `bad` when an entry
  // is not an id or its count cannot be right.  Returns the blocks that the call takes; `chunks`
  // is the last round's.
  int chunks = 0;
  auto change_refs = [&](int sign) {
    int take = 0;
    for (int r0 = 0; r0 < p.count; r0 += kPagesThreads) {
      const int K = min(kPagesThreads, p.count - r0);
      chunks = load_round(r0, take, true);
      if (r0 == 0 && sign > 0) cluster_wait();
      walk(chunks, K, [&](int it, int e0, int n) {
        const int by = WHAT == PAGES_FORK ? sh.refs[it] : -1;
        if (by == 0) return;  // the parent's first fork does it
        const bool part = WHAT == PAGES_FORK && sh.len[it] % b != 0;
        const int32_t* row = p.block_tables + (int64_t)sh.from[it] * p.max_blocks +
                             (WHAT == PAGES_FREE ? sh.to[it] : 0);
        int id[8], old[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int e = e0 + lane + 32 * u;
          id[u] = e < n ? row[e] : -1;
          if (e < n && !in_pool(id[u])) bad = true;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          old[u] = 1;
          if (!in_pool(id[u])) continue;
          if (part && e0 + lane + 32 * u == n - 1)
            old[u] = p.ref_counts[id[u]];
          else
            old[u] = atomicAdd(p.ref_counts + id[u], sign * by);
        }
        if (sign < 0) return;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          bad |= old[u] < 1;  // held without a reference, or freed more often than it is held
          if (WHAT == PAGES_FREE && old[u] == 1 && in_pool(id[u])) gone.insert((uint32_t)id[u]);
        }
      });
    }
    return take;
  };

  // ---- rows distinct (CTA 0), lengths, table entries and their counts, the blocks to take
  if (rank == 0) {
    __syncthreads();  // the bitmap is clear
    const int32_t* written = WHAT == PAGES_FORK ? p.other : p.rows;
    for (int i = tid; i < p.count; i += kPagesThreads) {
      const int row = written[i];
      if (row < 0 || row >= p.num_rows)
        bad = true;
      else
        bad |= (atomicOr(&sh.rows[row >> 5], 1u << (row & 31)) >> (row & 31)) & 1u;
    }
    if (WHAT == PAGES_FORK) {
      __syncthreads();
      for (int i = tid; i < p.count; i += kPagesThreads) {
        const int row = p.rows[i];
        if (row >= 0 && row < p.num_rows) bad |= (sh.rows[row >> 5] >> (row & 31)) & 1u;
      }
    }
  }
  int taken = 0;
  if (WHAT == PAGES_GROW) {
    for (int r0 = 0; r0 < p.count; r0 += kPagesThreads) chunks = load_round(r0, taken);
    cluster_wait();
  } else {
    taken = change_refs(1);
  }
  if (WHAT != PAGES_FREE) {
    bad |= taken > have_free;
    for (int i = rank * kPagesThreads + tid; i < taken; i += kCluster * kPagesThreads) {
      const int at = have_free - 1 - i;
      const int id = at >= 0 && (int64_t)at < p.num_blocks ? p.free_list[at] : -1;
      bad |= !in_pool(id) || p.ref_counts[id] != 0;
    }
  }
  if (__syncthreads_or(bad) && tid < kCluster) peer_or(peer_addr(&sh.bad, tid), 1u);
  cluster_sync();  // (free: every reference is dropped and the set complete)
  bool undo = *reinterpret_cast<volatile int*>(&sh.bad) != 0;
  int at = 0;
  const uint32_t per = (words + kPagesThreads - 1) / kPagesThreads;
  const uint32_t w0 = min(tid * per, words), w1 = min(w0 + per, words);
  if (WHAT == PAGES_FREE) {
    // freed ids in ascending order: this CTA's words, a contiguous run per thread
    int mine = 0;
    for (uint32_t w = w0; w < w1; ++w) mine += __popc(gone.mine[w]);
    int total;
    at = block_exclusive_scan(mine, sh.scan, &total);
    if (tid < kCluster) peer_store(peer_addr(&sh.totals[rank], tid), (uint32_t)total);
    cluster_sync();
    int before = 0, all = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
      const int t = *reinterpret_cast<volatile int*>(&sh.totals[r]);
      if (r < rank) before += t;
      all += t;
    }
    at += have_free + before;
    taken = -all;
    undo |= (int64_t)have_free + all > p.num_blocks;
  }
  if (undo) {
    if (WHAT != PAGES_GROW) change_refs(-1);
    // (an earlier error stays the recorded one)
    if (rank == 0 && tid == 0) record_error(p.status, PA_EINVAL);
    return;
  }

  // ---- write
  if (WHAT == PAGES_FREE) {
    for (uint32_t w = w0; w < w1; ++w)
      for (uint32_t m = gone.mine[w]; m; m &= m - 1)
        p.free_list[at++] = (int)(((uint32_t)rank * words + w) * 32 + __ffs(m) - 1);
  } else {
    int base = 0;
    for (int r0 = 0; r0 < p.count; r0 += kPagesThreads) {
      const int K = min(kPagesThreads, p.count - r0);
      if (!single) chunks = load_round(r0, base);
      walk(chunks, K, [&](int it, int e0, int n) {
        const int64_t row = (int64_t)sh.from[it] * p.max_blocks;
        const bool part = WHAT == PAGES_FORK && sh.len[it] % b != 0;
        int id[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int e = e0 + lane + 32 * u;
          if (e >= n) continue;
          id[u] = WHAT == PAGES_GROW ? p.free_list[have_free - 1 - sh.taken[it] - e]
                                     : p.block_tables[row + e];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int e = e0 + lane + 32 * u;
          if (e >= n) continue;
          if (WHAT == PAGES_GROW) {
            p.block_tables[row + sh.to[it] + e] = id[u];
            p.ref_counts[id[u]] = 1;
          } else {
            int page = id[u];
            if (part && e == n - 1) {  // partly filled: a new page
              page = p.free_list[have_free - 1 - sh.taken[it]];
              p.ref_counts[page] = 1;
              p.block_pairs[2 * (r0 + it)] = id[u];
              p.block_pairs[2 * (r0 + it) + 1] = page;
            }
            p.block_tables[(int64_t)sh.to[it] * p.max_blocks + e] = page;
          }
        }
      });
    }
    if (!single) cluster_sync();  // every CTA has read the lengths
  }
  // lengths, and pairs of forks of whole blocks (which copy nothing)
  for (int i = rank * kPagesThreads + tid; i < p.count; i += kCluster * kPagesThreads) {
    if (WHAT == PAGES_FORK) {
      const int n = single ? sh.len[i] : p.seq_lens[p.rows[i]];
      if (n % b == 0) p.block_pairs[2 * i] = p.block_pairs[2 * i + 1] = -1;
      p.seq_lens[p.other[i]] = n;
    }
    if (WHAT == PAGES_GROW) p.seq_lens[p.rows[i]] = p.other[i];
    if (WHAT == PAGES_FREE) p.seq_lens[p.rows[i]] = p.other ? p.other[i] : 0;
  }
  if (rank == 0 && tid == 0) *p.free_count = have_free - taken;
}

template <typename Kern, typename... Args>
cudaError_t launch_cluster(Kern kern, size_t smem, cudaStream_t stream, Args... args) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kPagesThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_copy_blocks(void* kb, void* vb, const int32_t* pairs, int64_t n,
                               int64_t block_bytes, int64_t num_blocks, int* status, int num_sms,
                               cudaStream_t stream) {
  if (n > kFusedPairs) {
    const uint32_t words = set_words(num_blocks);
    const cudaError_t e =
        launch_cluster(k_check_pairs, words * 4, stream, reinterpret_cast<const int2*>(pairs), n,
                       num_blocks, words, status);
    if (e != cudaSuccess) return e;
  }
  if (block_bytes % 16 == 0 && aligned(kb, 16) && (!vb || aligned(vb, 16))) {
    // four 16-byte units per thread once that still gives every SM a few CTAs
    if (n * 2 * block_bytes >= 16384 * 4 * (int64_t)num_sms)
      return copy_as<uint4, 4>(kb, vb, pairs, n, block_bytes, num_blocks, status, stream);
    return copy_as<uint4, 1>(kb, vb, pairs, n, block_bytes, num_blocks, status, stream);
  }
  if (block_bytes % 4 == 0 && aligned(kb, 4) && (!vb || aligned(vb, 4)))
    return copy_as<uint32_t, 4>(kb, vb, pairs, n, block_bytes, num_blocks, status, stream);
  return copy_as<uint8_t, 4>(kb, vb, pairs, n, block_bytes, num_blocks, status, stream);
}

cudaError_t launch_tree_commit(void* kb, void* vb, const int32_t* tables, const int32_t* ctx,
                               const int32_t* accepted, const int32_t* num_accepted, int32_t S,
                               int32_t max_accepted, int32_t max_blocks, int64_t row_bytes,
                               int32_t block_size, int64_t num_blocks, int* status,
                               cudaStream_t stream) {
  if (row_bytes % 16 == 0 && aligned(kb, 16) && aligned(vb, 16))
    return commit_as<uint4>(kb, vb, tables, ctx, accepted, num_accepted, S, max_accepted,
                            max_blocks, row_bytes, block_size, num_blocks, status, stream);
  if (row_bytes % 4 == 0 && aligned(kb, 4) && aligned(vb, 4))
    return commit_as<uint32_t>(kb, vb, tables, ctx, accepted, num_accepted, S, max_accepted,
                               max_blocks, row_bytes, block_size, num_blocks, status, stream);
  return commit_as<uint8_t>(kb, vb, tables, ctx, accepted, num_accepted, S, max_accepted,
                            max_blocks, row_bytes, block_size, num_blocks, status, stream);
}

cudaError_t launch_pages(int what, const PagesParams& p, cudaStream_t stream) {
  const uint32_t words = what == PAGES_FREE ? set_words(p.num_blocks) : 1;
  const size_t smem = sizeof(PagesShared) + (size_t)words * 4;
  if (what == PAGES_FORK) return launch_cluster(k_pages<PAGES_FORK>, smem, stream, p, words);
  if (what == PAGES_GROW) return launch_cluster(k_pages<PAGES_GROW>, smem, stream, p, words);
  return launch_cluster(k_pages<PAGES_FREE>, smem, stream, p, words);
}

}  // namespace pa
