// k_key_weights.cu -- the attention weight that every cached key receives, from the queries and the
// log-sum-exps of their attention: key_weights[s, g, j] += sum over the counted tokens t that see key j
// and over the heads h of kv head g's group of exp(scale q[t, h] . K_j - lse[h, t]).
//
// The general kernel.  A CTA takes tiles of 32 keys of one (sequence, kv head) and goes over the rows
// (token, head of the group) that see them, 32 at a time, in fp32 on the FMA pipes; a key's sum stays
// with its thread, and the eight row groups' sums are added in order at the end.  One CTA owns a key,
// so nothing is added by atomics, and equal inputs give equal bits.
#include <algorithm>

#include "k_tree_generic.cuh"

namespace pa {
namespace {

template <int DP>
constexpr size_t weights_smem() {
  return (size_t)(kBM + kBN) * (DP + 4) * 4;
}

template <typename TQ, typename TKV, int DP>
__global__ void __launch_bounds__(128) k_key_weights(const TreeParams p, const bool vec) {
  constexpr int LD = DP + 4;
  constexpr int kCols = DP / 4, kStep = 128 / kCols;
  extern __shared__ __align__(16) float s_mem[];
  float* sq = s_mem;
  float* sk = sq + kBM * LD;
  __shared__ int64_t s_row[kBN];
  __shared__ float s_lse[kBM];  // of the tile's rows, log2 units
  __shared__ int s_pos[kBM];
  __shared__ float s_sum[8][kBN];
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
  int64_t before = 0;  // units of the sequences before
  for (int s = 0; s < m.num_seqs; ++s) {
    const int4 sq4 = p.seqs[2 * s];
    const int qs = sq4.x, nq = sq4.y, n = sq4.z;
    if (nq == 0) continue;
    const int counted0 = p.observed > 0 ? max(0, nq - p.observed) : 0;  // first token that counts
    const int tiles = (n + kBN - 1) / kBN;
    const int64_t units = (int64_t)tiles * m.num_kv_heads;
    int64_t u = ((int64_t)blockIdx.x - before % gridDim.x + gridDim.x) % gridDim.x;
    before += units;
    const int32_t* trow = m.block_tables + (int64_t)s * m.max_blocks;
    for (; u < units; u += gridDim.x) {
      const int kvh = (int)(u % m.num_kv_heads), key0 = (int)(u / m.num_kv_heads) * kBN;
      // keys that no counted token sees get nothing: positions do not decrease within a sequence
      const int last = m.positions[qs + nq - 1], low = m.positions[qs + counted0];
      if (key0 > last || (m.window > 0 && key0 + kBN - 1 <= low - m.window && key0 >= p.first)) continue;
      const float sl = head_scale(m.k_scales, kvh, p.scale) * kLog2e;
      __syncthreads();  // the buffers of the unit before are free
      if (tid < kBN) {
        const int key = key0 + tid, id = key < n ? trow[key / m.block_size] : -1;
        s_row[tid] = id >= 0 && (int64_t)id < m.num_blocks
                         ? ((int64_t)id * m.block_size + key % m.block_size) * m.num_kv_heads + kvh
                         : -1;
      }
      __syncthreads();
      for (int k0 = tid / kCols; k0 < kBN; k0 += kStep) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        const int64_t at = s_row[k0] * D + col;
        if (at >= 0 && col < D) a = row4<TKV>(kb + at, D - col, vec);
        *reinterpret_cast<float4*>(sk + k0 * LD + col) = a;
      }
      float sum[2] = {0.f, 0.f};
      for (int row0 = counted0 * G; row0 < nq * G; row0 += kBM) {
        const int rows = min(kBM, nq * G - row0);
        // (the same for the whole CTA)
        if (m.positions[qs + (row0 + rows - 1) / G] < key0) continue;
        if (m.window > 0 && key0 >= p.first && key0 + kBN - 1 <= m.positions[qs + row0 / G] - m.window)
          break;
        __syncthreads();  // the tile before has been used
        for (int r = tid / kCols; r < kBM; r += kStep) {
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          const int R = row0 + r;
          if (r < rows && col < D)
            a = row4<TQ>(q + ((int64_t)(qs + R / G) * m.num_heads + kvh * G + R % G) * D + col, D - col,
                         vec);
          *reinterpret_cast<float4*>(sq + r * LD + col) = a;
        }
        if (tid < kBM) {
          const int R = row0 + tid;
          const bool have = tid < rows;
          s_pos[tid] = have ? m.positions[qs + R / G] : -1;
          // (a row without a finite score, lse -inf, gives no weight)
          const float l = have ? m.lse[(int64_t)(kvh * G + R % G) * m.num_tokens + qs + R / G] : 0.f;
          s_lse[tid] = l == -INFINITY ? INFINITY : l * kLog2e;
        }
        __syncthreads();
        uint64_t x2[4][2] = {};
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
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float even, odd;
            f2_unpack(x2[k][i], even, odd);
            // (a row past the last has position -1 and sees nothing)
            if (window_visible(p, s_pos[rg + k], key0 + c + 16 * i) && s_pos[rg + k] >= 0)
              sum[i] += exp2f((even + odd) * sl - s_lse[rg + k]);
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) s_sum[tid >> 4][c + 16 * i] = sum[i];
      __syncthreads();
      if (tid < kBN && key0 + tid < n) {
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) total += s_sum[k][tid];
        float* at = p.key_weights + ((int64_t)s * m.num_kv_heads + kvh) * p.weights_len + key0 + tid;
        *at += total;
      }
    }
  }
}

template <typename TQ, typename TKV, int DP>
cudaError_t weights_as(const TreeParams& p, bool vec, cudaStream_t stream) {
  auto kern = k_key_weights<TQ, TKV, DP>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)weights_smem<DP>());
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(4 * num_sms()), dim3(128), weights_smem<DP>(), stream, p, vec);
}

template <typename TQ, typename TKV>
cudaError_t weights_dims(const TreeParams& p, cudaStream_t stream) {
  const int D = p.m.head_dim;
  const bool vec = D % 4 == 0 && aligned(p.q, 4 * sizeof(TQ)) && aligned(p.k_blocks, 4 * sizeof(TKV));
  if (D <= 64) return weights_as<TQ, TKV, 64>(p, vec, stream);
  if (D <= 128) return weights_as<TQ, TKV, 128>(p, vec, stream);
  return weights_as<TQ, TKV, 256>(p, vec, stream);
}

}  // namespace

cudaError_t launch_key_weights_generic(const TreeParams& p, pa_dtype kv, cudaStream_t stream) {
  if (p.q_bf16) {
    if (kv == PA_BF16) return weights_dims<__nv_bfloat16, __nv_bfloat16>(p, stream);
    if (kv == PA_F32) return weights_dims<__nv_bfloat16, float>(p, stream);
    return weights_dims<__nv_bfloat16, e4m3_t>(p, stream);
  }
  if (kv == PA_BF16) return weights_dims<float, __nv_bfloat16>(p, stream);
  if (kv == PA_F32) return weights_dims<float, float>(p, stream);
  return weights_dims<float, e4m3_t>(p, stream);
}

}  // namespace pa
