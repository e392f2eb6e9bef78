// k_tree_generic.cuh -- the general kernel of tree attention and of the attention behind a window with
// first tokens (WIN): any types, head size up to 256 and block size.
//
// 32 query rows x 32 keys per step in fp32 on the FMA pipes: thread (rg = tid / 16, c = tid % 16)
// computes the scores of rows 4 rg .. 4 rg + 3 and keys c and c + 16, and dims 4c + 64i .. of the
// same rows' outputs.  It is bound by shared-memory reads (a 16-byte read takes as long as 16 of
// a warp's FMAs): 9 of them for the 64 FMAs per thread of four dims of Q K^T and one key of P V at
// head size 128, against 18 when a thread had one row, eight keys and a quarter of the dims
// (16 x 16 nodes x 4 heads over 2000 fp32 positions: 563 -> 299 us).  The arithmetic is packed, two
// fp32 to an instruction, and the loops written out by eight: 275 us, 31 TFLOP/s.
// Rows of the tiles are padded by four floats, so 16-byte reads of different rows hit different
// banks.
#pragma once

#include "k_tree.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
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
// WIN: behind a window with first tokens (k_window.cu), keys counted without the gap
template <typename TQ, typename TKV, int DP, bool WIN>
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

  TreeWalk<WIN> walk(p, blockIdx.x);
  TreeSegment sg;
  while (walk.next(p, sg)) {
    const int rows = sg.rows;
    int tok[4], pos[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      tok[k] = sg.qs + (rg + k < rows ? (sg.row0 + rg + k) / G : 0);
      pos[k] = m.window > 0 || WIN ? m.positions[tok[k]] : 0;
      if constexpr (WIN) pos[k] -= sg.gap * m.block_size;
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
        const int key = key0 + tid;
        int b = key / m.block_size;
        if (WIN && b >= sg.front) b += sg.gap;
        const int id = key < sg.n ? trow[b] : -1;
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
          x[k][i] = rg + k < rows && (WIN ? window_visible(p, pos[k], key0 + c + 16 * i)
                                          : tree_visible(p, sg, tok[k], pos[k], key0 + c + 16 * i))
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

template <typename TQ, typename TKV, int DP, bool WIN>
cudaError_t generic_as(const TreeParams& p, bool vec, cudaStream_t stream) {
  auto kern = k_tree_generic<TQ, TKV, DP, WIN>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)generic_smem<DP>());
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.grid), dim3(128), generic_smem<DP>(), stream, p, vec);
}

template <typename TQ, typename TKV, bool WIN>
cudaError_t generic_dims(const TreeParams& p, cudaStream_t stream) {
  const int D = p.m.head_dim;
  const bool vec = D % 4 == 0 && aligned(p.q, 4 * sizeof(TQ)) && aligned(p.k_blocks, 4 * sizeof(TKV)) &&
                   aligned(p.v_blocks, 4 * sizeof(TKV));
  if (D <= 64) return generic_as<TQ, TKV, 64, WIN>(p, vec, stream);
  if (D <= 128) return generic_as<TQ, TKV, 128, WIN>(p, vec, stream);
  return generic_as<TQ, TKV, 256, WIN>(p, vec, stream);
}

template <bool WIN>
cudaError_t generic_types(const TreeParams& p, pa_dtype kv, cudaStream_t stream) {
  if (p.q_bf16) {
    if (kv == PA_BF16) return generic_dims<__nv_bfloat16, __nv_bfloat16, WIN>(p, stream);
    if (kv == PA_F32) return generic_dims<__nv_bfloat16, float, WIN>(p, stream);
    return generic_dims<__nv_bfloat16, e4m3_t, WIN>(p, stream);
  }
  if (kv == PA_BF16) return generic_dims<float, __nv_bfloat16, WIN>(p, stream);
  if (kv == PA_F32) return generic_dims<float, float, WIN>(p, stream);
  return generic_dims<float, e4m3_t, WIN>(p, stream);
}

}  // namespace

}  // namespace pa
