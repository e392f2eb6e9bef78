// k_rope.cu -- rotary positions applied to the new tokens' queries and keys, with the keys and
// values scattered into the paged pools in the same pass.
//
// Math.  Pair i of a head's first R = rotary_dim elements is (x_i, x_{R/2+i}) in the half
// layout and (x_{2i}, x_{2i+1}) interleaved; at position p it is turned by the angle
// p * inv_freq[i] and multiplied by the attention factor f (long-context scalings):
//   y_a = f (x_a cos - x_b sin),  y_b = f (x_a sin + x_b cos)
// and elements past R are copied.  Everything is computed in fp32 and rounded once.
//
// Angles.  In fp32 the product p * inv_freq is off by up to 2^-24 p radians: 0.06 at a million
// positions.  Here each frequency becomes the fraction of a turn per position as a 64-bit
// fixed-point number (turn_per_position, once per CTA), and a position's angle is one 64-bit integer
// product that wraps at whole turns, exactly: off by less than 2^-33 turns at the farthest.  Its top
// 32 bits go to sincospif as a signed fraction of half a turn (off by at most 2^-25 half turns; the
// dropped bits are less than 2^-31).
//
// What bounds it: memory.  Every element of q, k and v is read once and written once, 16 bytes
// at a time; a rotated half-layout unit is the two 16-byte chunks of its pairs, so a thread
// has both sides of each pair in registers.  A CTA takes TOK tokens; their angles are computed
// once into shared memory and serve all H + Hkv heads.  The items of a token (rotated units, copied
// chunks and value chunks) are dealt to the threads in memory order; a thread takes its item through
// the CTA's tokens, four in flight.  Measured: 16381 tokens (32 + 2 x 8 heads of 128 out of one
// fused product, half of each rotated, e4m3 pools) 65 us, 5.7 TB/s, 0.85 of the copy bandwidth; 64
// tokens of the same heads 3.0 us in a captured graph, which is the launch and two dependent loads.
#include <algorithm>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kCheckedTokens = 2048;  // up to here every CTA checks all slots itself
constexpr int kMaxHalf = 128;         // rotary_dim / 2, at most
constexpr int kMaxTokens = 8;         // tokens of a CTA, at most

// Division of 0 <= n < 2^31 by a fixed d >= 1: with l = ceil(log2 d) and
// m = ceil(2^(31 + l) / d) < 2^32, floor(n m / 2^(31 + l)) is the quotient (the error of m adds
// less than n / 2^(31 + l) < 2^-l <= 1 / d).
struct FastDiv {
  uint32_t d, m, l;
  explicit FastDiv(uint32_t x) : d(x), m(0), l(0) {
    while ((1ull << l) < x) ++l;
    m = (uint32_t)(((1ull << (31 + l)) + x - 1) / x);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> (31 + l));
  }
};

// The fraction of a turn that w radians are, times 2^64 and rounded down (towards zero for w < 0):
// w = m 2^e with an integer m < 2^53, so it is bits 64 - e .. 127 - e of m times C = 2^128 / (2 pi).
// (In fp64 even a product's one rounding is 2^-53 of w, which far positions multiply; and the integer
// products are the faster ones here.)  |w| < 2^53, else 0.
__device__ __forceinline__ uint64_t turn_per_position(double w) {
  constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // C
  const uint64_t bits = (uint64_t)__double_as_longlong(w);
  const int field = (int)(bits >> 52) & 0x7ff;
  const uint64_t m = (bits & 0xfffffffffffffull) | (field ? 1ull << 52 : 0ull);
  const int s = 1075 - max(field, 1);  // -e: from the product's second word on
  const uint64_t low = __umul64hi(m, kLow), mid = m * kHigh + low;
  const uint64_t high = __umul64hi(m, kHigh) + (mid < low ? 1 : 0);
  uint64_t t = 0;
  if (s >= 0 && s < 128) t = s >= 64 ? high >> (s - 64) : s ? mid >> s | high << (64 - s) : mid;
  return bits >> 63 ? 0 - t : t;
}

struct Geometry {
  uint32_t per_token;  // items of one token
  FastDiv per_head;   // items of a rotated head: rotated units, then copied chunks
  FastDiv per_v;      // value chunks of a kv head
  int rot_units;      // rotated units of a head
};

// one chunk of VE elements: as it lies in memory, and its values in fp32
template <typename TS, int VE>
struct Chunk {
  static constexpr bool kWide = sizeof(TS) * VE == 16;
  uint32_t w[kWide ? 4 : VE];
  __device__ __forceinline__ void load(const TS* p) {
    if constexpr (kWide) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) w[i] = __float_as_uint(to_f32(p[i]));
    }
  }
  __device__ __forceinline__ void values(float (&x)[VE]) const {
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if constexpr (kWide && sizeof(TS) == 2)
        x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      else
        x[i] = __uint_as_float(w[i]);
    }
  }
};

// VE fp32 values in pool type DST (a pa_dtype), rounded to nearest even
template <int DST, int VE>
__device__ __forceinline__ void store_chunk(void* base, int64_t at, const float (&x)[VE]) {
  if constexpr (DST == PA_FP8_E4M3) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    if constexpr (VE % 4 == 0) {
      uint32_t w[VE / 4];
#pragma unroll
      for (int i = 0; i < VE / 4; ++i)
        w[i] = f32x2_to_e4m3x2(x[4 * i], x[4 * i + 1]) |
               ((uint32_t)f32x2_to_e4m3x2(x[4 * i + 2], x[4 * i + 3]) << 16);
      if constexpr (VE == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) p[i] = (uint8_t)(f32x2_to_e4m3x2(x[i], 0.f) & 0xffu);
    }
  } else if constexpr (DST == PA_BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + at;
    if constexpr (VE == 8) {
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
    } else if constexpr (VE == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
  } else {
    float* p = static_cast<float*>(base) + at;
    if constexpr (VE % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VE; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) p[i] = x[i];
    }
  }
}

// TS: type of q, k, v; DST: the pools' pa_dtype; VE: elements per chunk (16 bytes of TS, or 1 /
// 2 when shapes, strides or addresses do not allow that); IL: interleaved pairs; CHECKED: this
// kernel checks the slots (else k_validate_slots ran before).
template <typename TS, int DST, int VE, bool IL, bool CHECKED>
__global__ void __launch_bounds__(kThreads)
    k_rope_and_cache(const RopeParams p, const Geometry g, const int tok_per_cta) {
  static_assert(!IL || VE % 2 == 0, "interleaved pairs stay inside a chunk");
  __shared__ int s_skip;
  __shared__ uint64_t s_turn[kMaxHalf];
  __shared__ int32_t s_slot[kMaxTokens];
  extern __shared__ __align__(16) float s_trig[];  // [tok][half] cos, then sin
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) s_skip = status_set(p.status) ? 1 : 0;
  const int half = p.rotary_dim >> 1;
  for (int i = threadIdx.x; i < half; i += kThreads) s_turn[i] = turn_per_position(p.inv_freq[i]);
  __syncthreads();
  if (s_skip) return;
  if constexpr (CHECKED) {
    bool bad = false;
    for (int64_t t = threadIdx.x; t < p.num_tokens; t += kThreads) {
      const int32_t s = p.slots[t];
      bad |= s < 0 || (int64_t)s >= p.num_slots;
    }
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(p.status, PA_EINVAL);
      return;
    }
  }
  const int64_t t0 = (int64_t)blockIdx.x * tok_per_cta;
  const int ntok = (int)min((int64_t)tok_per_cta, p.num_tokens - t0);
  if ((int)threadIdx.x < ntok) {
    const int32_t s = p.slots[t0 + threadIdx.x];
    // (not CHECKED: the status may have been cleared since the slots were found bad)
    s_slot[threadIdx.x] = CHECKED || (s >= 0 && (int64_t)s < p.num_slots) ? s : -1;
  }
  float* s_cos = s_trig;
  float* s_sin = s_trig + tok_per_cta * half;
  for (int a = threadIdx.x; a < ntok * half; a += kThreads) {
    const int tk = a / half, i = a - tk * half;
    const uint64_t turn = (uint64_t)(int64_t)p.positions[t0 + tk] * s_turn[i];
    float sn, cs;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &sn, &cs);
    s_cos[a] = cs * p.attn_factor;
    s_sin[a] = sn * p.attn_factor;
  }
  __syncthreads();

  // an item's place in a token's rows is the same for all tokens of the CTA: worked out once, then
  // the tokens go through it U at a time
  const int H = p.q ? p.num_heads : 0, D = p.head_dim, R = p.rotary_dim;
  const int rot_items = (H + p.num_kv_heads) * (int)g.per_head.d;
  constexpr int U = 4;
  for (int it = blockIdx.y * kThreads + threadIdx.x; it < (int)g.per_token;
       it += gridDim.y * kThreads) {
    int head, off;
    bool rot = false;
    const TS* src;
    int64_t stride;
    if (it < rot_items) {
      head = (int)g.per_head.div((uint32_t)it);
      const int e = it - head * (int)g.per_head.d;
      rot = e < g.rot_units;
      off = rot ? e * VE : R + (e - g.rot_units) * VE;
      const bool is_q = head < H;
      src = is_q ? static_cast<const TS*>(p.q) + (int64_t)head * D
                 : static_cast<const TS*>(p.k) + (int64_t)(head - H) * D;
      stride = is_q ? p.q_stride : p.k_stride;
    } else {
      const int hv = (int)g.per_v.div((uint32_t)(it - rot_items));
      off = (it - rot_items - hv * (int)g.per_v.d) * VE;
      src = static_cast<const TS*>(p.v) + (int64_t)hv * D;
      stride = p.v_stride;
      head = H + p.num_kv_heads + hv;
    }
    src += off + t0 * stride;
    const bool two = !IL && rot;
    const bool to_q = head < H, is_v = head >= H + p.num_kv_heads;
    const int hk = head - H - (is_v ? p.num_kv_heads : 0);
    float sc = 1.f, inv = 1.f;
    bool divide = false;
    if (!to_q) {
      const float* scales = is_v ? p.v_scales : p.k_scales;
      sc = scales ? __ldg(scales + hk) : is_v ? p.v_scale : p.k_scale;
      // dividing by a power of two is multiplying by its inverse, to the bit
      divide = (__float_as_uint(sc) & 0x7fffffu) != 0 || sc < 2.3283064e-10f || sc > 4294967296.f;
      inv = divide ? 1.f : 1.f / sc;
    }
    for (int k0 = 0; k0 < ntok; k0 += U) {
      Chunk<TS, VE> ra[U], rb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + u >= ntok) break;
        ra[u].load(src + (k0 + u) * stride);
        if (two) rb[u].load(src + (k0 + u) * stride + half);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tk = k0 + u;
        if (tk >= ntok) break;
        float a[VE], b[VE];
        ra[u].values(a);
        if (two) rb[u].values(b);
        if (rot) {
          const float* cs = s_cos + tk * half + (IL ? off / 2 : off);
          const float* sn = s_sin + tk * half + (IL ? off / 2 : off);
          if constexpr (IL) {
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
              const float x = a[2 * i], y = a[2 * i + 1];
              a[2 * i] = x * cs[i] - y * sn[i];
              a[2 * i + 1] = x * sn[i] + y * cs[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              const float x = a[i], y = b[i];
              a[i] = x * cs[i] - y * sn[i];
              b[i] = x * sn[i] + y * cs[i];
            }
          }
        }
        if (to_q) {
          constexpr int SRC = sizeof(TS) == 2 ? PA_BF16 : PA_F32;
          const int64_t at = (t0 + tk) * p.q_out_stride + (int64_t)head * D + off;
          store_chunk<SRC, VE>(p.q_out, at, a);
          if (two) store_chunk<SRC, VE>(p.q_out, at + half, b);
          continue;
        }
        if (!CHECKED && s_slot[tk] < 0) continue;
        if (divide) {
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            a[i] = __fdiv_rn(a[i], sc);
            if (two) b[i] = __fdiv_rn(b[i], sc);
          }
        } else {
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            a[i] *= inv;
            if (two) b[i] *= inv;
          }
        }
        const int64_t at = ((int64_t)s_slot[tk] * p.num_kv_heads + hk) * D + off;
        void* pool = is_v ? p.v_blocks : p.k_blocks;
        store_chunk<DST, VE>(pool, at, a);
        if (two) store_chunk<DST, VE>(pool, at + half, b);
      }
    }
  }
}

template <typename TS, int DST, int VE, bool IL>
cudaError_t launch_as(const RopeParams& p, int num_sms, cudaStream_t stream) {
  const int D = p.head_dim, R = p.rotary_dim;
  const int rot_units = R / (IL ? VE : 2 * VE), per_head = rot_units + (D - R) / VE;
  const int heads = (p.q ? p.num_heads : 0) + p.num_kv_heads;
  const int64_t per_token = (int64_t)heads * per_head + (int64_t)p.num_kv_heads * (D / VE);
  if (per_token > (1 << 28)) return cudaErrorInvalidValue;
  // eight tokens to a CTA when that still gives every SM four CTAs, fewer for smaller batches;
  // with one, its items are spread over several CTAs
  int tok = kMaxTokens;
  while (tok > 1 && p.num_tokens < (int64_t)tok * 4 * num_sms) tok >>= 1;
  const int64_t most = (per_token + kThreads - 1) / kThreads;
  const int64_t parts = tok > 1 ? 1 : std::min<int64_t>(most, std::max<int64_t>(1, 2 * num_sms / p.num_tokens));
  const Geometry g{(uint32_t)per_token, FastDiv((uint32_t)std::max(1, per_head)),
                   FastDiv((uint32_t)(D / VE)), rot_units};
  const dim3 grid((unsigned)((p.num_tokens + tok - 1) / tok), (unsigned)std::min<int64_t>(parts, 65535));
  const size_t smem = (size_t)tok * R * 4;
  if (p.num_tokens <= kCheckedTokens)
    return launch_pdl(k_rope_and_cache<TS, DST, VE, IL, true>, grid, dim3(kThreads), smem, stream,
                      p, g, tok);
  const cudaError_t e = launch_validate_slots(p.slots, p.num_tokens, p.num_slots, p.status, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_rope_and_cache<TS, DST, VE, IL, false>, grid, dim3(kThreads), smem, stream,
                    p, g, tok);
}

template <typename TS, int DST>
cudaError_t launch_types(const RopeParams& p, int num_sms, cudaStream_t stream) {
  constexpr int VE = 16 / (int)sizeof(TS);
  constexpr size_t kDst = DST == PA_FP8_E4M3 ? 1 : DST == PA_BF16 ? 2 : 4;
  const int D = p.head_dim, R = p.rotary_dim;
  // 16-byte chunks: whole chunks on both sides of every pair and in the copied rest, rows and
  // tensors aligned for the loads and for the pools' stores.  Anything else, be it one tensor off its
  // boundary, goes one or (interleaved) two elements at a time, q, k and v alike: 16381 tokens out of
  // a fused product one element off 141 us interleaved and 274 us in halves, for 65 and 78 in
  // chunks; 64 tokens 4.9 us for 3.1.  It is there so that odd sizes and offsets are right.
  const bool vec = D % VE == 0 && R % (p.interleaved ? VE : 2 * VE) == 0 &&
                   (p.q == nullptr || (p.q_stride % VE == 0 && p.q_out_stride % VE == 0 &&
                                       aligned(p.q, 16) && aligned(p.q_out, 16))) &&
                   p.k_stride % VE == 0 && p.v_stride % VE == 0 && aligned(p.k, 16) &&
                   aligned(p.v, 16) && aligned(p.k_blocks, std::min<size_t>(16, VE * kDst)) &&
                   aligned(p.v_blocks, std::min<size_t>(16, VE * kDst));
  if (p.interleaved) {
    if (vec) return launch_as<TS, DST, VE, true>(p, num_sms, stream);
    return D % 2 == 0 ? launch_as<TS, DST, 2, true>(p, num_sms, stream) : cudaErrorInvalidValue;
  }
  return vec ? launch_as<TS, DST, VE, false>(p, num_sms, stream)
             : launch_as<TS, DST, 1, false>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeParams& p, pa_dtype src_dtype, pa_dtype kv_dtype,
                                  int num_sms, cudaStream_t stream) {
  if (src_dtype == PA_BF16) {
    if (kv_dtype == PA_BF16) return launch_types<__nv_bfloat16, PA_BF16>(p, num_sms, stream);
    if (kv_dtype == PA_FP8_E4M3) return launch_types<__nv_bfloat16, PA_FP8_E4M3>(p, num_sms, stream);
    return launch_types<__nv_bfloat16, PA_F32>(p, num_sms, stream);
  }
  if (kv_dtype == PA_BF16) return launch_types<float, PA_BF16>(p, num_sms, stream);
  if (kv_dtype == PA_FP8_E4M3) return launch_types<float, PA_FP8_E4M3>(p, num_sms, stream);
  return launch_types<float, PA_F32>(p, num_sms, stream);
}

}  // namespace pa
