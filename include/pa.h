/*
 * pa.h -- batched paged attention over a block-pooled KV cache, for GB300 (sm_103a).
 *
 * C ABI of libpa.so.  Every pointer argument named *_blocks, q, k, v, out, lse, the
 * int32 metadata arrays and any workspace is a DEVICE pointer that the caller owns;
 * the library allocates no device memory.  Every call is asynchronous on `stream`
 * (0 = the legacy default stream) and returns after enqueueing its kernels.
 *
 * Stream order.  A call observes everything enqueued before it on `stream` and everything
 * after it observes the call.  The varlen calls' planning kernel is launched with
 * programmatic dependent launch and reads the metadata arrays (query_start_loc, seq_lens,
 * positions, block_tables, per-head scales, per-block factors) before the kernel ahead of it
 * on the stream has finished; it waits for that kernel before writing anything.  So the
 * metadata must not be written by a kernel of the caller's that itself releases its
 * programmatic dependents (griddepcontrol.launch_dependents) before those writes.  Copies,
 * ordinary kernels and this library's own kernels ahead of the call are all safe.
 *
 * Layouts (row-major, as the TensorSharp "ManagedPagedAttention.cs" class summary
 * states them):
 *   q, out               [num_tokens, num_heads, head_dim]
 *   k, v (new tokens)    [num_tokens, num_kv_heads, head_dim]
 *   k_blocks, v_blocks   [num_blocks, block_size, num_kv_heads, head_dim]
 *   block_tables         int32 [num_seqs, max_blocks_per_seq]: position j of sequence s
 *                        lives in row j mod block_size of block block_tables[s][j / block_size]
 *                        (tinyllm "Paged attention for decode in C", section 2.1)
 *   query_start_loc      int32 [num_seqs + 1], query_start_loc[0] = 0,
 *                        query_start_loc[num_seqs] = num_tokens
 *   seq_lens             int32 [num_seqs]: cached positions of the sequence, new tokens included
 *   positions            int32 [num_tokens]: absolute position of each token in its sequence
 *   lse                  fp32 [num_heads, num_tokens], natural log (vllm.cpp cpu_mla_prefill.cpp)
 *
 * Errors.  Argument and shape errors are returned immediately and nothing is enqueued.
 * Errors in the device-resident metadata (a block id outside the pool, a table too short,
 * an empty context, a position outside its context, a slot outside the pool) are found on
 * the device by a validation kernel that runs before any output is written: the call then
 * writes NO output, and the error is recorded in a per-device status word that
 * pa_device_status() returns.  The recorded error is sticky: until pa_device_status() reads
 * and clears it, every later call on that device also skips its writes.  A bounded wait
 * that runs out inside a kernel records PA_ETIMEOUT the same way.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes: the error classes of the tinyllm decode interface (section 4:
 * TL_EINVAL, TL_ESHAPE; section 2.6: TL_EUNSUPPORTED) plus the CUDA and timeout cases. */
typedef enum {
  PA_OK = 0,
  PA_EINVAL = 1,       /* NULL pointer, bad metadata, sizes out of range */
  PA_ESHAPE = 2,       /* num_heads % num_kv_heads != 0, non-positive dims */
  PA_EUNSUPPORTED = 3, /* dtype or shape this build does not implement */
  PA_ECUDA = 4,        /* a CUDA runtime call failed */
  PA_ETIMEOUT = 5      /* a bounded wait inside a kernel ran out */
} pa_status;

/* Element types (vllm.cpp cpu_mla_prefill.cpp LoadF/StoreF: f32 and bf16), and fp8 e4m3
 * for K/V pools only ("paged_attention_v2_pytorch.py": kv_cache_dtype "fp8" with k_scale /
 * v_scale; tinyllm "Going further": fp8 KV caches, half the bytes per token).  PA_FP8_E4M3
 * is the OCP e4m3 "fn" format: 1 sign, 4 exponent (bias 7) and 3 mantissa bits, no
 * infinities, S.1111.111 NaN, largest finite value 448.  q, out and new K/V rows are f32 or
 * bf16. */
typedef enum { PA_F32 = 0, PA_BF16 = 1, PA_FP8_E4M3 = 2 } pa_dtype;

/* Flags of pa_varlen_forward_ex. */
enum { PA_FLAG_BITWISE = 1u };

/* Library version, major * 10000 + minor * 100 + patch. */
int pa_version(void);

/* Human-readable name of a status code (static string). */
const char* pa_status_string(pa_status status);

/* Synchronises `stream`, then returns and clears this device's sticky status word
 * (PA_OK if no kernel recorded an error).  Returns PA_ECUDA if the synchronisation
 * itself fails. */
pa_status pa_device_status(cudaStream_t stream);

/*
 * pa_slot_mapping -- the physical slot of every new token.
 * slot_mapping[t] = block_tables[s][p / block_size] * block_size + p % block_size for
 * token t of sequence s at position p = positions[t] (TensorSharp class summary,
 * "slot = blockId * blockSize + offsetInBlock"; tinyllm section 2.1).
 * A token whose position lies outside its table row, or whose block id lies outside
 * [0, num_blocks), gets slot -1 and records PA_EINVAL.
 */
pa_status pa_slot_mapping(const int32_t* query_start_loc, const int32_t* positions,
                          const int32_t* block_tables, int32_t num_seqs, int64_t num_tokens,
                          int32_t max_blocks_per_seq, int32_t block_size, int64_t num_blocks,
                          int32_t* slot_mapping, cudaStream_t stream);

/*
 * pa_reshape_and_cache -- scatter the new tokens' K and V rows into the pool
 * (TensorSharp WriteKvToPagedPool): the num_kv_heads * head_dim elements of token t go to
 * block slot_mapping[t] / block_size, row slot_mapping[t] % block_size, of each pool.
 * A pure copy: bit-exact (for PA_FP8_E4M3 the new rows are e4m3 codes already; to quantise
 * f32 / bf16 rows into an fp8 pool use pa_reshape_and_cache_ex).  Every slot is checked on
 * the device before any row is written;
 * one slot outside [0, num_blocks * block_size) writes nothing and records PA_EINVAL.
 * Duplicate slots are undefined.
 */
pa_status pa_reshape_and_cache(const void* k, const void* v, void* k_blocks, void* v_blocks,
                               const int32_t* slot_mapping, int64_t num_tokens,
                               int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                               int64_t num_blocks, pa_dtype kv_dtype, cudaStream_t stream);

/*
 * pa_slot_mapping_and_cache -- pa_slot_mapping followed by pa_reshape_and_cache on the same
 * stream, as one launch when num_tokens <= 2048 and num_seqs <= 2047 (a decode step; larger
 * batches take the two launches).  Writes slot_mapping [num_tokens] (-1 for an invalid token)
 * and scatters the new K/V rows of every token into its slot.  Every token's slot is computed
 * and checked before any row is written: a token that no sequence's range
 * [query_start_loc[s], query_start_loc[s + 1]) holds, a malformed query_start_loc, a position
 * outside its table row or a block id outside [0, num_blocks) writes no row and records
 * PA_EINVAL.  Layouts and dtypes as in pa_slot_mapping and pa_reshape_and_cache (a copy, so
 * bit-exact).  Duplicate slots are undefined.
 */
pa_status pa_slot_mapping_and_cache(const void* k, const void* v, void* k_blocks, void* v_blocks,
                                    const int32_t* query_start_loc, const int32_t* positions,
                                    const int32_t* block_tables, int32_t num_seqs,
                                    int64_t num_tokens, int32_t max_blocks_per_seq,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    int64_t num_blocks, pa_dtype kv_dtype, int32_t* slot_mapping,
                                    cudaStream_t stream);

/*
 * pa_reshape_and_cache_ex -- the scatter of pa_reshape_and_cache with a conversion: new rows
 * of src_dtype (f32 or bf16) go into pools of kv_dtype (f32, bf16 or fp8 e4m3), element x of
 * K stored as x / k_scale and of V as x / v_scale, the quotient taken in fp32 (IEEE division)
 * and rounded to kv_dtype to nearest, ties to even; an fp8 store saturates to +-448
 * ("paged_attention_v2_pytorch.py": the pool holds K / k_scale, so that K = k_scale * pool).
 * k_scale and v_scale must be finite and positive (PA_EINVAL otherwise).  Slots are checked as
 * in pa_reshape_and_cache.  Same pool layout [num_blocks, block_size, num_kv_heads, head_dim].
 */
pa_status pa_reshape_and_cache_ex(const void* k, const void* v, void* k_blocks, void* v_blocks,
                                  const int32_t* slot_mapping, int64_t num_tokens,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                  int64_t num_blocks, pa_dtype src_dtype, pa_dtype kv_dtype,
                                  float k_scale, float v_scale, cudaStream_t stream);

/*
 * pa_reshape_and_cache_per_head -- pa_reshape_and_cache_ex with one dequantisation scale per
 * kv head (tinyllm "Going further": fp8 KV caches with scales per head): head g of a new row
 * is stored as x / k_scales[g] (x / v_scales[g]).  k_scales, v_scales: DEVICE arrays of
 * num_kv_heads floats owned by the caller, or NULL for 1 on every head.  A scale that is not
 * finite and positive is recorded as PA_EINVAL in the device status (it is only read on the
 * device) and nothing is written; other errors as pa_reshape_and_cache_ex.
 */
pa_status pa_reshape_and_cache_per_head(const void* k, const void* v, void* k_blocks,
                                        void* v_blocks, const int32_t* slot_mapping,
                                        int64_t num_tokens, int32_t num_kv_heads,
                                        int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                        pa_dtype src_dtype, pa_dtype kv_dtype,
                                        const float* k_scales, const float* v_scales,
                                        cudaStream_t stream);

/*
 * pa_reshape_and_cache_per_block -- pa_reshape_and_cache_ex with one dequantisation factor per
 * (pool block, kv head) (tinyllm "Going further": fp8 KV caches with scales per block): head g
 * of a new row written to slot s is stored as x / k_block_scales[(s / block_size) *
 * num_kv_heads + g] (x / v_block_scales[...]).  k_block_scales, v_block_scales: DEVICE arrays
 * [num_blocks, num_kv_heads] of floats owned by the caller, both required (NULL: PA_EINVAL).
 * A factor of a block some row is written to that is not a finite positive normal float (at
 * least 2^-126) is recorded as PA_EINVAL in the device status and nothing is written; other
 * errors as
 * pa_reshape_and_cache_ex.  The caller chooses the factors (for example from a block's
 * largest magnitude when it is allocated); the library does not change them.
 */
pa_status pa_reshape_and_cache_per_block(const void* k, const void* v, void* k_blocks,
                                         void* v_blocks, const int32_t* slot_mapping,
                                         int64_t num_tokens, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t block_size,
                                         int64_t num_blocks, pa_dtype src_dtype,
                                         pa_dtype kv_dtype, const float* k_block_scales,
                                         const float* v_block_scales, cudaStream_t stream);

/*
 * pa_varlen_forward_workspace_size -- bytes of device workspace pa_varlen_forward needs
 * for these sizes (the per-call plan of work items and split-KV partial states).
 */
size_t pa_varlen_forward_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t max_blocks_per_seq, int32_t block_size);

/*
 * pa_varlen_forward -- batched varlen paged attention (TensorSharp Forward /
 * ComputeSingleQueryAttention; tinyllm section 2.2).  One call serves any mix of prefill
 * chunks and decode tokens.  For token t of sequence s at position p and head h, with
 * kv head g = h / (num_heads / num_kv_heads):
 *     end   = causal ? p + 1 : seq_lens[s]
 *     start = sliding_window > 0 ? max(0, end - sliding_window) : 0
 *     out[t, h] = softmax_j(scale * q[t, h] . K_j) V_j   over positions j in [start, end)
 * where K_j, V_j are pool rows of kv head g found through the block table.  out has
 * q_dtype.  k_blocks/v_blocks have kv_dtype (PA_FP8_E4M3: the codes' values, i.e. scales 1;
 * see pa_varlen_forward_ex for scaled pools).
 * Validation (tinyllm section 2.6), for every sequence with at least one query token:
 * seq_lens[s] >= 1, ceil(seq_lens[s] / block_size) <= max_blocks_per_seq, those table
 * entries in [0, num_blocks), positions in [0, seq_lens[s]); query_start_loc starts at 0,
 * never decreases and ends at num_tokens.  Failures record PA_EINVAL and leave out
 * untouched.  workspace must hold pa_varlen_forward_workspace_size(...) bytes, 256-byte
 * aligned; it is scratch owned by the caller and must not be shared by calls that overlap
 * on the device.
 */
pa_status pa_varlen_forward(const void* q, const void* k_blocks, const void* v_blocks, void* out,
                            const int32_t* query_start_loc, const int32_t* seq_lens,
                            const int32_t* positions, const int32_t* block_tables,
                            int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                            int64_t num_blocks, int32_t max_blocks_per_seq, pa_dtype q_dtype,
                            pa_dtype kv_dtype, float scale, int32_t causal,
                            int32_t sliding_window, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/*
 * pa_varlen_forward_ex -- pa_varlen_forward with optional extras (with sinks and lse NULL and
 * both scales 1 the call is pa_varlen_forward):
 *   sinks  [num_heads] fp32, device.  Per-head attention sink logits on the score scale
 *          (TensorSharp ForwardWithSinks): a virtual position with score sinks[h] and value
 *          zero, so with the visible scores s_j
 *              out[t, h] = sum_j e^(s_j - m) V_j / (e^(sinks[h] - m) + sum_j e^(s_j - m)),
 *          m = max(sinks[h], max_j s_j).  -inf means no sink for that head.  Finite values
 *          and -inf are defined; NaN and +inf are not.
 *   lse    [num_heads, num_tokens] fp32, device, written (the vllm.cpp MLA-prefill layout):
 *              lse[h, t] = log(e^sinks[h] + sum_j e^(s_j))   (natural log, sink term when given)
 *          and -inf when the sum is empty (no visible position and no sink).  It is what
 *          pa_merge_attn_states takes to combine two partial attentions of the same queries.
 *   k_scale, v_scale  dequantisation scales of the pools ("paged_attention_v2_pytorch.py":
 *          K = k_scale * k_blocks, V = v_scale * v_blocks before the attention), finite and
 *          > 0 (PA_EINVAL otherwise).  The scores above are scale * q . K_j with the scaled K.
 *          kv_dtype PA_FP8_E4M3 (pools written by pa_reshape_and_cache_ex) is accepted here:
 *          the pool's codes widen exactly to f16; on the tensor-core path q (bf16) enters the
 *          products as f16, so q entries must lie within f16's range (|q| <= 65504; entries
 *          below 2^-14 keep f16's subnormal precision), and the softmax weights enter the PV
 *          product as f16 (2^-11 relative).  fp8 pools take the tensor-core kernels for head
 *          size 128 with 16-position blocks (warp-MMA for decode tokens, tcgen05 for prefill
 *          chunks, as bf16 pools do) and the generic kernel otherwise.
 *   flags  0, or PA_FLAG_BITWISE: every sequence runs on the 16-row warp-MMA kernel (bf16 or
 *          fp8 pools, head size 64 / 128, 16-position blocks), including prefill-class
 *          sequences that would otherwise take the tensor-core prefill kernel.  That kernel
 *          folds each query row over the same 16-position blocks, in the same order and
 *          grouping, whatever the other rows of the batch are, so a token's out row and lse
 *          have the same bits computed as a decode token (q_len 1) or inside a prefill chunk,
 *          alone or in any batch (tinyllm 2.4: decode equals FlashAttention bit for bit, so
 *          prefill with one kernel and decode with the other agree).  Without the flag this
 *          holds for every sequence of at most 64 query rows per kv head; longer ones take
 *          the tcgen05 kernel, whose 128-key tiles group the sums differently (results within
 *          the tolerance, not bitwise).  Other bits: PA_EINVAL.
 * sinks and lse are read or written only for tokens of sequences with query tokens, and lse
 * is left untouched on a validation failure, like out.
 */
pa_status pa_varlen_forward_ex(const void* q, const void* k_blocks, const void* v_blocks,
                               void* out, const int32_t* query_start_loc,
                               const int32_t* seq_lens, const int32_t* positions,
                               const int32_t* block_tables, int32_t num_seqs, int64_t num_tokens,
                               int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int64_t num_blocks,
                               int32_t max_blocks_per_seq, pa_dtype q_dtype, pa_dtype kv_dtype,
                               float scale, int32_t causal, int32_t sliding_window,
                               const float* sinks, float* lse, float k_scale, float v_scale,
                               uint32_t flags, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream);

/*
 * pa_varlen_forward_per_head -- pa_varlen_forward_ex with one dequantisation scale per kv
 * head instead of one per pool: query head h (kv head g = h / (num_heads / num_kv_heads))
 * attends over K = k_scales[g] * k_blocks and V = v_scales[g] * v_blocks (tinyllm "Going
 * further": scales per head).  k_scales, v_scales: DEVICE arrays of num_kv_heads floats owned
 * by the caller, or NULL for 1 on every head; a scale that is not finite and positive is
 * recorded as PA_EINVAL in the device status and out / lse are left untouched.  All other
 * arguments, kernels and errors as pa_varlen_forward_ex.
 */
pa_status pa_varlen_forward_per_head(const void* q, const void* k_blocks, const void* v_blocks,
                                     void* out, const int32_t* query_start_loc,
                                     const int32_t* seq_lens, const int32_t* positions,
                                     const int32_t* block_tables, int32_t num_seqs,
                                     int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                     int32_t max_blocks_per_seq, pa_dtype q_dtype,
                                     pa_dtype kv_dtype, float scale, int32_t causal,
                                     int32_t sliding_window, const float* sinks, float* lse,
                                     const float* k_scales, const float* v_scales,
                                     uint32_t flags, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream);

/*
 * pa_varlen_forward_per_block -- pa_varlen_forward_ex over e4m3 pools with one dequantisation
 * factor per (pool block, kv head) (tinyllm "Going further": scales per block): position j of
 * a sequence, in pool block id = block_tables[s][j / block_size], is read by query head h (kv
 * head g = h / (num_heads / num_kv_heads)) as K = k_block_scales[id * num_kv_heads + g] *
 * k_blocks[...] and V = v_block_scales[...] * v_blocks[...].  k_block_scales, v_block_scales:
 * DEVICE arrays [num_blocks, num_kv_heads] of floats owned by the caller, both required (NULL:
 * PA_EINVAL).  The factors of every block a sequence with query tokens reads (the first
 * ceil(seq_lens[s] / block_size) entries of its table row) must be finite positive normal
 * floats (at least 2^-126), else PA_EINVAL is recorded in the device status and out / lse are left untouched.  kv_dtype must
 * be PA_FP8_E4M3 and the call must qualify for the warp-MMA path (q bf16, head_dim 128,
 * block_size 16, 16-byte aligned tensors), else PA_EUNSUPPORTED before anything is enqueued.
 * Both kernels multiply each block's scores by its K factor in fp32, exactly.  V: the
 * warp-MMA kernel (decode tokens) multiplies the block's softmax weights by the factor over
 * the largest factor the warp has met so far, before the weights are rounded to f16, and that
 * reference multiplies the warp's fp32 output; the tcgen05 kernel (prefill chunks) multiplies
 * the block's widened codes by the factor over its item's reference (the factor of the item's
 * first block), rounded to f16, and the reference multiplies the output.  An item with a V
 * ratio outside [2^-12, 146] is recomputed by the warp-MMA kernel.  So any finite positive
 * factors keep the f16 values in range.  Other arguments and errors as pa_varlen_forward_ex.
 */
pa_status pa_varlen_forward_per_block(const void* q, const void* k_blocks, const void* v_blocks,
                                      void* out, const int32_t* query_start_loc,
                                      const int32_t* seq_lens, const int32_t* positions,
                                      const int32_t* block_tables, int32_t num_seqs,
                                      int64_t num_tokens, int32_t num_heads,
                                      int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                      int64_t num_blocks, int32_t max_blocks_per_seq,
                                      pa_dtype q_dtype, pa_dtype kv_dtype, float scale,
                                      int32_t causal, int32_t sliding_window, const float* sinks,
                                      float* lse, const float* k_block_scales,
                                      const float* v_block_scales, uint32_t flags,
                                      void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream);

/*
 * pa_cache_and_attend -- one decode / prefill step over the cache: pa_slot_mapping_and_cache
 * of the new tokens' rows (k_new, v_new [num_tokens, num_kv_heads, head_dim] of kv_dtype;
 * slot_mapping [num_tokens] written) followed by pa_varlen_forward of q over the updated pools,
 * with the same arguments, results and errors as those two calls made one after the other.
 * For batches of up to 2048 tokens and 2047 sequences the slot mapping and scatter run as one
 * kernel launched right after the attention's planning kernel, overlapping it (neither reads
 * what the other writes), instead of in front of it.
 */
pa_status pa_cache_and_attend(const void* k_new, const void* v_new, const void* q,
                              void* k_blocks, void* v_blocks, void* out,
                              const int32_t* query_start_loc, const int32_t* seq_lens,
                              const int32_t* positions, const int32_t* block_tables,
                              int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                              int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                              int64_t num_blocks, int32_t max_blocks_per_seq, pa_dtype q_dtype,
                              pa_dtype kv_dtype, float scale, int32_t causal,
                              int32_t sliding_window, int32_t* slot_mapping, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/*
 * pa_varlen_forward_noalloc -- pa_varlen_forward for callers that cannot allocate device
 * memory.  The pages have no counterpart: it exists for the library's users, not for the
 * method.  Some callers cannot hand this library a workspace: a host framework that gives an
 * op only its input and output buffers and owns all other device memory, a runtime whose
 * allocator is out of reach of the calling code, or a serving step that must not risk the
 * device synchronisation of cudaMalloc / cudaFree.  This call computes exactly what
 * pa_varlen_forward computes (same arguments, minus the workspace) and keeps its per-call
 * plan in a 4 MiB array inside the library, one copy per device, held until the process
 * exits.  It allocates nothing and calls no allocating routine.
 *   - The first call on a device looks up that device's copy of the array (with the
 *     device current); make that first call before capturing the stream into a graph.
 *   - A batch whose pa_varlen_forward_workspace_size(...) exceeds 4 MiB returns PA_EINVAL
 *     at once and enqueues nothing.
 *   - All calls on a device share the array: calls that may overlap on the GPU (different
 *     streams without ordering between them) race and must not be issued.  Calls on one
 *     stream are ordered and safe.  Each call writes every word of the array it later reads,
 *     so nothing has to start at zero.
 */
pa_status pa_varlen_forward_noalloc(const void* q, const void* k_blocks, const void* v_blocks,
                                    void* out, const int32_t* query_start_loc,
                                    const int32_t* seq_lens, const int32_t* positions,
                                    const int32_t* block_tables, int32_t num_seqs,
                                    int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                                    int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                    int32_t max_blocks_per_seq, pa_dtype q_dtype,
                                    pa_dtype kv_dtype, float scale, int32_t causal,
                                    int32_t sliding_window, cudaStream_t stream);

/*
 * pa_decode_splitkv_partials -- phase 1 of split-KV decode ("paged_attention_v2_pytorch.py",
 * partition loop).  One query per sequence, q [num_seqs, num_heads, head_dim], at position
 * seq_lens[s] - 1 (causal by construction).  Partition p covers positions
 * [p * partition_size, min((p + 1) * partition_size, seq_lens[s])), intersected with the
 * window [max(0, seq_lens[s] - sliding_window), seq_lens[s]) when sliding_window > 0.
 * For every (s, h, p < max_num_partitions):
 *     max_logits[s, h, p] = max_j scale * q . K_j            (-inf if no position)
 *     exp_sums[s, h, p]   = sum_j exp(scale * q . K_j - max)  (0 if no position)
 *     tmp_out[s, h, p, :] = sum_j exp(...) V_j / exp_sum      (zeros if no position)
 * tmp_out holds the NORMALISED partition output (the reading under which the page's
 * reduction is a log-sum-exp merge).  max_logits / exp_sums are fp32 [S, H, P]; tmp_out fp32
 * [S, H, P, D].  Validation: seq_lens[s] >= 1, the table covers ceil(seq_len / block_size)
 * blocks with ids in [0, num_blocks), ceil(seq_len / partition_size) <= max_num_partitions.
 * partition_size must be a positive multiple of block_size.
 */
pa_status pa_decode_splitkv_partials(const void* q, const void* k_blocks, const void* v_blocks,
                                     float* max_logits, float* exp_sums, float* tmp_out,
                                     const int32_t* seq_lens, const int32_t* block_tables,
                                     int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                     int32_t max_blocks_per_seq, int32_t partition_size,
                                     int32_t max_num_partitions, pa_dtype q_dtype,
                                     pa_dtype kv_dtype, float scale, int32_t sliding_window,
                                     cudaStream_t stream);

/*
 * pa_decode_splitkv_partials_ex -- pa_decode_splitkv_partials over scaled pools
 * ("paged_attention_v2_pytorch.py": kv_cache_dtype, k_scale, v_scale; K = k_scale * k_blocks
 * and V = v_scale * v_blocks, both finite and > 0, else PA_EINVAL).  kv_dtype may be
 * PA_FP8_E4M3 (bf16 q and head size 128 take the warp-MMA kernel, with the f16 operand
 * rounding described at pa_varlen_forward_ex).  pa_decode_splitkv_partials is this call with
 * both scales 1; the reduce step needs no scales.
 */
pa_status pa_decode_splitkv_partials_ex(
    const void* q, const void* k_blocks, const void* v_blocks, float* max_logits,
    float* exp_sums, float* tmp_out, const int32_t* seq_lens, const int32_t* block_tables,
    int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq, int32_t partition_size,
    int32_t max_num_partitions, pa_dtype q_dtype, pa_dtype kv_dtype, float scale,
    int32_t sliding_window, float k_scale, float v_scale, cudaStream_t stream);

/*
 * pa_decode_splitkv_partials_per_head -- pa_decode_splitkv_partials_ex with one scale per kv
 * head: k_scales, v_scales are DEVICE arrays of num_kv_heads floats (NULL: 1), validated on
 * the device as in pa_varlen_forward_per_head (PA_EINVAL recorded, partials untouched).
 */
pa_status pa_decode_splitkv_partials_per_head(
    const void* q, const void* k_blocks, const void* v_blocks, float* max_logits,
    float* exp_sums, float* tmp_out, const int32_t* seq_lens, const int32_t* block_tables,
    int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq, int32_t partition_size,
    int32_t max_num_partitions, pa_dtype q_dtype, pa_dtype kv_dtype, float scale,
    int32_t sliding_window, const float* k_scales, const float* v_scales, cudaStream_t stream);

/*
 * pa_decode_splitkv_partials_per_block -- pa_decode_splitkv_partials_ex with one factor per
 * (pool block, kv head), as pa_varlen_forward_per_block (both arrays required; factors of the
 * blocks the sequences read validated on the device: PA_EINVAL recorded, partials untouched;
 * e4m3 pools on the warp-MMA path only, else PA_EUNSUPPORTED).
 */
pa_status pa_decode_splitkv_partials_per_block(
    const void* q, const void* k_blocks, const void* v_blocks, float* max_logits,
    float* exp_sums, float* tmp_out, const int32_t* seq_lens, const int32_t* block_tables,
    int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq, int32_t partition_size,
    int32_t max_num_partitions, pa_dtype q_dtype, pa_dtype kv_dtype, float scale,
    int32_t sliding_window, const float* k_block_scales, const float* v_block_scales,
    cudaStream_t stream);

/*
 * pa_decode_splitkv_reduce -- phase 2 ("Phase 2: Cross-partition reduction").  For each
 * (s, h) over partitions p < ceil(seq_lens[s] / partition_size):
 *     lse_p = max_logits + log(exp_sums), or -inf when max_logits is +/-inf or exp_sums <= 0
 *     M = max_p lse_p;  w_p = exp(lse_p - M);  out = sum_p w_p tmp_out_p * (1 / sum_p w_p)
 * and when every lse_p is -inf, out = tmp_out of partition 0 (the both-minus-infinity rule of
 * vllm.cpp MergeAttnStatesKernel, extended to P partitions).  Partitions combine in
 * increasing p.  out is [num_seqs, num_heads, head_dim] in out_dtype.
 */
pa_status pa_decode_splitkv_reduce(void* out, const float* max_logits, const float* exp_sums,
                                   const float* tmp_out, const int32_t* seq_lens,
                                   int32_t num_seqs, int32_t num_heads, int32_t head_dim,
                                   int32_t partition_size, int32_t max_num_partitions,
                                   pa_dtype out_dtype, cudaStream_t stream);

/* pa_decode_splitkv -- pa_decode_splitkv_partials followed by pa_decode_splitkv_reduce on
 * the same stream; the partial buffers are caller-owned scratch. */
pa_status pa_decode_splitkv(const void* q, const void* k_blocks, const void* v_blocks, void* out,
                            float* max_logits, float* exp_sums, float* tmp_out,
                            const int32_t* seq_lens, const int32_t* block_tables,
                            int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, int64_t num_blocks,
                            int32_t max_blocks_per_seq, int32_t partition_size,
                            int32_t max_num_partitions, pa_dtype q_dtype, pa_dtype kv_dtype,
                            float scale, int32_t sliding_window, cudaStream_t stream);

/*
 * pa_merge_attn_states -- merge two attention states of the same queries (vllm.cpp
 * cpu_mla_prefill.cpp, MergeAttnStatesKernel).  out/prefix_out/suffix_out [T, H, D] in dtype;
 * lse arrays fp32 [H, T]; out_lse may be NULL.  Tokens t >= prefill_tokens_with_context
 * (when that is >= 0) copy the suffix and its lse.  Otherwise an infinite lse of either sign
 * counts as -inf; if both are -inf the prefix output is emitted with lse -inf; else
 *     p_scale = p_se / (p_se + s_se), s_scale = s_se / (p_se + s_se),
 *     p_se = exp(p_lse - max), s_se = exp(s_lse - max),
 *     out = prefix * p_scale + suffix * s_scale,  out_lse = log(p_se + s_se) + max.
 */
pa_status pa_merge_attn_states(void* out, float* out_lse, const void* prefix_out,
                               const float* prefix_lse, const void* suffix_out,
                               const float* suffix_lse, int64_t num_tokens, int32_t num_heads,
                               int32_t head_dim, int64_t prefill_tokens_with_context,
                               pa_dtype dtype, cudaStream_t stream);

/*
 * pa_gather_kv -- copy sequences' cached rows into dense buffers (vllm.cpp
 * GatherMlaCacheKernel).  Output rows [cu_seq_lens[s], cu_seq_lens[s + 1]) receive the pool
 * rows (all kv heads) at positions (r - cu_seq_lens[s]) + seq_starts[s] of sequence s;
 * seq_starts may be NULL (all 0).  k_out/v_out are [cu_seq_lens[num_seqs], num_kv_heads,
 * head_dim]; v_blocks and v_out may both be NULL.  A position past the table row or a block
 * id outside the pool records PA_EINVAL and writes nothing.  Bit-exact copy.
 */
pa_status pa_gather_kv(const void* k_blocks, const void* v_blocks, void* k_out, void* v_out,
                       const int32_t* cu_seq_lens, const int32_t* seq_starts,
                       const int32_t* block_tables, int32_t num_seqs, int64_t num_out_rows,
                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                       int64_t num_blocks, int32_t max_blocks_per_seq, pa_dtype kv_dtype,
                       cudaStream_t stream);

/* ---- speculative decoding over the cache --------------------------------------------------
 *
 * A drafted step of a sequence: a tree of candidate tokens is cached behind its context
 * (pa_rope_and_cache), the tree attends to the context and to each node's ancestors
 * (pa_tree_attention), and the accepted path's rows are moved together (pa_tree_commit).  The
 * pages of forked, growing, shortened and ended sequences are kept by pa_fork_sequences,
 * pa_grow_sequences, pa_trim_sequences and pa_free_sequences; pa_copy_blocks makes the copies
 * that forks ask for, in every layer's pools.
 *
 * Where a call is several launches, another stream's pa_device_status() may clear the error that the
 * first one recorded before the next one reads it.  Such a call may then write those of its outputs
 * whose indices are valid; nothing outside its arrays is read or written.
 */

/* Long-context scalings of the rotary frequencies (pa_rope_frequencies). */
enum {
  PA_ROPE_PLAIN = 0,  /* f_i = base^(-2 i / rotary_dim) */
  PA_ROPE_LINEAR = 1, /* f_i / factor */
  PA_ROPE_NTK = 2,    /* base times factor^(rotary_dim / (rotary_dim - 2)) */
  PA_ROPE_YARN = 3,   /* f_i / factor for the slow pairs, f_i for the fast ones, a ramp over the
                         pair index between those that turn beta_slow and beta_fast times over
                         original_max_position; attention factor 0.1 ln(factor) + 1 */
  PA_ROPE_BANDS = 4   /* the same two ends, with a ramp over the turns f_i * original_max_position
                         / (2 pi) between low_freq_factor and high_freq_factor */
};
typedef struct {
  int32_t kind;   /* PA_ROPE_* */
  double factor;  /* >= 1; every kind but PA_ROPE_PLAIN */
  double original_max_position;              /* PA_ROPE_YARN, PA_ROPE_BANDS */
  double beta_fast, beta_slow;               /* PA_ROPE_YARN, usually 32 and 1 */
  double low_freq_factor, high_freq_factor;  /* PA_ROPE_BANDS, usually 1 and 4 */
} pa_rope_scaling;

/*
 * pa_rope_frequencies -- the rotary frequencies (radians per position) of the rotary_dim / 2
 * pairs, in fp64, for pa_rope_and_cache.  A host function: inv_freq and attn_factor (may be
 * NULL) are HOST pointers, scaling (NULL: plain) too.  rotary_dim positive and even (PA_ESHAPE),
 * base > 1, factor >= 1, original_max_position > 0, beta_fast > beta_slow > 0, high_freq_factor >
 * low_freq_factor > 0 where the kind uses them (PA_EINVAL).
 */
pa_status pa_rope_frequencies(int32_t rotary_dim, double base, const pa_rope_scaling* scaling,
                              double* inv_freq, float* attn_factor);

/*
 * pa_rope_and_cache -- rotary positions for the new tokens' queries and keys, and the scatter of
 * their keys and values into the pools, in one pass.
 *   q, q_out  [num_tokens, num_heads, head_dim] of src_dtype (both NULL: keys and values only);
 *             k, v [num_tokens, num_kv_heads, head_dim] of src_dtype.  Consecutive tokens lie
 *             *_stride elements apart (at least a token's row; e.g. views of one fused q/k/v
 *             product), a token's heads are contiguous.  q_out may be q with the same stride;
 *             otherwise the outputs overlap no input.
 *   positions [num_tokens] any int32, inv_freq [rotary_dim / 2] fp64 DEVICE (finite radians per
 *             position).  Pair i of a head's first rotary_dim elements, (x_i, x_(i + rotary_dim/2))
 *             or (x_2i, x_(2i+1)) when interleaved, becomes
 *               attn_factor * (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq[i];
 *             elements from rotary_dim on are unchanged.  The angle is off by less than 1.03 *
 *             2^-25 half turns at any position, for frequencies below 2^53 (fp32 products lose it
 *             at far positions); arithmetic in fp32.
 *   pools     as in pa_reshape_and_cache_ex: K stored as rotated value / scale, V as value / scale,
 *             rounded once to kv_dtype (e4m3 saturates), into row slot_mapping[t].  The scales are
 *             k_scale / v_scale, or k_scales / v_scales [num_kv_heads] DEVICE (NULL: the scalars;
 *             given, the scalar has to be 1).  Every slot is checked before anything is written
 *             (q_out included); a slot outside the pool, or a per-head scale that is not finite
 *             and positive, records PA_EINVAL.  Duplicate slots are undefined.
 * rotary_dim even, at most head_dim (PA_ESHAPE) and 256 (PA_EUNSUPPORTED); interleaved pairs need
 * an even head_dim (PA_EUNSUPPORTED).
 */
pa_status pa_rope_and_cache(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                            const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            void* k_blocks, void* v_blocks, const int32_t* positions,
                            const int32_t* slot_mapping, const double* inv_freq,
                            int32_t rotary_dim, int32_t interleaved, float attn_factor,
                            int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, int64_t num_blocks,
                            pa_dtype src_dtype, pa_dtype kv_dtype, float k_scale, float v_scale,
                            const float* k_scales, const float* v_scales, cudaStream_t stream);

/* pa_tree_attention_workspace_size -- bytes of device workspace pa_tree_attention needs for these
 * sizes (the plan of the call and the partial states of split items). */
size_t pa_tree_attention_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t max_blocks_per_seq, int32_t block_size);

/* pa_tree_attention_form -- how pa_tree_attention goes about a call of these sizes on the current
 * device (tensors on 16-byte boundaries, a positive scale): *row_tiles 0: the general kernel, in
 * three launches; 1 or 2: the tensor cores, items of that many tiles of query rows, *cluster CTAs
 * to each in one launch, or (*cluster 0) shares of all items in three launches.  row_tiles and
 * cluster are HOST pointers.  Sizes as there; without tokens PA_EINVAL.  It goes by the width of the
 * table, not by the lengths (which are on the device): where a step is captured over tables as wide
 * as the longest allowed sequence, short sequences take the shares, too. */
pa_status pa_tree_attention_form(int32_t num_seqs, int64_t num_tokens, int32_t mask_words,
                                 int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t max_blocks_per_seq, int32_t block_size, pa_dtype q_dtype,
                                 pa_dtype kv_dtype, int32_t* row_tiles, int32_t* cluster);

/*
 * pa_tree_attention -- attention of trees of drafted tokens over the paged cache.  Sequence s has
 * n = query_start_loc[s + 1] - query_start_loc[s] nodes, cached as its LAST n positions: node i
 * (token query_start_loc[s] + i) lies at position seq_lens[s] - n + i of the cache, behind a
 * context of seq_lens[s] - n positions.  positions[t] is the token's logical position (its
 * context length plus its depth, usually).  Token t of sequence s attends to
 *     every context position j, and every node i whose bit (i % 32) of
 *     tree_mask[t * mask_words + i / 32] is set (its ancestors and itself),
 * of which a sliding_window w > 0 leaves the keys with logical position > positions[t] - w (j for
 * a context position, positions[] of a node).  out = softmax(scale * q . K) V over those keys; a
 * token that sees no key gets 0 and lse -inf; one with a score of NaN or +inf gets NaN in both.
 * Bits of nodes >= n are ignored.  positions are read only when there is a window.
 * Types, sinks, lse, k_scale / v_scale and k_scales / v_scales as in pa_varlen_forward_ex and
 * pa_varlen_forward_per_head (a per-head array needs a scalar of 1); kv_dtype PA_FP8_E4M3 reads
 * the codes' values times the scales (bf16 q: its elements count to 2^-17 of their row's largest,
 * a row with an infinity counts as NaN; the softmax weights in f16).  Every cached V row of the
 * sequences has to be finite (a masked node's V enters the products with weight zero); K rows of masked
 * keys, and rows at or past seq_lens[s], may hold anything.
 * Validation, on the device before anything is written: query_start_loc starts at 0, never
 * decreases and ends at num_tokens; for a sequence with nodes n <= 32 * mask_words, n <=
 * seq_lens[s], its table covers seq_lens[s] positions with ids in [0, num_blocks), positions >= 0
 * when there is a window; per-head scales finite and positive.  Failures record PA_EINVAL and
 * leave out and lse untouched.  mask_words > 64 is PA_EUNSUPPORTED.  A call without tokens does
 * nothing.
 * workspace: pa_tree_attention_workspace_size(...) bytes, 256-byte aligned, scratch of the caller
 * that calls which overlap on the device must not share.  The results of a call depend on its
 * inputs alone (no atomics on values); how a context is split, and so the last bits of a row,
 * depend on the sizes and the lengths of the whole batch.
 */
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
                            cudaStream_t stream);

/*
 * pa_tree_commit -- keep the accepted path of each sequence's tree: position context_lens[s] + i
 * gets the K and V rows of position context_lens[s] + accepted[s * max_accepted + i], for i <
 * num_accepted[s], as if all rows were read before any is written.  Bit-exact copies (pools of any
 * kv_dtype; with per-block dequantisation factors only where the blocks' factors agree).  The
 * accepted nodes of a sequence strictly increase (a path's nodes do, parents being numbered before
 * their children).  0 <= num_accepted[s] <= max_accepted, nodes >= 0 and strictly increasing, the
 * positions inside the table and their ids in [0, num_blocks): otherwise PA_EINVAL is recorded and
 * nothing is written.  Entries past num_accepted[s] are ignored.  A block that is written belongs
 * to one sequence only (pa_fork_sequences gives every child its own last block).
 */
pa_status pa_tree_commit(void* k_blocks, void* v_blocks, const int32_t* block_tables,
                         const int32_t* context_lens, const int32_t* accepted,
                         const int32_t* num_accepted, int32_t num_seqs, int32_t max_accepted,
                         int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                         int64_t num_blocks, int32_t max_blocks_per_seq, pa_dtype kv_dtype,
                         cudaStream_t stream);

/*
 * pa_copy_blocks -- copy whole pool blocks: for every pair (src, dst) of block_pairs
 * [num_pairs, 2] (DEVICE, 8-byte aligned), block dst of each pool gets block src; (-1, -1) pairs
 * are skipped.  A source may repeat; destinations are distinct and no destination is a source:
 * this and the ids' range are checked before anything is written (PA_EINVAL recorded).  v_blocks
 * may be NULL.  Per-block dequantisation factors [num_blocks, num_kv_heads] move with the same
 * call, as f32 pools of block size 1 and head size 1.  More than 256 pairs need num_blocks <=
 * 2^23 (PA_EUNSUPPORTED).
 */
pa_status pa_copy_blocks(void* k_blocks, void* v_blocks, const int32_t* block_pairs,
                         int64_t num_pairs, int32_t num_kv_heads, int32_t head_dim,
                         int32_t block_size, int64_t num_blocks, pa_dtype kv_dtype,
                         cudaStream_t stream);

/*
 * Page bookkeeping, on the device and in the stream's order:
 *   block_tables [num_rows, max_blocks_per_seq], seq_lens [num_rows]: row r's first
 *                ceil(seq_lens[r] / block_size) entries are the blocks it holds;
 *   ref_counts   [num_blocks]: rows that hold each block;
 *   free_list    [num_blocks], free_count [1]: the ids of the blocks that nobody holds are
 *                free_list[0 .. *free_count - 1], each once (the caller sets this up).
 * Blocks are taken from the end of the free list.  Each call checks everything that it uses before
 * it writes: a row outside [0, num_rows), a written row listed twice, a length that is negative or
 * beyond the table, an entry that it shares or lets go outside the pool or without a reference, a
 * block taken from the free list that is outside the pool or has a reference, too few free blocks,
 * or a count outside [0, num_blocks] records PA_EINVAL and leaves every array as it was.  Entries
 * that stay as they are (all that a growing row holds, those in front of a trimmed row's end) and
 * free blocks that are not taken are not looked at.  num_rows <= 65536, num_blocks <= 2^23 and
 * num_rows * max_blocks_per_seq < 2^31, else
 * PA_EUNSUPPORTED.  Calls on the same arrays must not overlap on the device.
 *
 * pa_fork_sequences -- fork f makes row children[f] a copy of row parents[f]: whole blocks are
 * shared (their counts rise by one), a partly filled last block is replaced by a new one, for
 * which block_pairs[f] = (parent's block, new block); (-1, -1) when there is none.  Forks take
 * their blocks in list order.  A row may be the parent of several forks, but children are
 * distinct and none is a parent; what a child's row held before is forgotten, not freed.  Give
 * block_pairs [num_forks, 2] to pa_copy_blocks for every layer's pools.
 */
pa_status pa_fork_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* parents,
                            const int32_t* children, int32_t num_forks, int32_t num_rows,
                            int32_t max_blocks_per_seq, int32_t block_size, int32_t* ref_counts,
                            int32_t* free_list, int32_t* free_count, int64_t num_blocks,
                            int32_t* block_pairs, cudaStream_t stream);

/* pa_grow_sequences -- lengthen row sequences[i] to new_lens[i] >= its length, taking the blocks
 * this needs (in list order, ascending position) and writing them behind the row's blocks. */
pa_status pa_grow_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* sequences,
                            const int32_t* new_lens, int32_t num_sequences, int32_t num_rows,
                            int32_t max_blocks_per_seq, int32_t block_size, int32_t* ref_counts,
                            int32_t* free_list, int32_t* free_count, int64_t num_blocks,
                            cudaStream_t stream);

/* pa_trim_sequences -- shorten row sequences[i] to new_lens[i], 0 <= new_lens[i] <= its length
 * (after a drafted step: to the context and the accepted tokens).  The blocks behind
 * ceil(new_lens[i] / block_size) are let go as in pa_free_sequences.  A last block that stays
 * partly filled is not replaced: a row cut inside a block that other rows hold, too, shares that
 * block with them, so fork the row before anything is written behind its end. */
pa_status pa_trim_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* sequences,
                            const int32_t* new_lens, int32_t num_sequences, int32_t num_rows,
                            int32_t max_blocks_per_seq, int32_t block_size, int32_t* ref_counts,
                            int32_t* free_list, int32_t* free_count, int64_t num_blocks,
                            cudaStream_t stream);

/* pa_free_sequences -- end the rows in `sequences` (distinct): every block they hold loses a
 * reference for each row that holds it, blocks without references are appended to the free list
 * in ascending order, and the rows' lengths become 0 (their table entries stay). */
pa_status pa_free_sequences(int32_t* block_tables, int32_t* seq_lens, const int32_t* sequences,
                            int32_t num_sequences, int32_t num_rows, int32_t max_blocks_per_seq,
                            int32_t block_size, int32_t* ref_counts, int32_t* free_list,
                            int32_t* free_count, int64_t num_blocks, cudaStream_t stream);

/* ---- caches of bounded size ---------------------------------------------------------------
 *
 * Long sequences either see a window of the cache and its first tokens (pa_window_attention), or keep
 * the keys that queries looked at: each step adds up the attention weight that every cached key
 * receives (pa_attention_key_weights), and now and then those with the least of it are evicted
 * (pa_evict_keys) and the pages behind the sequences' new ends given back (pa_trim_sequences).  Keys
 * keep the rotary positions they were cached with; `positions` of these calls count cached keys, so
 * after an eviction a new token lies at the sequence's new length.
 *
 * As above, another stream's pa_device_status() may clear a recorded error between the launches of a
 * call: it may then write those of its outputs whose indices are valid, nothing outside its arrays.  An
 * error that is recorded while an attention call runs (another stream's, or a wait that runs out) may leave
 * out, lse and the sums in key_weights written in part.  Neither holds of pa_evict_keys.
 */

/* pa_window_attention_workspace_size -- bytes of device workspace pa_window_attention needs for these
 * sizes. */
size_t pa_window_attention_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                          int32_t num_kv_heads, int32_t head_dim,
                                          int32_t max_blocks_per_seq, int32_t block_size);

/*
 * pa_window_attention -- causal varlen paged attention behind a sliding window whose first tokens stay
 * visible.  Token t of sequence s at position p = positions[t] attends to the keys j <= p with
 *     j > p - sliding_window  or  j < first_tokens
 * (sliding_window 0: all j <= p, whatever first_tokens).  One call serves any mix of prompt chunks and
 * decoding tokens.  out = softmax(scale * q . K) V over those keys; a row with a score of NaN or +inf
 * gets NaN in out and lse.  Types, sinks (logits, besides the first tokens), lse, k_scale / v_scale and
 * k_scales / v_scales as in pa_varlen_forward_ex and pa_varlen_forward_per_head (a per-head array needs
 * a scalar of 1).  bf16 q over e4m3 pools enters the products with 17 bits of its row's largest element
 * or more (a row with an infinity comes out as NaN).  Softmax weights enter the products with V with 16
 * bits, of large batches of prompt chunks, and over e4m3 pools, with 11 (f16, or off by 2^-32 of the row's
 * largest); those batches' bf16 V as f16, exact from 2^-14 on and off by 2^-25 at most below,
 * but as it is where no value of 2^-9 or more is found in a kv head of a sequence (8 values of the first row of
 * each block that the sequence reads are looked at).
 * K rows of keys that a token does not see may hold anything.  So may V rows at or past seq_lens[s],
 * and those of blocks between the first tokens' and the first that the sequence's tokens reach: these
 * are not read, and their table entries not looked at (a server may have given them away).  All other V
 * rows of the sequence have to be finite (an unseen one enters the products with weight zero), their
 * magnitudes, scaled, up to 2^100 (the sums before the division are fp32, of weights up to 2^8).
 * Validation, on the device before anything is written: query_start_loc starts at 0, never decreases
 * and ends at num_tokens; for a sequence with tokens, seq_lens[s] >= 1, its table covers seq_lens[s]
 * positions with ids in [0, num_blocks) where they are read, and its tokens' positions lie in
 * [0, seq_lens[s]) and do not decrease; per-head scales finite and positive.  Failures record PA_EINVAL
 * and leave out and lse untouched.  sliding_window and first_tokens >= 0 (PA_EINVAL).  A call without
 * tokens does nothing.
 * The outputs overlap no input and not one another.
 * A batch with num_tokens <= num_seqs is taken for one of decoding tokens: a prompt chunk among as many
 * sequences without tokens is right, but slow (leave those sequences out).
 * workspace: pa_window_attention_workspace_size(...) bytes, 256-byte aligned, scratch of the caller
 * that calls which overlap on the device must not share.  The results depend on the inputs alone (no
 * atomics on values); how keys are split, and so the last bits of a row, depend on the whole batch.
 */
pa_status pa_window_attention(const void* q, const void* k_blocks, const void* v_blocks, void* out,
                              const int32_t* query_start_loc, const int32_t* seq_lens,
                              const int32_t* positions, const int32_t* block_tables, int32_t num_seqs,
                              int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int64_t num_blocks,
                              int32_t max_blocks_per_seq, pa_dtype q_dtype, pa_dtype kv_dtype,
                              float scale, int32_t sliding_window, int32_t first_tokens,
                              const float* sinks, float* lse, float k_scale, float v_scale,
                              const float* k_scales, const float* v_scales, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/* pa_attention_key_weights_workspace_size -- bytes of device workspace pa_attention_key_weights needs. */
size_t pa_attention_key_weights_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_heads,
                                               int32_t num_kv_heads, int32_t head_dim,
                                               int32_t max_blocks_per_seq, int32_t block_size);

/*
 * pa_attention_key_weights -- pa_window_attention that also adds up the attention weight of every key:
 *     key_weights[s, g, j] += sum over tokens t of sequence s and heads h of kv head g's group of
 *                             exp(scale * q[t, h] . K_j - lse[h, t])
 * for the keys j that t sees.  observed_tokens > 0 counts each sequence's last so many tokens only
 * (of a long prompt, say), 0 all of them.  key_weights [num_seqs, num_kv_heads, weights_len] fp32
 * DEVICE; entries of keys that no counted token sees, and those at or past seq_lens[s], are left as
 * they are.  A sequence with tokens and seq_lens[s] > weights_len is refused (PA_EINVAL recorded), and a
 * refused call leaves key_weights untouched, too.  A row whose lse is NaN spoils the keys it sees, and no
 * others.  Weights below 2^-126 may count as 0; scale * k_scale >= 2^-100.
 * All other arguments, results and errors as pa_window_attention, and its workspace
 * pa_attention_key_weights_workspace_size(...) bytes (for decoding tokens, whose scores wait there for the
 * log-sum-exps, up to 256 MB or 8 KB for each (sequence, kv head), whichever is more).
 */
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
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* pa_evict_keys_workspace_size -- bytes of device workspace pa_evict_keys needs for these sizes: 4096, and
 * where a table row covers more than 8192 positions a word for each (sequence, kv head, position). */
size_t pa_evict_keys_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t max_blocks_per_seq,
                                    int32_t block_size);

/*
 * pa_evict_keys -- cut every sequence with new_lens[s] < seq_lens[s] to new_lens[s] keys, each kv head
 * its own.  With n = seq_lens[s], kept are the first f = min(keep_first, new_lens[s]) keys, the last
 * r = min(keep_recent, new_lens[s] - f), and of the keys [f, n - r) the new_lens[s] - f - r with the
 * largest key_weights[s, g, .] (ties: the lowest index; NaN counts as larger than any number;
 * key_weights NULL: all are alike).  Kept keys below new_lens[s] - r stay in place, the other kept ones
 * of [f, n - r) fill the places that become free there in ascending order, and the last r move up to
 * [new_lens[s] - r, new_lens[s]).  K and V rows (bit-exact copies, pools of any kv_dtype; with per-block
 * dequantisation factors only where the blocks' factors agree) and the weights move alike, and the
 * weights of [new_lens[s], n) become 0, ready for new keys.  Lengths and tables stay: give the same
 * new_lens to pa_trim_sequences.  Sequences with new_lens[s] >= n are left as they are.
 * Checked before any row or weight is written: n and new_lens[s] not negative, the table covers n
 * positions with ids in [0, num_blocks) (where keys are evicted), n <= weights_len (given weights):
 * otherwise PA_EINVAL is recorded and nothing is written.  The call is whole: it goes by what this check
 * found, an error recorded before it included, so errors that other streams record or clear meanwhile
 * change nothing.  A block that is written belongs to one sequence only.  num_seqs and num_kv_heads <=
 * 65535 and at most 524288 keys to a sequence (the smaller of the table's width and, given weights,
 * weights_len), num_blocks * block_size < 2^31, else PA_EUNSUPPORTED.
 * workspace: pa_evict_keys_workspace_size(...) bytes, 256-byte aligned, scratch of the caller that calls
 * which overlap on the device must not share.
 */
pa_status pa_evict_keys(void* k_blocks, void* v_blocks, const int32_t* block_tables,
                        const int32_t* seq_lens, const int32_t* new_lens, float* key_weights,
                        int64_t weights_len, int32_t keep_first, int32_t keep_recent, int32_t num_seqs,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks,
                        int32_t max_blocks_per_seq, pa_dtype kv_dtype, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
