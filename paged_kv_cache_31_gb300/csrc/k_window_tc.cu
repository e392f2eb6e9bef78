// k_window_tc.cu -- launches of the attention behind a window with first tokens on the tensor cores
// (k_tree_tc.cuh, kWindow and kMarked): batches of prompt chunks that are too small for k_prefill_tc.cu, of
// head size 64 or of a group that 128 rows are no multiple of, cut into even shares (2 chunks of 300 and 500
// tokens behind 1000 and 3000 positions, 32 + 8 heads: 60 us, e4m3 61), and the items it marked.
#include "k_tree_tc.cuh"

namespace pa {
namespace {

template <int D, bool FP8, int MODE = kWindow>
cudaError_t launch_as(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const TreeParams& p, uint64_t limit, uint32_t stall, cudaStream_t stream) {
  using S = Shape<D, FP8>;
  auto kern = k_tree_tc<D, FP8, MODE>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.grid), dim3(S::kThreads), S::kSmem, stream, tq, tk, tv, p, limit,
                    stall);
}

}  // namespace

cudaError_t launch_window_tc(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const TreeParams& p, bool fp8, uint64_t wait_limit, uint32_t stall,
                             cudaStream_t stream) {
  if (p.tc.plan) return launch_as<128, false, kMarked>(tq, tk, tv, p, wait_limit, stall, stream);
  if (fp8) return launch_as<128, true>(tq, tk, tv, p, wait_limit, stall, stream);
  if (p.m.head_dim == 128) return launch_as<128, false>(tq, tk, tv, p, wait_limit, stall, stream);
  return launch_as<64, false>(tq, tk, tv, p, wait_limit, stall, stream);
}

}  // namespace pa
