// k_tree_tc.cu -- launches of tree attention on the tensor cores (k_tree_tc.cuh).
#include <algorithm>
#include <atomic>

#include "k_tree_tc.cuh"

namespace pa {
namespace {

template <int D, bool FP8, bool CL>
cudaError_t launch_as(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const TreeParams& p, uint64_t limit, uint32_t stall, cudaStream_t stream) {
  using S = Shape<D, FP8>;
  auto kern = k_tree_tc<D, FP8, CL ? kClusters : kShares>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  if constexpr (!CL)
    return launch_pdl(kern, dim3(p.grid), dim3(S::kThreads), S::kSmem, stream, tq, tk, tv, p, limit,
                      stall);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p, limit, stall);
}

template <int D, bool FP8>
int resident(int c) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c);
  cfg.blockDim = dim3(Shape<D, FP8>::kThreads);
  cfg.dynamicSmemBytes = Shape<D, FP8>::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = c;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kern = k_tree_tc<D, FP8, kClusters>;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<D, FP8>::kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

template <int D, bool FP8>
cudaError_t launch_mode(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const TreeParams& p, uint64_t limit, uint32_t stall, cudaStream_t stream) {
  return p.cluster ? launch_as<D, FP8, true>(tq, tk, tv, p, limit, stall, stream)
                   : launch_as<D, FP8, false>(tq, tk, tv, p, limit, stall, stream);
}

}  // namespace

int tree_clusters_resident(int device, bool fp8, int head_dim, int c) {
  // [device][variant][cluster size 2, 4, 8]: number + 1, 0 while it is not known
  static std::atomic<int> known[64][3][3];
  const int variant = fp8 ? 2 : head_dim == 128, at = c == 2 ? 0 : c == 4 ? 1 : 2;
  if (device < 0 || device >= 64) return 0;
  const int k = known[device][variant][at].load(std::memory_order_relaxed);
  if (k) return k - 1;
  const int n = fp8 ? resident<128, true>(c) : variant ? resident<128, false>(c) : resident<64, false>(c);
  known[device][variant][at].store(n + 1, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_tree_tc(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const TreeParams& p, bool fp8, uint64_t wait_limit, uint32_t stall,
                           cudaStream_t stream) {
  if (fp8) return launch_mode<128, true>(tq, tk, tv, p, wait_limit, stall, stream);
  if (p.m.head_dim == 128) return launch_mode<128, false>(tq, tk, tv, p, wait_limit, stall, stream);
  return launch_mode<64, false>(tq, tk, tv, p, wait_limit, stall, stream);
}

}  // namespace pa
