// bf16 instances of the windowed decode, and how many clusters of any instance's CTAs (a
// whole SM each) the GPU holds.
#include "span_decode.cuh"

namespace pa {
cudaError_t run_span_bf16(int head_dim, const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  return head_dim == 128 ? span::run_span<SpanPool::kBf16, 128, 8>(p, grid, smem, stream)
                         : span::run_span<SpanPool::kBf16, 64, 8>(p, grid, smem, stream);
}

int span_cluster_room(int splits, int num_sms) {
  if (splits <= 1) return num_sms;
  static std::atomic<int> known[64][kSpanCluster + 1];       // 0: not asked yet
  int device = 0;
  if (span::configure_span<SpanPool::kBf16, 128, 8>(&device) == cudaSuccess) {
    std::atomic<int>& room = known[device & 63][splits];
    int n = room.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(splits));
    cfg.blockDim = dim3(kSpanThreads);
    cfg.dynamicSmemBytes = kSpanSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, span::span_decode_kernel<SpanPool::kBf16, 128, 8>, &cfg) == cudaSuccess && n > 0) {
      n *= splits;
      room.store(n, std::memory_order_relaxed);
      return n;
    }
  }
  cudaGetLastError();
  return num_sms / 2;
}
}  // namespace pa
