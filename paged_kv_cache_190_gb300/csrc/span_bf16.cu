// bf16 instances of the windowed decode, and how many clusters of any instance's CTAs (a
// whole SM each) the GPU holds.
#include "span_decode.cuh"

namespace pa {
cudaError_t run_span_bf16(int head_dim, const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  return head_dim == 128 ? span::run_span<SpanPool::kBf16, 128, 8>(p, grid, smem, stream)
                         : span::run_span<SpanPool::kBf16, 64, 8>(p, grid, smem, stream);
}

void span_cluster_rooms(int num_sms, int (&room)[kSpanCluster + 1]) {
  static std::atomic<int> known[64][kSpanCluster + 1];       // 0: not asked yet
  room[0] = 0;
  room[1] = num_sms;
  int device = 0;
  const bool ready = span::configure_span<SpanPool::kBf16, 128, 8>(&device) == cudaSuccess;
  for (int splits = 2; splits <= kSpanCluster; ++splits) {
    std::atomic<int>& n = known[device & 63][splits];
    room[splits] = n.load(std::memory_order_relaxed);
    if (room[splits] > 0) continue;
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
    int clusters = 0;
    if (ready && cudaOccupancyMaxActiveClusters(&clusters, span::span_decode_kernel<SpanPool::kBf16, 128, 8>, &cfg) ==
                     cudaSuccess && clusters > 0) {
      room[splits] = clusters * splits;
      n.store(room[splits], std::memory_order_relaxed);
    } else {
      cudaGetLastError();                                    // (not this call's error)
      room[splits] = num_sms / 2;
    }
  }
}
}  // namespace pa
