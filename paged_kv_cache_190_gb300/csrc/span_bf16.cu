// bf16 instances of the windowed decode.
#include "span_decode.cuh"

namespace pa {
cudaError_t run_span_bf16(int head_dim, const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  return head_dim == 128 ? span::run_span<SpanPool::kBf16, 128, 8>(p, grid, smem, stream)
                         : span::run_span<SpanPool::kBf16, 64, 8>(p, grid, smem, stream);
}
}  // namespace pa
