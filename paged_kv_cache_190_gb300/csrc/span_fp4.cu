// The instance for 4-bit rows (1 to 8 query rows of a kv head).
#include "span_decode.cuh"

namespace pa {
cudaError_t run_span_fp4(const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  return span::run_span<SpanPool::kFp4, 128, 8>(p, grid, smem, stream);
}
}  // namespace pa
