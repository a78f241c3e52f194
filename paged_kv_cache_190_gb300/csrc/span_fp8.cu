// The e4m3 instance (a scale for each page and head; 1 to 8 query rows of a kv head).
#include "span_decode.cuh"

namespace pa {
cudaError_t run_span_fp8(const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  return span::run_span<SpanPool::kFp8, 128, 8>(p, grid, smem, stream);
}
}  // namespace pa
