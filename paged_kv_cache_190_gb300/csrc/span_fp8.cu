// e4m3 instances (a scale for each page and head): up to 4 query rows of a kv head share
// one value product for both parts of their weights, 8 rows take two.
#include "span_decode.cuh"

namespace pa {
cudaError_t run_span_fp8(const SpanParams& p, int grid, int smem, cudaStream_t stream) {
  return p.rows <= 4 ? span::run_span<SpanPool::kFp8, 128, 4>(p, grid, smem, stream)
                     : span::run_span<SpanPool::kFp8, 128, 8>(p, grid, smem, stream);
}
}  // namespace pa
