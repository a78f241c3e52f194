// float32 instances of the windowed decode: one for each number of query rows of a kv
// head (they live in registers).
#include "span_decode.cuh"

namespace pa {
namespace {
template <int D>
cudaError_t run(const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  switch (p.rows) {
    case 1: return span::run_span<SpanPool::kF32, D, 1>(p, grid, smem, stream);
    case 2: return span::run_span<SpanPool::kF32, D, 2>(p, grid, smem, stream);
    case 4: return span::run_span<SpanPool::kF32, D, 4>(p, grid, smem, stream);
    default: return span::run_span<SpanPool::kF32, D, 8>(p, grid, smem, stream);
  }
}
}  // namespace
cudaError_t run_span_f32(int head_dim, const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  return head_dim == 128 ? run<128>(p, grid, smem, stream) : run<64>(p, grid, smem, stream);
}
}  // namespace pa
