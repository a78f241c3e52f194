// C ABI entry points of the windowed decode, of the decode over e4m3 pools with a scale
// for each page and head, and of the decode over 4-bit rows: argument checks on the host, then the launcher.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/pa.h"
#include "pa_host.h"
#include "span_decode.h"

namespace {

bool shape_ok(int head_dim, int block_size) {
  return (head_dim == 64 || head_dim == 128) && (block_size == 16 || block_size == 32);
}

int run(pa::SpanPool pool, void* out, const void* q, const void* k_cache, const void* v_cache,
        const int32_t* block_tables, const int32_t* context_lens, float scale,
        const float* k_scales, const float* v_scales, int num_kv_heads, int num_seqs,
        int num_q_heads, int q_len, int head_dim, int block_size, int num_blocks,
        int max_blocks_per_seq, int max_context_len, int window, int sinks, void* workspace,
        size_t workspace_bytes, int32_t* device_errors, void* stream) {
  if (num_kv_heads <= 0 || num_q_heads <= 0 || num_seqs < 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || max_context_len < 0 || q_len < 1 || window < 0 || sinks < 0)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0 || (window == 0 && sinks > 0)) return PA_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(q_len) * (num_q_heads / num_kv_heads);
  if (rows != 1 && rows != 2 && rows != 4 && rows != 8) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size ||
      max_context_len >= pa::kNoWindow ||
      static_cast<int64_t>(num_blocks) * num_kv_heads > INT32_MAX ||
      static_cast<int64_t>(num_seqs) * num_kv_heads > INT32_MAX / pa::kSpanCluster)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
  if (pool == pa::SpanPool::kFp8 && (!k_scales || !v_scales)) return PA_ERR_INVALID_ARG;
  using pa::aligned16;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID_ARG;
  const int sms = pa::current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < pa::span_workspace_size(static_cast<int>(rows), num_kv_heads, head_dim, sms))
    return PA_ERR_WORKSPACE;
  pa::SpanArgs a = {};
  a.pool = pool;
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.tables = block_tables;
  a.lens = context_lens;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.scale = scale;
  a.num_seqs = num_seqs;
  a.q_len = q_len;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.max_len = max_context_len;
  a.window = window;
  a.sinks = sinks;
  a.workspace = workspace;
  a.device_errors = device_errors;
  a.num_sms = sms;
  a.wait_limit = pa::wait_limit();
  return pa::launch_span_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pa_decode_window_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                       int head_dim, int block_size, int max_context_len,
                                       int window, int sinks) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_context_len < 0 || window < 0 ||
      sinks < 0 || num_q_heads % num_kv_heads != 0)
    return 0;
  const int rows = num_q_heads / num_kv_heads;
  if (!shape_ok(head_dim, block_size) || rows > 8) return 0;
  const int sms = pa::current_sm_count();
  return sms <= 0 ? 0 : pa::span_workspace_size(rows, num_kv_heads, head_dim, sms);
}

int pa_decode_window(void* out, const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, const int32_t* context_lens, float scale,
                     int num_kv_heads, int num_seqs, int num_q_heads, int q_len, int head_dim,
                     int block_size, int num_blocks, int max_blocks_per_seq, int max_context_len,
                     int window, int sinks, pa_dtype dtype, void* workspace,
                     size_t workspace_bytes, int32_t* device_errors, void* stream) {
  if ((dtype != PA_F32 && dtype != PA_BF16) || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  return run(dtype == PA_F32 ? pa::SpanPool::kF32 : pa::SpanPool::kBf16, out, q, k_cache, v_cache,
             block_tables, context_lens, scale, nullptr, nullptr, num_kv_heads, num_seqs,
             num_q_heads, q_len, head_dim, block_size, num_blocks, max_blocks_per_seq,
             max_context_len, window, sinks, workspace, workspace_bytes, device_errors, stream);
}

int pa_decode_fp8_block(void* out, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, const int32_t* context_lens, float scale,
                        const float* k_scales, const float* v_scales, int num_kv_heads,
                        int num_seqs, int num_q_heads, int q_len, int head_dim, int block_size,
                        int num_blocks, int max_blocks_per_seq, int max_context_len, int window,
                        int sinks, void* workspace, size_t workspace_bytes,
                        int32_t* device_errors, void* stream) {
  if (head_dim != 128 || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  return run(pa::SpanPool::kFp8, out, q, k_cache, v_cache, block_tables, context_lens, scale,
             k_scales, v_scales, num_kv_heads, num_seqs, num_q_heads, q_len, head_dim, block_size,
             num_blocks, max_blocks_per_seq, max_context_len, window, sinks, workspace,
             workspace_bytes, device_errors, stream);
}

int pa_decode_fp4(void* out, const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, const int32_t* context_lens, float scale,
                  int num_kv_heads, int num_seqs, int num_q_heads, int q_len, int head_dim,
                  int block_size, int num_blocks, int max_blocks_per_seq, int max_context_len,
                  int window, int sinks, void* workspace, size_t workspace_bytes,
                  int32_t* device_errors, void* stream) {
  if (head_dim != 128 || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  return run(pa::SpanPool::kFp4, out, q, k_cache, v_cache, block_tables, context_lens, scale,
             nullptr, nullptr, num_kv_heads, num_seqs, num_q_heads, q_len, head_dim, block_size,
             num_blocks, max_blocks_per_seq, max_context_len, window, sinks, workspace,
             workspace_bytes, device_errors, stream);
}

}  // extern "C"
