// C ABI entry points of the prompt attention: argument checks on the host, then the launcher.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/pa.h"
#include "pa_host.h"
#include "prefill.h"

extern "C" {

size_t pa_prefill_workspace_size(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads,
                                 int head_dim) {
  if (num_tokens < 0 || num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  const int sms = pa::current_sm_count();
  return sms <= 0 ? 0 : pa::prefill_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, sms);
}

int pa_prefill(void* out, const void* q, const void* k_cache, const void* v_cache,
               const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_starts,
               float scale, int num_kv_heads, int num_seqs, int num_tokens, int num_q_heads,
               int head_dim, int block_size, int num_blocks, int max_blocks_per_seq,
               int max_context_len, int window, int sinks, pa_dtype dtype, void* workspace,
               size_t workspace_bytes, int32_t* device_errors, void* stream) {
  if ((dtype != PA_F32 && dtype != PA_BF16) || (head_dim != 64 && head_dim != 128) ||
      (block_size != 16 && block_size != 32))
    return PA_ERR_UNSUPPORTED;
  if (num_kv_heads <= 0 || num_q_heads <= 0 || num_seqs < 0 || num_tokens < 0 || num_blocks <= 0 ||
      max_blocks_per_seq < 0 || max_context_len < 0 || window < 0 || sinks < 0)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0 || (window == 0 && sinks > 0)) return PA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(pa::prefill_scale_log2(scale))) return PA_ERR_INVALID_ARG;
  const int group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_UNSUPPORTED;
  // (rows and items are numbered in 31 bits)
  if (static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size ||
      max_context_len >= pa::kPrefillNoWindow ||
      static_cast<int64_t>(num_blocks) * num_kv_heads > INT32_MAX ||
      (static_cast<int64_t>(num_tokens) + num_seqs) * num_q_heads > INT32_MAX / 2)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !q_starts)
    return PA_ERR_INVALID_ARG;
  using pa::aligned16;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PA_ERR_INVALID_ARG;
  const int sms = pa::current_sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < pa::prefill_workspace_size(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, sms))
    return PA_ERR_WORKSPACE;
  pa::PrefillArgs a = {};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.tables = block_tables;
  a.lens = context_lens;
  a.starts = q_starts;
  a.scale = scale;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.max_len = max_context_len;
  a.window = window;
  a.sinks = sinks;
  a.f32 = dtype == PA_F32;
  a.workspace = workspace;
  a.device_errors = device_errors;
  a.num_sms = sms;
  a.wait_limit = pa::wait_limit();
  return pa::launch_prefill(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
