// C ABI entry points of the rotating appends: argument checks on the host, then the
// launcher.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/pa.h"
#include "pa_host.h"
#include "pa_rope.h"

namespace {

// What the appends check alike.  Returns PA_OK with nothing to do left in
// num_tokens == 0.
int check(const pa::RopeArgs& a, int elt) {
  if (a.num_tokens < 0 || a.num_q_heads < 0 || a.num_kv_heads <= 0 || a.num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (a.rot_dim < 0 || a.rot_dim > a.head_dim || a.rot_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (a.rot_dim == 0 && a.num_q_heads > 0) return PA_ERR_INVALID_ARG;   // q would only be copied
  if (a.rot_dim > 0 && a.max_position <= 0) return PA_ERR_INVALID_ARG;
  // groups of lanes: at most one for each row (their numbers are 32-bit in the kernels)
  if (static_cast<int64_t>(a.num_tokens) * (a.num_q_heads + 2ll * a.num_kv_heads) > INT32_MAX)
    return PA_ERR_INVALID_ARG;
  if (a.num_tokens == 0) return PA_OK;
  if (!a.k || !a.v || !a.k_cache || !a.v_cache || !a.slots) return PA_ERR_INVALID_ARG;
  if (a.num_q_heads > 0 && (!a.q || !a.q_out)) return PA_ERR_INVALID_ARG;
  if (a.rot_dim > 0 && (!a.positions || !a.cos_sin)) return PA_ERR_INVALID_ARG;
  if (a.positions && a.max_position <= 0) return PA_ERR_INVALID_ARG;
  using pa::aligned16;
  if (!aligned16(a.q) || !aligned16(a.q_out) || !aligned16(a.k) || !aligned16(a.v) ||
      !aligned16(a.k_cache) || !aligned16(a.v_cache) || !aligned16(a.cos_sin))
    return PA_ERR_INVALID_ARG;
  for (const int64_t s : {a.num_q_heads > 0 ? a.q_stride : 0, a.k_stride, a.v_stride})
    if (s < 0 || s * elt % 16 != 0) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

bool shape_ok(int head_dim, int block_size) {
  return (head_dim == 64 || head_dim == 128) && (block_size == 16 || block_size == 32);
}

int run(const pa::RopeArgs& a, int elt, void* stream) {
  const int rc = check(a, elt);
  if (rc != PA_OK || a.num_tokens == 0) return rc;
  return pa::launch_rope_and_cache(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa::RopeArgs args(void* q_out, const void* q, const void* k, const void* v, void* k_cache,
                  void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                  const float* cos_sin, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                  int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rot_dim,
                  int interleaved, int max_position, int block_size, int num_blocks,
                  int32_t* device_errors) {
  pa::RopeArgs a = {};
  a.q_out = q_out;
  a.q = q;
  a.k = k;
  a.v = v;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.slots = slot_mapping;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.interleaved = interleaved != 0;
  a.max_position = max_position;
  a.block_size = block_size;
  a.block_log2 = block_size == 32 ? 5 : 4;
  a.num_blocks = num_blocks;
  a.device_errors = device_errors;
  return a;
}

}  // namespace

extern "C" {

int pa_rope_and_cache(void* q_out, const void* q, const void* k, const void* v, void* k_cache,
                      void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                      const float* cos_sin, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                      int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                      int rot_dim, int interleaved, int max_position, int block_size,
                      int num_blocks, pa_dtype dtype, int32_t* device_errors, void* stream) {
  if ((dtype != PA_F32 && dtype != PA_BF16) || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  pa::RopeArgs a = args(q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_stride,
                        k_stride, v_stride, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        rot_dim, interleaved, max_position, block_size, num_blocks, device_errors);
  a.pool = dtype == PA_F32 ? pa::RopePool::kF32 : pa::RopePool::kBf16;
  return run(a, dtype == PA_F32 ? 4 : 2, stream);
}

int pa_rope_and_cache_fp8(void* q_out, const void* q, const void* k, const void* v, void* k_cache,
                          void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                          const float* cos_sin, const float* k_scale, const float* v_scale,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride, int num_tokens,
                          int num_q_heads, int num_kv_heads, int head_dim, int rot_dim,
                          int interleaved, int max_position, int block_size, int num_blocks,
                          int32_t* device_errors, void* stream) {
  if (head_dim != 128 || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  if (num_tokens > 0 && (!k_scale || !v_scale)) return PA_ERR_INVALID_ARG;
  pa::RopeArgs a = args(q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_stride,
                        k_stride, v_stride, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        rot_dim, interleaved, max_position, block_size, num_blocks, device_errors);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.pool = pa::RopePool::kFp8Head;
  return run(a, 2, stream);
}

int pa_rope_and_cache_fp8_block(void* q_out, const void* q, const void* k, const void* v,
                                void* k_cache, void* v_cache, const int64_t* slot_mapping,
                                const int64_t* positions, const float* cos_sin, float* k_scales,
                                float* v_scales, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, int num_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int rot_dim, int interleaved,
                                int max_position, int block_size, int num_blocks,
                                int32_t* device_errors, void* stream) {
  if (head_dim != 128 || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  if (num_tokens > 0 && (!k_scales || !v_scales)) return PA_ERR_INVALID_ARG;
  pa::RopeArgs a = args(q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_stride,
                        k_stride, v_stride, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        rot_dim, interleaved, max_position, block_size, num_blocks, device_errors);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.pool = pa::RopePool::kFp8Page;
  return run(a, 2, stream);
}

int pa_rope_and_cache_fp4(void* q_out, const void* q, const void* k, const void* v, void* k_cache,
                          void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                          const float* cos_sin, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                          int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                          int rot_dim, int interleaved, int max_position, int block_size,
                          int num_blocks, int32_t* device_errors, void* stream) {
  if (head_dim != 128 || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  pa::RopeArgs a = args(q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_stride,
                        k_stride, v_stride, num_tokens, num_q_heads, num_kv_heads, head_dim,
                        rot_dim, interleaved, max_position, block_size, num_blocks, device_errors);
  a.pool = pa::RopePool::kFp4;
  return run(a, 2, stream);
}

int pa_read_pages_fp4(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                      const int64_t* src_dst_pairs, int num_pairs, int num_kv_heads, int head_dim,
                      int block_size, int num_src_blocks, int num_dst_blocks,
                      int32_t* device_errors, void* stream) {
  if (head_dim != 128 || !shape_ok(head_dim, block_size)) return PA_ERR_UNSUPPORTED;
  if (num_pairs < 0 || num_kv_heads <= 0 || num_src_blocks <= 0 || num_dst_blocks <= 0 ||
      num_kv_heads > pa::kMostReadRows / block_size)
    return PA_ERR_INVALID_ARG;
  if (num_pairs == 0) return PA_OK;
  if (!k_out || !v_out || !k_cache || !v_cache || !src_dst_pairs) return PA_ERR_INVALID_ARG;
  // rows are written 32 bytes at a time
  if (!pa::aligned32(k_out) || !pa::aligned32(v_out) || !pa::aligned16(k_cache) ||
      !pa::aligned16(v_cache))
    return PA_ERR_INVALID_ARG;
  const cudaError_t e = pa::launch_read_pages_fp4(
      k_out, v_out, k_cache, v_cache, src_dst_pairs, num_pairs, num_kv_heads * block_size,
      num_src_blocks, num_dst_blocks, device_errors, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_copy_scales(const float* src_k_scales, const float* src_v_scales, float* dst_k_scales,
                   float* dst_v_scales, const int64_t* src_dst_pairs, int num_pairs,
                   int num_kv_heads, int num_src_blocks, int num_dst_blocks,
                   int32_t* device_errors, void* stream) {
  if (num_pairs < 0 || num_kv_heads <= 0 || num_src_blocks <= 0 || num_dst_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (num_pairs == 0) return PA_OK;
  if (!src_k_scales || !src_v_scales || !dst_k_scales || !dst_v_scales || !src_dst_pairs)
    return PA_ERR_INVALID_ARG;
  const cudaError_t e = pa::launch_copy_scales(
      src_k_scales, src_v_scales, dst_k_scales, dst_v_scales, src_dst_pairs, num_pairs,
      num_kv_heads, num_src_blocks, num_dst_blocks, device_errors, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
