// Launcher interface of the rotating appends (rope_cache.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace pa {

enum class RopePool { kF32, kBf16, kFp8Head, kFp8Page, kFp4 };

struct RopeArgs {
  void* q_out;                 // [num_tokens][num_q_heads][head_dim], contiguous
  const void* q;               // token strides in elements
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  void* k_cache;
  void* v_cache;
  const int64_t* slots;
  const int64_t* positions;    // null with rot_dim 0: every token is live
  const float* cos_sin;        // [max_position][rot_dim]
  const float* k_scale;        // kFp8Head: [num_kv_heads]
  const float* v_scale;
  float* k_scales;             // kFp8Page: [num_blocks][num_kv_heads]
  float* v_scales;
  int num_tokens, num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved;
  int max_position, block_size, block_log2, num_blocks;
  RopePool pool;
  int32_t* device_errors;
};

cudaError_t launch_rope_and_cache(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_copy_scales(const float* src_k, const float* src_v, float* dst_k, float* dst_v,
                               const int64_t* pairs, int num_pairs, int num_kv_heads, int num_src,
                               int num_dst, int32_t* device_errors, cudaStream_t stream);
// Pages of 4-bit rows as bf16 pages (read_pages.cu).  A grid has 65535 parts of a page at the most.
constexpr int kReadPartRows = 32;
constexpr int kMostReadRows = 65535 * kReadPartRows;
cudaError_t launch_read_pages_fp4(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                                  const int64_t* pairs, int num_pairs, int page_rows, int num_src,
                                  int num_dst, int32_t* device_errors, cudaStream_t stream);

}  // namespace pa
