// Interface between the windowed / page-scaled decode's host side (span_launch.cu),
// its kernel instances (span_bf16.cu, span_f32.cu, span_fp8.cu) and the C ABI
// (capi_span.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace pa {

enum class SpanPool { kF32, kBf16, kFp8 };

constexpr int kSpanWarps = 8;                     // consumer warps of a CTA
constexpr int kSpanThreads = (kSpanWarps + 1) * 32;
constexpr int kSpanRing = 8;                      // most stages of a CTA's ring
constexpr int kSpanSmem = 227 * 1024;
constexpr int kSpanCluster = 8;                   // most CTAs that share a sequence in one launch
constexpr int kNoWindow = 1 << 30;

// Tokens that a warp takes from one stage: a tile of 4 KiB of K and 4 KiB of V
// (2 KiB each for bf16 heads of 64).
__host__ __device__ constexpr int span_tile_tokens(SpanPool pool, int head_dim) {
  return pool == SpanPool::kFp8 ? 32 : pool == SpanPool::kBf16 ? 16 : head_dim == 128 ? 8 : 16;
}
__host__ __device__ constexpr int span_row_bytes(SpanPool pool, int head_dim) {
  return head_dim * (pool == SpanPool::kFp8 ? 1 : pool == SpanPool::kBf16 ? 2 : 4);
}
__host__ __device__ constexpr int span_stage_bytes(SpanPool pool, int head_dim) {
  return 2 * kSpanWarps * span_tile_tokens(pool, head_dim) * span_row_bytes(pool, head_dim);
}

// float32: with this many query rows a head's q does not fit the registers (a lane would
// hold rows * head_dim / 8 floats of it).
__host__ __device__ constexpr bool span_q_shared(SpanPool pool, int head_dim, int rows) {
  return pool == SpanPool::kF32 && rows * head_dim / 8 > 64;
}

// Byte offsets of a CTA's shared memory behind its ring of stages.
struct SpanSmem {
  int macc, ml, sc, meta, ps, qs, scan, bars, flag, total;
};
__host__ __device__ constexpr SpanSmem span_smem(SpanPool pool, int head_dim, int rows, int ring) {
  SpanSmem s{};
  int off = ring * span_stage_bytes(pool, head_dim);
  s.macc = off;
  off += kSpanWarps * rows * head_dim * 4;        // a warp's state, handed over to be merged
  s.ml = off;
  off += kSpanWarps * rows * 2 * 4;
  s.sc = off;
  off += pool == SpanPool::kFp8 ? ring * 32 * 4 : 0;
  s.meta = off;
  off += ring * 4;
  off = (off + 15) / 16 * 16;
  s.ps = off;
  off += pool == SpanPool::kF32 ? kSpanWarps * span_tile_tokens(pool, head_dim) * rows * 4 : 0;
  off = (off + 15) / 16 * 16;
  s.qs = off;
  off += span_q_shared(pool, head_dim, rows) ? kSpanWarps * rows * head_dim * 4 : 0;
  s.scan = off;
  off += 16 * 8;
  s.bars = off;
  off += 2 * ring * 8;
  s.flag = off;
  off += 8;
  s.total = (off + 15) / 16 * 16;
  return s;
}

struct SpanParams {
  CUtensorMap map_k, map_v;
  void* out;
  const char* q;
  const int32_t* tables;
  const int32_t* lens;
  const float* k_scales;                          // kFp8: [num_blocks][pool_heads]
  const float* v_scales;
  float scale_log2;                               // scale * log2(e): logits in base 2
  int num_seqs, q_len, group, group_log2, rows, num_q_heads, pool_heads;
  int hg_log2, ngroups;                           // kv heads of a CTA (log2), CTA head groups
  int block_size, num_blocks, max_blocks, max_len, window, sinks;
  int ring;
  int splits;                                     // CTAs of a cluster that share a segment; 0: shares
  uint32_t over_splits;                           // ceil(2^32 / splits): the high word of a product divides
  int joint_slots;                                // clusters: states that a CTA has room for
  float* part_out;                                // shares: [2 CTAs][hg * rows][head_dim]
  float* part_lse;                                // shares: [2 CTAs][hg * rows]
  int32_t* device_errors;
  uint32_t wait_limit;
};

struct SpanArgs {
  SpanPool pool;
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* tables;
  const int32_t* lens;
  const float* k_scales;
  const float* v_scales;
  float scale;
  int num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_blocks;
  int max_len, window, sinks;
  void* workspace;
  int32_t* device_errors;
  int num_sms;
  int64_t wait_limit;
};

size_t span_workspace_size(int rows, int num_kv_heads, int head_dim, int num_sms);
cudaError_t launch_span_decode(const SpanArgs& a, cudaStream_t stream);

// room[n]: the CTAs that clusters of n can have at once on the current device (its processor
// clusters have SMs left over: of 152, 120 for clusters of 8).
void span_cluster_rooms(int num_sms, int (&room)[kSpanCluster + 1]);
cudaError_t run_span_bf16(int head_dim, const SpanParams& p, dim3 grid, int smem, cudaStream_t stream);
cudaError_t run_span_f32(int head_dim, const SpanParams& p, dim3 grid, int smem, cudaStream_t stream);
cudaError_t run_span_fp8(const SpanParams& p, dim3 grid, int smem, cudaStream_t stream);

}  // namespace pa
