// Interface of the prompt attention: its host side and plan (prefill_launch.cu), the
// kernels (prefill_bf16.cu, prefill_f32.cu) and the C ABI (capi_prefill.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace pa {

constexpr int kPrefillKeys = 128;                 // keys of a step
constexpr int kPrefillRows = 256;                 // query rows of an item: two products of 128
constexpr int kPrefillRowsF32 = 64;               // float32 pools
constexpr int kPrefillKeysF32 = 64;
constexpr int kPrefillNoWindow = 1 << 30;

struct PrefillParams {
  CUtensorMap map_k, map_v, map_q;                // bf16 pools
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* starts;
  int32_t* header;                                // [0] tiles in the list
  int2* list;                                     // {sequence, tile}, the longest first
  int room;                                       // entries that the list has room for
  float scale_log2;                               // scale * log2(e): logits in base 2
  int num_seqs, num_tokens, group, group_log2, num_q_heads, num_kv_heads, block_size, block_log2;
  int num_blocks, max_blocks, max_len, window, sinks;
  int32_t* device_errors;
  uint32_t wait_limit;
};

struct PrefillArgs {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* starts;
  float scale;
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_blocks;
  int max_len, window, sinks;
  bool f32;
  void* workspace;
  int32_t* device_errors;
  int num_sms;
  int64_t wait_limit;
};

size_t prefill_workspace_size(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim);
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream);
cudaError_t run_prefill_bf16(int head_dim, const PrefillParams& p, int grid, cudaStream_t stream);
cudaError_t run_prefill_f32(int head_dim, const PrefillParams& p, int grid, cudaStream_t stream);

#ifdef __CUDACC__
// A sequence's part of the call: rows q0 .. q0 + n - 1, the last n of `len` tokens.
struct PrefillSeq {
  int q0, n, len;
};
__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillParams& p, int b) {
  PrefillSeq s;
  const int a = p.starts[b], e = p.starts[b + 1];
  s.q0 = min(max(a, 0), p.num_tokens);
  s.n = (a < 0 || e > p.num_tokens) ? 0 : max(e - s.q0, 0);
  s.len = min(max(p.lens[b], 0), p.max_len);
  return s;
}

// What a tile of rows has to read: keys [0, end) without those that no row sees, as a list
// of steps of KEYS keys; step v starts at key (v + (v >= ns ? shift : 0)) * KEYS.
struct PrefillTile {
  int row0, tokens;                               // first row of q, new tokens of the tile
  int pos0;                                       // the first one's position (may be negative)
  int end;                                        // keys behind the last one that any row sees
  int lo;                                         // first key that the first row's window reaches
  int ns, shift, steps;
};
template <int KEYS>
__device__ __forceinline__ PrefillTile prefill_tile(const PrefillParams& p, const PrefillSeq& s, int tile,
                                                    int tile_tokens) {
  PrefillTile t;
  const int j0 = tile * tile_tokens;
  t.row0 = s.q0 + j0;
  t.tokens = min(tile_tokens, s.n - j0);
  t.pos0 = s.len - s.n + j0;
  t.end = max(0, t.pos0 + t.tokens);
  t.lo = max(0, t.pos0 + 1 - p.window);
  t.ns = (min(p.sinks, t.end) + KEYS - 1) / KEYS;
  t.shift = t.lo / KEYS - t.ns;
  if (t.shift <= 0) t.ns = t.shift = 0;
  t.steps = (t.end + KEYS - 1) / KEYS - t.shift;
  return t;
}
// Item k of CTA c of `ctas`: there and back, so that a CTA's long items and short ones add up.
__device__ __forceinline__ int prefill_item(int k, int c, int ctas) {
  return k * ctas + ((k & 1) ? ctas - 1 - c : c);
}
#endif

}  // namespace pa
