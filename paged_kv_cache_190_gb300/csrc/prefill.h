// Interface of the prompt attention: its host side and plan (prefill_launch.cu), the
// kernels (prefill_bf16.cu, prefill_f32.cu) and the C ABI (capi_prefill.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#include "pa_device.cuh"
#endif

namespace pa {

constexpr int kPrefillKeys = 128;                 // keys of a step
constexpr int kPrefillRows = 256;                 // query rows of an item: two products of 128
constexpr int kPrefillRowsF32 = 32;               // float32 pools: the smaller of their two tiles
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
  int32_t* header;                                // the plan: see prefill_launch.cu
  int4* tiles;                                    // {sequence, tile, steps (at least 1)}, the longest first
  int room;                                       // entries that it has room for
  int4* begin;                                    // shares: {item, its first step, steps} of each CTA
  int may_share, ctas;                            // the host's leave to cut items; CTAs
  int direct;                                     // no plan: CTA i takes item i
  float* part_out;                                // shares: [2 ctas][slot_rows][head_dim]
  float* part_lse;                                // shares: [2 ctas][slot_rows]
  int slot_rows;
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

// Logits are taken in base 2.
inline float prefill_scale_log2(float scale) {
  return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
}
size_t prefill_workspace_size(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                              int num_sms);
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream);
cudaError_t run_prefill_bf16(int head_dim, const PrefillParams& p, int grid, cudaStream_t stream);
cudaError_t run_prefill_f32(int head_dim, int rows, const PrefillParams& p, int grid, cudaStream_t stream);

#ifdef __CUDACC__
// A sequence's part of the call: rows q0 .. q0 + n - 1, the last n of `len` tokens.
struct PrefillSeq {
  int q0, n, len;
};
__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillParams& p, int a, int e, int len) {
  PrefillSeq s;
  s.q0 = min(max(a, 0), p.num_tokens);
  s.n = (a < 0 || e > p.num_tokens) ? 0 : max(e - s.q0, 0);
  s.len = min(max(len, 0), p.max_len);
  return s;
}
__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillParams& p, int b) {
  return prefill_seq(p, p.starts[b], p.starts[b + 1], p.lens[b]);
}
// Is a start, a length, or that there are fewer tokens than new ones an error of the data?
__device__ __forceinline__ bool prefill_bad(const PrefillParams& p, int a, int e, int len) {
  return a < 0 || e < a || e > p.num_tokens || len < 0 || len > p.max_len ||
         prefill_seq(p, a, e, len).n > prefill_seq(p, a, e, len).len;
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
// Item k of CTA c: item i is kv head i % heads of the list's tile i / heads.  Dealt out there and
// back, so that a CTA's long ones and short ones add up.
__device__ __forceinline__ int prefill_deal(int k, int c, int ctas) { return k * ctas + ((k & 1) ? ctas - 1 - c : c); }

// The items of a CTA, one after another: a kv head and a tile of rows, with steps v0 .. v1 - 1
// of its keys; whole ones, and then those of its share.
struct PrefillItem {
  int b, h, v0, v1;
  int slot;                                       // of its partial result, -1: whole
  PrefillTile t;
};
template <int KEYS>
struct PrefillWalk {
  const PrefillParams& p;
  int tile_tokens, items, k, rounds, left;        // left: steps of the share, -1: not begun
  int e;
  __device__ __forceinline__ PrefillWalk(const PrefillParams& p_, int tile_tokens_) : p(p_), tile_tokens(tile_tokens_) {
    k = e = 0;
    if (p.direct) {
      items = left = rounds = 0;
      return;
    }
    items = p.header[0] * p.num_kv_heads;
    left = p.header[1] ? -1 : 0;
    rounds = left ? items / static_cast<int>(gridDim.x) : 1 << 30;
  }
  // What is wrong with sequence b's data, if anything is, goes to the caller's error word.
  __device__ __forceinline__ void look_at(int b) const {
    const int a = p.starts[b], e2 = p.starts[b + 1], len = p.lens[b];
    if (prefill_bad(p, a, e2, len)) report(p.device_errors, PA_DEVERR_BAD_LENGTH);
  }
  // The CTA's only item, found by each warp from the sequences' starts.  One warp of the first
  // CTA looks at every sequence's data, those behind its own item's too.
  __device__ __forceinline__ bool own(PrefillItem& it) {
    if (k++ > 0) return false;
    const int lane = threadIdx.x & 31, tile = blockIdx.x / p.num_kv_heads;
    const bool looks = blockIdx.x == 0 && threadIdx.x < 32;
    int before = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
      PrefillSeq s{0, 0, 0};
      if (b0 + lane < p.num_seqs) {
        s = prefill_seq(p, b0 + lane);
        if (looks) look_at(b0 + lane);
      }
      const int nt = (s.n + tile_tokens - 1) / tile_tokens;
      int x = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t mine = __ballot_sync(0xffffffffu, before + x > tile);
      if (mine) {
        const int l = __ffs(mine) - 1;
        s.q0 = __shfl_sync(0xffffffffu, s.q0, l);
        s.n = __shfl_sync(0xffffffffu, s.n, l);
        s.len = __shfl_sync(0xffffffffu, s.len, l);
        const int t = tile - before - __shfl_sync(0xffffffffu, x - nt, l);
        it.b = b0 + l;
        it.h = blockIdx.x % p.num_kv_heads;
        it.slot = -1;
        it.t = prefill_tile<KEYS>(p, s, t, tile_tokens);
        it.v0 = 0;
        it.v1 = max(1, it.t.steps);
        if (looks)
          for (int b = b0 + 32 + lane; b < p.num_seqs; b += 32) look_at(b);
        return true;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    return false;
  }
  __device__ __forceinline__ bool next(PrefillItem& it) {
    if (p.direct) return own(it);
    int i, n;
    it.slot = -1;
    it.v0 = 0;
    if (k < rounds) {
      i = prefill_deal(k++, blockIdx.x, gridDim.x);
      if (i >= items) return false;               // (no later round has one for this CTA)
      n = 1 << 30;
    } else {
      int slot = 2 * blockIdx.x + 1;
      if (left < 0) {
        const int4 at = p.begin[blockIdx.x];
        e = at.x;
        it.v0 = at.y;
        left = at.z;
        slot = 2 * blockIdx.x;
      }
      if (left <= 0) return false;
      i = e++;
      n = left;
      it.slot = slot;
    }
    const int4 entry = p.tiles[i / p.num_kv_heads];
    it.h = i % p.num_kv_heads;
    it.v1 = entry.z - it.v0 > n ? it.v0 + n : entry.z;
    if (it.slot >= 0) {
      left -= it.v1 - it.v0;
      if (it.v0 == 0 && it.v1 == entry.z) it.slot = -1;
    }
    it.b = entry.x;
    it.t = prefill_tile<KEYS>(p, prefill_seq(p, entry.x), entry.y, tile_tokens);
    return true;
  }
};
#endif

}  // namespace pa
