// Host side of the prompt attention: checks of sizes, tensor maps, and the plan, which lists
// the tiles of query rows with the longest first.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "decode_instances.cuh"
#include "pa_device.cuh"
#include "prefill.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 256;

// One block: the tiles of all sequences, sorted by how many steps they take (a counting
// sort over 256 lengths), the longest first: dealt out in turns they then end together.
// Which of two equally long tiles comes first is left open; no result depends on it.
template <int KEYS>
__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const PrefillParams p, int tile_rows) {
  __shared__ int most, count[kPlanBuckets], next[kPlanBuckets];
  wait_prior_grids();
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = tile_rows >> p.group_log2;
  if (threadIdx.x == 0) most = 1;
  if (threadIdx.x < kPlanBuckets) count[threadIdx.x] = 0;
  __syncthreads();
  bool bad = false;
  int longest = 1;
  for (int b = threadIdx.x; b < p.num_seqs; b += kPlanThreads) {
    const PrefillSeq s = prefill_seq(p, b);
    const int a = p.starts[b], e = p.starts[b + 1], len = p.lens[b];
    bad |= a < 0 || e < a || e > p.num_tokens || len < 0 || len > p.max_len || s.n > s.len;
    // (a sequence's last tile has the most steps, but for one more at a window's border)
    if (s.n > 0) longest = max(longest, prefill_tile<KEYS>(p, s, (s.n - 1) / tokens, tokens).steps);
  }
  if (bad) report(p.device_errors, PA_DEVERR_BAD_LENGTH);
  atomicMax(&most, longest);
  __syncthreads();
  auto bucket = [&](int steps) {
    return static_cast<int>(min(static_cast<long long>(kPlanBuckets - 1),
                                static_cast<long long>(steps) * (kPlanBuckets - 1) / most));
  };
  for (int pass = 0; pass < 2; ++pass) {
    for (int b = warp; b < p.num_seqs; b += kPlanThreads / 32) {
      const PrefillSeq s = prefill_seq(p, b);
      for (int t = lane; t * tokens < s.n; t += 32) {
        const int k = kPlanBuckets - 1 - bucket(prefill_tile<KEYS>(p, s, t, tokens).steps);
        if (pass == 0) atomicAdd(&count[k], 1);
        else {
          // (room enough but for q_starts that decrease, whose last tiles are left out)
          const int at = atomicAdd(&next[k], 1);
          if (at < p.room) p.list[at] = make_int2(b, t);
        }
      }
    }
    __syncthreads();
    if (pass == 0) {
      if (threadIdx.x < 32) {                              // where each bucket begins
        int sum = 0;
        for (int i = lane * (kPlanBuckets / 32); i < (lane + 1) * (kPlanBuckets / 32); ++i) sum += count[i];
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        int at = x - sum;
        for (int i = lane * (kPlanBuckets / 32); i < (lane + 1) * (kPlanBuckets / 32); ++i) {
          next[i] = at;
          at += count[i];
        }
        if (lane == 31) p.header[0] = min(x, p.room);
      }
      __syncthreads();
    }
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Tiles that the sequences can have in all.
int64_t most_tiles(int64_t num_tokens, int64_t num_seqs, int group, int tile_rows) {
  return num_tokens * group / tile_rows + std::min(num_seqs, num_tokens);
}

}  // namespace

size_t prefill_workspace_size(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int) {
  // (the smaller tile: enough for every type)
  return 256 + align256(8 * static_cast<size_t>(most_tiles(num_tokens, num_seqs, num_q_heads / num_kv_heads,
                                                           kPrefillRowsF32)));
}

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
  PrefillParams p;
  std::memset(&p, 0, sizeof(p));
  const int group = a.num_q_heads / a.num_kv_heads, D = a.head_dim;
  p.out = a.out;
  p.q = a.q;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.tables = a.tables;
  p.lens = a.lens;
  p.starts = a.starts;
  char* ws = static_cast<char*>(a.workspace);
  p.header = reinterpret_cast<int32_t*>(ws);
  p.list = reinterpret_cast<int2*>(ws + 256);
  p.room = static_cast<int>(most_tiles(a.num_tokens, a.num_seqs, group, a.f32 ? kPrefillRowsF32 : kPrefillRows));
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.group = group;
  p.group_log2 = group >= 8 ? 3 : group >= 4 ? 2 : group >= 2 ? 1 : 0;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.block_size = a.block_size;
  p.block_log2 = a.block_size == 32 ? 5 : 4;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.max_len = a.max_len;
  p.window = a.window > 0 && a.window < kPrefillNoWindow ? a.window : kPrefillNoWindow;
  p.sinks = a.window > 0 ? std::min(a.sinks, a.max_len) : 0;
  p.device_errors = a.device_errors;
  p.wait_limit = a.wait_limit < 0 ? kMaxPolls : static_cast<uint32_t>(a.wait_limit);
  if (!a.f32) {
    // the pools as {64 columns, token of the page, page and head, slab of 64 columns}; q as
    // {columns, head of the group, kv head, token}
    const uint64_t pages = static_cast<uint64_t>(a.num_blocks) * a.num_kv_heads, row = 2ull * D;
    const uint64_t dims[4] = {64, static_cast<uint64_t>(a.block_size), pages, static_cast<uint64_t>(D / 64)};
    const uint64_t strides[3] = {row, row * a.block_size, 128};
    const uint32_t k_box[4] = {64, static_cast<uint32_t>(a.block_size), 1, 1};
    const uint32_t v_box[4] = {64, static_cast<uint32_t>(a.block_size), 1, static_cast<uint32_t>(D / 64)};
    cudaError_t e = make_bf16_map(&p.map_k, a.k_cache, 4, dims, strides, k_box);
    if (e == cudaSuccess) e = make_bf16_map(&p.map_v, a.v_cache, 4, dims, strides, v_box);
    const uint64_t q_dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(group),
                                static_cast<uint64_t>(a.num_kv_heads), static_cast<uint64_t>(a.num_tokens)};
    const uint64_t q_strides[3] = {row, row * group, row * a.num_q_heads};
    const uint32_t q_box[4] = {64, static_cast<uint32_t>(group), 1, static_cast<uint32_t>(128 / group)};
    if (e == cudaSuccess) e = make_bf16_map(&p.map_q, a.q, 4, q_dims, q_strides, q_box);
    if (e != cudaSuccess) return e;
  }
  const int rows = a.f32 ? kPrefillRowsF32 : kPrefillRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.f32 ? cudaLaunchKernelEx(&cfg, prefill_plan_kernel<kPrefillKeysF32>, p, rows)
                              : cudaLaunchKernelEx(&cfg, prefill_plan_kernel<kPrefillKeys>, p, rows);
  if (e != cudaSuccess) return e;
  const int64_t items = most_tiles(a.num_tokens, a.num_seqs, group, rows) * a.num_kv_heads;
  const int64_t resident = static_cast<int64_t>(a.num_sms) * (a.f32 ? 2 : 1);
  const int grid = static_cast<int>(std::min(items, resident));
  return a.f32 ? run_prefill_f32(D, p, grid, stream) : run_prefill_bf16(D, p, grid, stream);
}

}  // namespace pa
