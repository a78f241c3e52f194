// Host side of the prompt attention: tensor maps, the plan, which lists the tiles of query
// rows and deals them out, and the kernel that joins what shares have cut.
#include <cuda.h>
#include <cuda_bf16.h>
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
//   header: [0] tiles, [1] the steps of a share (0: items stay whole), [2] steps in all
// Few long items do not come out even: where the busiest CTA would take kShareCost steps more
// than its part, all steps are laid end to end and every CTA takes an equal run of them; an
// item that a run's end cuts leaves partial results for prefill_join_kernel (which cost about
// as much as those steps).
constexpr int kWholeRounds = 6;                            // items of a CTA that come out even
constexpr int kShareCost = 12;
constexpr int kMostShared = 1 << 27;                       // keys: steps of all items within 31 bits
constexpr int kLeastShare = 4;                             // steps: less is not worth a partial
template <int KEYS>
__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const PrefillParams p, int tile_rows) {
  __shared__ int most, tiles, count[kPlanBuckets], next[kPlanBuckets], sums[kPlanThreads / 32], busiest;
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
          if (at < p.room) p.list[at] = make_int4(b, t, max(1, prefill_tile<KEYS>(p, s, t, tokens).steps), 0);
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
        if (lane == 31) {
          tiles = min(x, p.room);
          p.header[0] = tiles;
        }
      }
      __syncthreads();
    }
  }
  // ---- shares
  const int heads = p.num_kv_heads, n = tiles;
  const long long items = static_cast<long long>(n) * heads;
  const bool few = p.may_share && n <= kPlanThreads && items < static_cast<long long>(kWholeRounds) * p.ctas;
  if (!few) {
    if (threadIdx.x == 0) p.header[1] = 0;
    return;
  }
  // the steps of the busiest CTA, were the items dealt out whole
  if (threadIdx.x == 0) busiest = 0;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < p.ctas) {
    int sum = 0;
    for (int k = 0; k * p.ctas < items; ++k) {
      const int i = k * p.ctas + ((k & 1) ? p.ctas - 1 - static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x));
      if (i < items) sum += p.list[i / heads].z;
    }
    atomicMax(&busiest, sum);
  }
  const int w = static_cast<int>(threadIdx.x) < n ? p.list[threadIdx.x].z : 0;
  int x = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = x - w, total = 0;
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < warp) before += sums[i];
    total += sums[i];
  }
  total *= heads;
  const int each = max(kLeastShare, (total + p.ctas - 1) / p.ctas);
  const bool share = busiest > each + kShareCost;
  if (threadIdx.x == 0) {
    p.header[1] = share ? each : 0;
    p.header[2] = total;
  }
  if (share && w > 0) {
    const int from = before * heads, to = from + w * heads;
    p.list[threadIdx.x].w = before;
    for (int c = (from + each - 1) / each; c * each < to; ++c)
      p.begin[c] = make_int4(threadIdx.x, (c * each - from) / w, (c * each - from) % w, 0);
  }
}

// The items that shares have cut: block (x, y) has 8 rows of the item that share x ends but
// does not begin, a warp each:  out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M).
constexpr int kJoinWarps = 8;
template <int CPL>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill_join_kernel(const PrefillParams p) {
  constexpr int D = CPL * 32;
  wait_prior_grids();
  allow_next_grid();
  const int share = p.header[1], total = p.header[2], c = blockIdx.x;
  if (share == 0 || c * share >= total) return;
  const int4 at = p.begin[c], entry = p.list[at.x];
  if (at.z == 0 || entry.z - at.z > min(share, total - c * share)) return;   // nothing cut before, or it goes on
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kJoinWarps + warp;
  const int tile_tokens = kPrefillRows >> p.group_log2;
  const PrefillTile t = prefill_tile<kPrefillKeys>(p, prefill_seq(p, entry.x), entry.y, tile_tokens);
  if ((r >> p.group_log2) >= t.tokens) return;
  const int from = (entry.w * p.num_kv_heads) + at.y * entry.z;              // where the item begins
  const int c1 = from / share;
  // a share's first item is its slot 2 c, any other that it leaves unfinished 2 c + 1
  const int first = 2 * c1 + (from == c1 * share ? 0 : 1);
  float M = -3.0e38f, S = 0.f, acc[CPL] = {};
  for (int i = c1; i <= c; ++i) {
    const int64_t row = static_cast<int64_t>(i == c1 ? first : 2 * i) * p.slot_rows + r;
    const float lse = p.part_lse[row];
    float v[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) v[k] = p.part_out[row * D + lane * CPL + k];
    const float mn = fmaxf(M, lse), keep = fast_exp2(M - mn), w = fast_exp2(lse - mn);
    M = mn;
    S = fmaf(S, keep, w);
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = fmaf(acc[k], keep, w * v[k]);
  }
  const float inv = S > 0.f || S != S ? 1.f / S : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
      ((static_cast<int64_t>(t.row0) + (r >> p.group_log2)) * p.num_q_heads + at.y * p.group + (r & (p.group - 1))) * D + lane * CPL);
#pragma unroll
  for (int k = 0; k < CPL / 2; ++k) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    dst[k] = *reinterpret_cast<const uint32_t*>(&b2);
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Tiles that the sequences can have in all.
int64_t most_tiles(int64_t num_tokens, int64_t num_seqs, int group, int tile_rows) {
  return num_tokens * group / tile_rows + std::min(num_seqs, num_tokens);
}

// Offsets of a call's scratch: header, list (room for the smaller tile: enough for every
// type), each CTA's start, the partial results of shares.
struct Scratch {
  size_t list, begin, lse, out, total;
  int slot_rows;
};
Scratch scratch(int64_t num_tokens, int64_t num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int ctas) {
  const int group = num_q_heads / num_kv_heads;
  Scratch s;
  s.slot_rows = static_cast<int>(std::min<int64_t>(kPrefillRows, num_tokens * group));
  s.list = 256;
  s.begin = s.list + align256(16 * static_cast<size_t>(most_tiles(num_tokens, num_seqs, group, kPrefillRowsF32)));
  s.lse = s.begin + align256(16 * static_cast<size_t>(ctas));
  s.out = s.lse + align256(2 * static_cast<size_t>(ctas) * s.slot_rows * 4);
  s.total = s.out + 2 * static_cast<size_t>(ctas) * s.slot_rows * head_dim * 4;
  return s;
}

}  // namespace

size_t prefill_workspace_size(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                              int num_sms) {
  return scratch(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, num_sms).total;
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
  const Scratch at = scratch(a.num_tokens, a.num_seqs, a.num_q_heads, a.num_kv_heads, D, a.num_sms);
  p.list = reinterpret_cast<int4*>(ws + at.list);
  p.begin = reinterpret_cast<int4*>(ws + at.begin);
  p.part_lse = reinterpret_cast<float*>(ws + at.lse);
  p.part_out = reinterpret_cast<float*>(ws + at.out);
  p.slot_rows = at.slot_rows;
  p.ctas = a.num_sms;
  // (cut items only where the sequences may have items too few and long enough for it)
  const int64_t least_items = static_cast<int64_t>(a.num_tokens) * group / kPrefillRows * a.num_kv_heads;
  p.may_share = !a.f32 && a.max_len > kLeastShare * kPrefillKeys && a.max_len <= kMostShared && least_items < static_cast<int64_t>(kWholeRounds) * a.num_sms;
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
  cudaError_t e = a.f32 ? cudaLaunchKernelEx(&cfg, prefill_plan_kernel<kPrefillKeysF32>, p, rows)
                              : cudaLaunchKernelEx(&cfg, prefill_plan_kernel<kPrefillKeys>, p, rows);
  if (e != cudaSuccess) return e;
  const int64_t items = most_tiles(a.num_tokens, a.num_seqs, group, rows) * a.num_kv_heads;
  if (a.f32) return run_prefill_f32(D, p, static_cast<int>(std::min<int64_t>(items, 2 * a.num_sms)), stream);
  e = run_prefill_bf16(D, p, p.may_share ? a.num_sms : static_cast<int>(std::min<int64_t>(items, a.num_sms)), stream);
  if (e != cudaSuccess || !p.may_share) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_sms), static_cast<unsigned>((at.slot_rows + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  return D == 128 ? cudaLaunchKernelEx(&cfg, prefill_join_kernel<4>, p) : cudaLaunchKernelEx(&cfg, prefill_join_kernel<2>, p);
}

}  // namespace pa
