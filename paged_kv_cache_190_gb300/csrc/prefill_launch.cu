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

constexpr int kPlanBuckets = 256;
constexpr int kPlanSeqs = 1024, kPlanTiles = 1536;          // kept in shared memory

template <int CPL>
__device__ __forceinline__ void load_cols(const float* p, float* v) {
  if constexpr (CPL == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(p);
    v[0] = t.x; v[1] = t.y;
  }
}

// Exclusive sum of a block's values; `all` is their sum in every thread.
template <int THREADS>
__device__ __forceinline__ int block_before(int x, int* sums, int& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();                                         // (the last sums have been read)
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  int before = y - x;
  all = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) before += sums[i];
    all += sums[i];
  }
  return before;
}

// Sum of a warp's numbers, or `cap` if that is less.
__device__ __forceinline__ uint32_t capped_sum(uint32_t x, uint32_t cap) {
  const uint32_t high = __reduce_add_sync(0xffffffffu, x >> 16), low = __reduce_add_sync(0xffffffffu, x & 0xffffu);
  const uint64_t sum = (static_cast<uint64_t>(high) << 16) + low;
  return sum < cap ? static_cast<uint32_t>(sum) : cap;
}

// One block: the tiles of all sequences, sorted by how many steps they take (a counting
// sort over 256 lengths), the longest first: dealt out in turns they then end together.
//   header: [0] tiles, [1] whether there are shares
// Starts that decrease let sequences claim the same rows, and so more tiles than the rows have:
// such a call is left out (its tiles in all may pass 31 bits, and this block would list them for
// minutes).  Starts that do not decrease never come to more than p.room.
// Whole items are dealt out in rounds.  Where the busiest CTA would take kShareCost steps more
// than its part that way, the items of the last, incomplete round are laid end to end and each
// CTA takes a run of them that makes up for what it has less than the others; an item that a
// run's end cuts leaves partial results for prefill_join_kernel (which cost about as much as
// those steps).  6 chunks behind up to 15000 tokens take 248 us this way, 318 in whole items
// alone; 64 tokens behind 8000 36.7 and 98.7, 12 chunks of 300 behind 3000 168 and 183.  The leave
// to cut costs the plan and the join where nothing is cut in the end: 20 chunks of 256 behind 1000
// 105.0, without it 101.8; one prompt of 600 tokens 20.2, and 13.9 where it needs no plan either.
// (Shares of all items even out no better, and the tiles of one sequence and head,
// which whole rounds read together, then read their keys from HBM again and again: 1.1 GB
// and 260 us in the kernel alone where this reads 0.3 GB in 240.)
constexpr int kShareCost = 12;
constexpr int kMostRounds = 8;                             // (at most kPlanTiles tiles then)
constexpr int kMostShared = 1 << 27;                       // keys: steps of all items within 31 bits
constexpr int kLeastShare = 4;                             // steps: less is not worth a partial
template <int KEYS, int THREADS>
__global__ void __launch_bounds__(THREADS) prefill_plan_kernel(const PrefillParams p, int tile_rows) {
  __shared__ int most, count[kPlanBuckets], next[kPlanBuckets], sums[THREADS / 32], busiest;
  __shared__ uint32_t claimed[THREADS / 32];               // tiles of the sequences of each warp
  __shared__ int item_from[THREADS];
  __shared__ PrefillSeq seqs[kPlanSeqs];
  __shared__ int2 unsorted[kPlanTiles];
  __shared__ int sorted[kPlanTiles];                       // steps
  allow_next_grid();
  const int me = threadIdx.x, warp = me >> 5, lane = me & 31;
  const int tokens = tile_rows >> p.group_log2;
  if (me == 0) most = 1;
  if (me < kPlanBuckets) count[me] = 0;
  wait_prior_grids();
  __syncthreads();
  bool bad = false;
  int longest = 1;
  const uint32_t too_many = static_cast<uint32_t>(p.room) + 1;   // (below 2^31: where sums stop)
  uint32_t claims = 0;
  for (int b = me; b < p.num_seqs; b += THREADS) {
    const int a = p.starts[b], e = p.starts[b + 1], len = p.lens[b];
    const PrefillSeq s = prefill_seq(p, a, e, len);
    if (b < kPlanSeqs) seqs[b] = s;
    bad |= prefill_bad(p, a, e, len);
    // (a sequence's last tile has the most steps, but for one more at a window's border)
    if (s.n > 0) longest = max(longest, prefill_tile<KEYS>(p, s, (s.n - 1) / tokens, tokens).steps);
    claims = min(claims + static_cast<uint32_t>((s.n + tokens - 1) / tokens), too_many);
  }
  if (bad) report(p.device_errors, PA_DEVERR_BAD_LENGTH);
  longest = __reduce_max_sync(0xffffffffu, longest);
  claims = capped_sum(claims, too_many);
  if (lane == 0) {
    atomicMax(&most, longest);
    claimed[warp] = claims;
  }
  __syncthreads();
  if (capped_sum(lane < THREADS / 32 ? claimed[lane] : 0u, too_many) == too_many) {
    if (me < 2) p.header[me] = 0;
    return;
  }
  const float buckets = static_cast<float>(kPlanBuckets - 1) / static_cast<float>(most);
  auto bucket = [&](int steps) { return kPlanBuckets - 1 - min(kPlanBuckets - 1, static_cast<int>(static_cast<float>(steps) * buckets)); };
  auto tiles_do = [&](auto f) {                            // f(sequence, tile, steps) for all tiles
    for (int b = warp; b < p.num_seqs; b += THREADS / 32) {
      const PrefillSeq s = b < kPlanSeqs ? seqs[b] : prefill_seq(p, b);
      for (int t = lane; t * tokens < s.n; t += 32) f(b, t, prefill_tile<KEYS>(p, s, t, tokens).steps);
    }
  };
  tiles_do([&](int, int, int steps) { atomicAdd(&count[bucket(steps)], 1); });
  __syncthreads();
  int tiles;
  const int before = block_before<THREADS>(me < kPlanBuckets ? count[me] : 0, sums, tiles);   // where each bucket begins
  if (me < kPlanBuckets) next[me] = before;
  if (me == 0) p.header[0] = tiles;
  __syncthreads();
  const bool here = tiles <= kPlanTiles;
  tiles_do([&](int b, int t, int steps) {
    const int at = atomicAdd(&next[bucket(steps)], 1);
    if (here) unsorted[at] = make_int2(b, t);
    else p.tiles[at] = make_int4(b, t, max(1, steps), 0);
  });
  __syncthreads();
  // (which of the tiles of a bucket came first is chance, and shares cut items by their place:
  // in the order of their numbers, so that a call's result is always the same)
  if (here)
    for (int i = me; i < tiles; i += THREADS) {
      const int2 x = unsorted[i];
      const PrefillSeq s = x.x < kPlanSeqs ? seqs[x.x] : prefill_seq(p, x.x);
      const int steps = prefill_tile<KEYS>(p, s, x.y, tokens).steps;
      const int k = bucket(steps), end = next[k], begin = end - count[k];
      int at = begin;
      for (int j = begin; j < end; ++j) {
        const int2 y = unsorted[j];
        at += y.x < x.x || (y.x == x.x && y.y < x.y) ? 1 : 0;
      }
      sorted[at] = max(1, steps);
      p.tiles[at] = make_int4(x.x, x.y, max(1, steps), 0);
    }
  __syncthreads();
  // ---- what comes out uneven goes out in shares
  const int heads = p.num_kv_heads, ctas = p.ctas;
  const long long items = static_cast<long long>(tiles) * heads;
  const int rounds = static_cast<int>(items / ctas), whole = rounds * ctas, rest = static_cast<int>(items) - whole;
  if (!p.may_share || !here || items > static_cast<long long>(kMostRounds) * ctas) {
    if (me == 0) p.header[1] = 0;
    return;
  }
  if (me == 0) busiest = 0;
  __syncthreads();
  int mine = 0;                                            // steps of CTA `me`'s whole items
  if (me < ctas) {
    int last = 0;
    for (int k = 0; k <= rounds; ++k) {
      const int i = prefill_deal(k, me, ctas);
      const int steps = i < items ? sorted[i / heads] : 0;
      if (k < rounds) mine += steps; else last = steps;
    }
    atomicMax(&busiest, mine + last);
  }
  const int w = me < rest ? sorted[(whole + me) / heads] : 0;
  int rest_steps, whole_steps, all_room;
  const int from = block_before<THREADS>(w, sums, rest_steps);
  block_before<THREADS>(mine, sums, whole_steps);
  const int each = (rest_steps + whole_steps + ctas - 1) / ctas;
  const bool share = busiest > each + kShareCost;
  if (me == 0) p.header[1] = share ? 1 : 0;
  if (!share) return;
  // CTA `me` has room for so many steps of the rest (rooms under kLeastShare are left out:
  // the others' are larger by that)
  int room = me < ctas ? max(0, each + kLeastShare - mine) : 0;
  if (room < kLeastShare) room = 0;
  const int at = block_before<THREADS>(room, sums, all_room);
  if (me < rest) item_from[me] = from;
  __syncthreads();
  if (me < ctas) {
    int lo = 0, hi = rest - 1;                             // the last item that begins at or before `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (item_from[mid] <= at) lo = mid; else hi = mid - 1;
    }
    p.begin[me] = make_int4(whole + lo, at - item_from[lo], max(0, min(room, rest_steps - at)), 0);
  }
}

// The items that shares have cut: block (c, y) has 16 rows of the item that CTA c ends but does
// not begin, one after another a warp:  out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M).
constexpr int kJoinWarps = 8, kJoinRows = 16;
template <int CPL>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill_join_kernel(const PrefillParams p) {
  constexpr int D = CPL * 32;
  wait_prior_grids();
  allow_next_grid();
  if (p.header[1] == 0) return;
  const int c = blockIdx.x;
  const int4 at = p.begin[c];
  if (at.z == 0 || at.y == 0) return;                      // no share, or it begins with an item
  const int4 entry = p.tiles[at.x / p.num_kv_heads];
  if (entry.z - at.y > at.z) return;                       // the item goes on
  const int h = at.x % p.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_tokens = kPrefillRows >> p.group_log2;
  const PrefillTile t = prefill_tile<kPrefillKeys>(p, prefill_seq(p, entry.x), entry.y, tile_tokens);
  for (int r = blockIdx.y * kJoinRows + warp; r < (blockIdx.y + 1) * kJoinRows; r += kJoinWarps) {
    if ((r >> p.group_log2) >= t.tokens) return;
    float M = -3.0e38f, S = 0.f, acc[CPL] = {};
    // partials of up to 32 CTAs at a time, c itself and those before it
    for (int back = c; back >= 0; back -= 32) {
      const int cc = back - lane;
      int4 b = make_int4(-1, 0, 0, 0);
      if (cc >= 0) b = p.begin[cc];
      const bool has = b.z > 0, same = b.x == at.x;
      // (a share that begins with another item has this one as its last)
      const uint32_t ends = __ballot_sync(0xffffffffu, has && (!same || b.y == 0));
      const int n = ends ? __ffs(ends) : 32;
      const bool in = has && lane < n;
      const int64_t row = static_cast<int64_t>(2 * cc + (same ? 0 : 1)) * p.slot_rows + r;
      const float lse = in ? p.part_lse[row] : -INFINITY;
      float mx = lse;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(M, mx), keep = fast_exp2(M - mn), f = in ? fast_exp2(lse - mn) : 0.f;
      float sum = f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      M = mn;
      S = fmaf(S, keep, sum);
#pragma unroll
      for (int k = 0; k < CPL; ++k) acc[k] *= keep;
      uint32_t todo = __ballot_sync(0xffffffffu, in);
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        if (!((todo >> j) & 1u)) continue;
        const int64_t rj = __shfl_sync(0xffffffffu, row, j);
        const float fj = __shfl_sync(0xffffffffu, f, j);
        float v[CPL];
        load_cols<CPL>(p.part_out + rj * D + lane * CPL, v);
#pragma unroll
        for (int k = 0; k < CPL; ++k) acc[k] = fmaf(fj, v[k], acc[k]);
      }
      if (ends) break;
    }
    const float inv = S > 0.f || S != S ? 1.f / S : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
        ((static_cast<int64_t>(t.row0) + (r >> p.group_log2)) * p.num_q_heads + h * p.group + (r & (p.group - 1))) * D + lane * CPL);
#pragma unroll
    for (int k = 0; k < CPL / 2; ++k) {
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
      dst[k] = *reinterpret_cast<const uint32_t*>(&b2);
    }
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
  size_t tiles, begin, lse, out, total;
  int slot_rows;
};
Scratch scratch(int64_t num_tokens, int64_t num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int ctas) {
  const int group = num_q_heads / num_kv_heads;
  Scratch s;
  s.slot_rows = static_cast<int>(std::min<int64_t>(kPrefillRows, num_tokens * group));
  s.tiles = 256;
  s.begin = s.tiles + align256(16 * static_cast<size_t>(most_tiles(num_tokens, num_seqs, group, kPrefillRowsF32)));
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
  p.tiles = reinterpret_cast<int4*>(ws + at.tiles);
  p.begin = reinterpret_cast<int4*>(ws + at.begin);
  p.part_lse = reinterpret_cast<float*>(ws + at.lse);
  p.part_out = reinterpret_cast<float*>(ws + at.out);
  p.slot_rows = at.slot_rows;
  p.ctas = a.num_sms;
  // (cut items only where the sequences may have items too few and long enough for it)
  const int64_t least_items = static_cast<int64_t>(a.num_tokens) * group / kPrefillRows * a.num_kv_heads;
  p.may_share = !a.f32 && a.max_len > kLeastShare * kPrefillKeys && a.max_len <= kMostShared && least_items <= static_cast<int64_t>(kMostRounds) * a.num_sms &&
                a.num_sms * kMostRounds <= kPlanTiles;
  // float32: tiles of 64 rows, of 32 where two of those an SM are more than there are (5 short
  // prompts 23.0 us, with tiles of 64 31.9; a tile of 64 reads its keys half as often).  8 heads of
  // 64, tiles of 32 and 64: one prompt of 100 tokens 11.0 and 13.9, 10 of 120 20.0 and 21.8, 10 of
  // 240 46.6 and 41.4, 20 of 240 86.4 and 62.7; 5 of 110, on the wrong side of it, 16.4 and 14.3
  const int rows = !a.f32 ? kPrefillRows
      : most_tiles(a.num_tokens, a.num_seqs, group, 64) * a.num_kv_heads > 2 * a.num_sms ? 64 : kPrefillRowsF32;
  p.room = static_cast<int>(most_tiles(a.num_tokens, a.num_seqs, group, rows));
  p.scale_log2 = prefill_scale_log2(a.scale);
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
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int64_t items = most_tiles(a.num_tokens, a.num_seqs, group, rows) * a.num_kv_heads;
  // one item a CTA at most, and none long enough to be cut: each CTA finds its own, without
  // a plan (37 tokens of one prompt 6.3 us, 9.0 with one; 512 tokens 12.0 and 14.7, 2 of 500 12.5
  // and 15.4; float32, 4 of 64 19.7 and 22.6)
  p.direct = !p.may_share && items <= (a.f32 ? 2 : 1) * a.num_sms;
  cudaError_t e = cudaSuccess;
  if (!p.direct) {
    // (the steps of a plan are barriers of its block: 251 us against 248 for 6 chunks with 1024
    // threads, 397 against 381 for 4 prompts of 4096; more sequences or tiles want them, from
    // fewer on than this: 250 sequences of 20 tokens behind 700 take 188 us here, 181 with 1024)
    const bool small = a.num_seqs <= 256 && most_tiles(a.num_tokens, a.num_seqs, group, rows) <= 1024 && a.num_sms <= 256;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(small ? 256 : 1024);
    auto plan = a.f32 ? (small ? prefill_plan_kernel<kPrefillKeysF32, 256> : prefill_plan_kernel<kPrefillKeysF32, 1024>)
                      : (small ? prefill_plan_kernel<kPrefillKeys, 256> : prefill_plan_kernel<kPrefillKeys, 1024>);
    e = cudaLaunchKernelEx(&cfg, plan, p, rows);
    if (e != cudaSuccess) return e;
  }
  if (a.f32) return run_prefill_f32(D, rows, p, static_cast<int>(std::min<int64_t>(items, 2 * a.num_sms)), stream);
  e = run_prefill_bf16(D, p, p.may_share ? a.num_sms : static_cast<int>(std::min<int64_t>(items, a.num_sms)), stream);
  if (e != cudaSuccess || !p.may_share) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_sms), static_cast<unsigned>((at.slot_rows + kJoinRows - 1) / kJoinRows));
  cfg.blockDim = dim3(kJoinWarps * 32);
  return D == 128 ? cudaLaunchKernelEx(&cfg, prefill_join_kernel<4>, p) : cudaLaunchKernelEx(&cfg, prefill_join_kernel<2>, p);
}

}  // namespace pa
