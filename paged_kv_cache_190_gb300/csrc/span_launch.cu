// Host side of the windowed / page-scaled decode: how a call is spread over the GPU,
// the tensor maps, and the kernel that joins segments cut by a share's end.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include "pa_device.cuh"
#include "span_list.cuh"

namespace pa {
namespace {

constexpr int kJoinWarps = 8;

template <int CPL>
__device__ __forceinline__ void load_part(const float* p, float* v) {
  if constexpr (CPL == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(p);
    v[0] = t.x; v[1] = t.y;
  }
}

// A segment cut into n partials: out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M).
// Block (x, y): BY_SEGMENT, segment x (no more of them than shares); else the segment that
// share x ends but does not begin.  WIDE, row y by 8 warps that take partials in turn (few
// segments: each spans many shares); else 8 rows, a warp each.  Where the cuts are follows
// from the lengths and is worked out before the wait for the attention kernel: that one
// lets this grid start once its own inputs are complete.  After it a lane holds a partial's
// weight, 32 partials at a time, so that all their rows are on their way together.
template <int TU, bool BF16, int CPL, bool BY_SEGMENT, bool WIDE>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) span_join_kernel(const SpanParams p, int ctas) {
  constexpr int D = CPL * 32;
  __shared__ float sm[kJoinWarps], ss[kJoinWarps];
  __shared__ float sacc[WIDE ? kJoinWarps : 1][D];
  __shared__ long long sums[kJoinWarps], found[2];
  __shared__ int where[2];
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // stages before each thread's run of sequences, and in all
  const int per = (p.num_seqs + kJoinWarps * 32 - 1) / (kJoinWarps * 32);
  const int s0 = min(static_cast<int>(threadIdx.x) * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
  long long sum = 0;
  for (int b = s0; b < s1; ++b) sum += span::make_span<TU>(p, p.lens[b]).nst;
  long long x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  if (threadIdx.x == 0) where[0] = -1;
  __syncthreads();
  long long before = x - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  total *= p.ngroups;
  before *= p.ngroups;
  const long long share = span::share_of(total, ctas);
  const long long at = share * blockIdx.x;                   // where share x begins
  for (int b = s0; b < s1; ++b) {
    const int nst = span::make_span<TU>(p, p.lens[b]).nst;
    const long long n = static_cast<long long>(nst) * p.ngroups;
    int grp = -1;
    if (BY_SEGMENT)
      grp = static_cast<int>(blockIdx.x) / p.ngroups == b ? static_cast<int>(blockIdx.x) % p.ngroups : -1;
    else if (before <= at && at < before + n)
      grp = static_cast<int>((at - before) / nst);
    if (grp >= 0) {
      where[0] = b;
      where[1] = grp;
      found[0] = before + static_cast<long long>(grp) * nst;
      found[1] = found[0] + nst;
    }
    before += n;
  }
  __syncthreads();
  // the share in which the segment ends, and the one in which it began
  const int c = BY_SEGMENT ? static_cast<int>((found[1] - 1) / share) : static_cast<int>(blockIdx.x);
  const bool mine = where[0] >= 0 && found[1] <= share * (c + 1) && found[0] < share * c;
  wait_prior_grids();
  if (!mine) return;
  const int R = p.rows << p.hg_log2;
  const int r = WIDE ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y) * kJoinWarps + warp;
  if (r >= R) return;                                        // (never with WIDE)
  const int c1 = static_cast<int>(found[0] / share), n = c - c1 + 1;
  // a share's first partial is its entry 2 c; its last segment's, if that is another one, 2 c + 1
  const int first = 2 * c1 + (found[0] == share * c1 ? 0 : 1);
  auto row_of = [&](int i) { return static_cast<int64_t>(i == 0 ? first : 2 * (c1 + i)) * R + r; };
  constexpr int STEP = WIDE ? kJoinWarps : 1;
  float M = -3.0e38f, S = 0.f, acc[CPL] = {};
  for (int i0 = WIDE ? warp : 0; i0 < n; i0 += 32 * STEP) {
    const int mine = i0 + lane * STEP;
    const float lse = mine < n ? p.part_lse[row_of(mine)] : -INFINITY;
    float mx = lse;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(M, mx);
    const float keep = fast_exp2(M - mn), w = fast_exp2(lse - mn);
    float sum = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    S = fmaf(S, keep, sum);
    M = mn;
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] *= keep;
    const int m = min(32, (n - i0 + STEP - 1) / STEP);
#pragma unroll 8
    for (int j = 0; j < m; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      float v[CPL];
      load_part<CPL>(p.part_out + row_of(i0 + j * STEP) * D + lane * CPL, v);
#pragma unroll
      for (int k = 0; k < CPL; ++k) acc[k] = fmaf(wj, v[k], acc[k]);
    }
  }
  if constexpr (WIDE) {
    if (lane == 0) {
      sm[warp] = M;
      ss[warp] = S;
    }
#pragma unroll
    for (int k = 0; k < CPL; ++k) sacc[warp][lane * CPL + k] = acc[k];
    __syncthreads();
    if (warp != 0) return;
    M = sm[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) M = fmaxf(M, sm[w]);
    S = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = fast_exp2(sm[w] - M);
      S = fmaf(f, ss[w], S);
#pragma unroll
      for (int k = 0; k < CPL; ++k) acc[k] = fmaf(f, sacc[w][lane * CPL + k], acc[k]);
    }
  }
  const float inv = S > 0.f || S != S ? 1.f / S : 0.f;
  const int head = (where[1] << p.hg_log2) + r / p.rows, row = r % p.rows;
  const int64_t o = ((static_cast<int64_t>(where[0]) * p.q_len + (row >> p.group_log2)) * p.num_q_heads +
                     head * p.group + (row & (p.group - 1))) * D + lane * CPL;
  if constexpr (BF16) {
    uint32_t w[CPL / 2];
#pragma unroll
    for (int k = 0; k < CPL / 2; ++k) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
      w[k] = *reinterpret_cast<const uint32_t*>(&t);
    }
    uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + o);
    if constexpr (CPL == 4) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
    else *d = w[0];
  } else {
    float* d = static_cast<float*>(p.out) + o;
#pragma unroll
    for (int k = 0; k < CPL; ++k) d[k] = acc[k] * inv;
  }
}

template <int TU, bool BF16, int CPL>
cudaError_t launch_join(const SpanParams& p, int64_t segments, int ctas, cudaStream_t stream) {
  const int R = p.rows << p.hg_log2;
  const bool by_segment = segments <= ctas;
  const bool wide = segments * 16 <= ctas;                   // each segment is cut into many partials
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(by_segment ? segments : ctas),
                     static_cast<unsigned>(wide ? R : (R + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide         ? cudaLaunchKernelEx(&cfg, span_join_kernel<TU, BF16, CPL, true, true>, p, ctas)
         : by_segment ? cudaLaunchKernelEx(&cfg, span_join_kernel<TU, BF16, CPL, true, false>, p, ctas)
                      : cudaLaunchKernelEx(&cfg, span_join_kernel<TU, BF16, CPL, false, false>, p, ctas);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// A pool as {128 bytes of a row (f32: the row), token of the page, page and head, slab},
// in boxes of box_tokens tokens of hg heads with every slab of their rows.
cudaError_t make_map(CUtensorMap* map, const void* pool, SpanPool kind, int head_dim, int block_size,
                     int64_t head_pages, int box_tokens, int hg) {
  const auto encode = encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const int elt = kind == SpanPool::kFp8 ? 1 : kind == SpanPool::kBf16 ? 2 : 4;
  const int row = head_dim * elt;
  const bool f32 = kind == SpanPool::kF32;
  const int inner = f32 ? head_dim : 128 / elt;
  const int slabs = f32 ? 1 : row / 128;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(block_size),
                              static_cast<cuuint64_t>(head_pages), static_cast<cuuint64_t>(slabs)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(row) * block_size, 128};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), static_cast<cuuint32_t>(box_tokens),
                             static_cast<cuuint32_t>(hg), static_cast<cuuint32_t>(slabs)};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = kind == SpanPool::kFp8    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : kind == SpanPool::kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = encode(map, type, slabs > 1 ? 4 : 3, const_cast<void*>(pool), dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, f32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Heads that a CTA takes together: the largest power of two up to `most` that divides them.
int heads_together(int num_kv_heads, int most) {
  int hg = most;
  while (num_kv_heads % hg) hg /= 2;
  return hg;
}

// In shares, up to 8 (e4m3) or 2.  Boxes under 8 KiB cost the copy engine more than their
// bytes: e4m3 pages of 16 tokens, 885 MB, take 144 us with 8 heads a box (16 KiB), 152 with
// 4, 171 with 2, 213 with 1.  bf16 rows are twice as long, and with 2 heads a segment leaves
// a quarter of the partials: 129.4 us against 132.2 with 8 (833 MB), 49.5 against 52.0
// (269 MB, 8 rows a head).
int share_heads(SpanPool pool, int num_kv_heads) {
  return heads_together(num_kv_heads, pool == SpanPool::kFp8 ? 8 : 2);
}

// Room for the states that a CTA of a cluster joins.
int joint_bytes(int head_dim, int rows, int hg, int splits) {
  return splits > 1 ? (hg * rows + splits) * (head_dim + 2) * 4 : 0;
}
// Stages that the shared memory has room for.
int ring_stages(SpanPool pool, int head_dim, int rows, int hg, int splits) {
  const int room = kSpanSmem - 1024 - span_smem(pool, head_dim, rows, 0).total - joint_bytes(head_dim, rows, hg, splits);
  return std::min<int>(kSpanRing, room / (span_stage_bytes(pool, head_dim) + 160));
}

// How a call is spread, by what was measured for 1 to 64 sequences of 256 to 4096 tokens
// (8 kv heads, pages of 16; in 10 ns): a CTA takes its start and so much a stage, more where
// its boxes are small; joining a cluster's states takes longer the more of them there are;
// and no stage of all SMs takes less than HBM does.  Shares start later (a pass over the
// lengths, a second kernel) but spread evenly, while a cluster ends with its sequence: the
// caller's bound is the longest sequence's, so lengths that no window evens out are taken
// to be 0.7 of it in the mean.  (us, clusters and shares, e4m3: 1 sequence of 256 tokens
// 5.1 and 7.6, 4 of 1024 6.4 and 10.1, 16 of 2048 14.5 and 18.8, 64 of 2048 to 4096 88 and
// 72; bf16: 4 of 4096 10.7 and 13.4, 16 windows of 4096 44.4 and 49.5, 64 of 256 9.9 and 14.2.)
// Clusters of any size up to 8, not of powers of two alone (e4m3: 10 sequences of 1024 8.8 us
// in clusters of 3, 9.9 without; 12 of 2048 13.4 in 5s, 14.5; bf16: 10 of 1024 8.9 and 10.3).
// float32 rows are computed one by one: with 1, 4 and 8 of them a stage takes 0.93, 1.13 and
// 1.50 us (one head a CTA), 0.66, 0.87 and 1.35 (8 heads).  Nothing is chosen that leaves the
// ring a single stage (8 such heads of 8 rows in clusters: 130 us, where 2 stages take 90).
// More short sequences than SMs: the end of a segment takes a CTA of the shares 1.7 us (one
// head of one row) to 7 (8 of 8), which long ones hide behind their copies; so more heads a segment, or a CTA
// for each segment, one after another on an SM (bf16, 8 kv heads: 232 sequences of 10 to 36
// tokens, 8 rows, 12.1 us so, in shares 25.5 with 2 heads and 19.3 with 8; 512 of 20 to 40
// 22.6, 33.9 and 21.5; 160 of 1000 135, 109.4 and 109.3).
struct Spread {
  int hg = 0, splits = 0;                                    // splits 0: shares
  int64_t stages = 0, cost = 0;
};
Spread choose_spread(SpanPool pool, int head_dim, int rows, int64_t num_seqs, int num_kv_heads, int64_t blocks,
                     bool even, int num_sms) {
  const int stage_bytes = span_stage_bytes(pool, head_dim);
  constexpr int kShares = 800;
  // a stage of every SM at 6.7 TB/s, and what the calls' stages take at that rate
  const int64_t together = 145ll * stage_bytes / 65536;
  const int64_t all = (num_seqs * num_kv_heads * blocks + kSpanWarps - 1) / kSpanWarps;
  const int64_t hbm = together * all / num_sms * (even ? 10 : 7) / 10;
  Spread best;
  const bool fp8 = pool == SpanPool::kFp8;
  const auto stage_cost = [&](int hg) {
    const int full = fp8 ? (hg == 8 ? 106 : hg == 4 ? 109 : hg == 2 ? 130 : 176)
                         : (hg == 8 ? 63 : hg == 4 ? 67 : hg == 2 ? 79 : 103);
    const int stage = full * (32768 + stage_bytes) / 98304;  // half a stage (bf16 heads of 64) takes two thirds
    return pool == SpanPool::kF32 ? stage + 7 * (rows - 1) : stage;
  };
  int room[kSpanCluster + 1];
  span_cluster_rooms(num_sms, room);
  best.cost = INT64_MAX;
  for (const int hg : {share_heads(pool, num_kv_heads), heads_together(num_kv_heads, kSpanWarps)}) {
    const int64_t segment = 150 + hg * (30 + 5 * (rows - 1));
    const int64_t copies = hg == share_heads(pool, num_kv_heads) ? hbm : hbm * 26 / 25;
    const int64_t cost = kShares + std::max({copies, together, (all + num_sms - 1) / num_sms * stage_cost(hg),
                                             num_seqs * (num_kv_heads / hg) * segment / num_sms});
    if (cost < best.cost) {
      best.hg = hg;
      best.cost = cost;
    }
  }
  for (int hg = heads_together(num_kv_heads, kSpanWarps); hg >= 1; hg /= 2) {
    const int64_t segs = num_seqs * (num_kv_heads / hg);
    const int64_t nst = (blocks + kSpanWarps / hg - 1) / (kSpanWarps / hg);
    const int start = fp8 ? (hg >= 4 ? 450 : hg == 2 ? 380 : 360) : (hg >= 4 ? 410 : hg == 2 ? 315 : 300);
    const int stage = stage_cost(hg);
    for (int splits = 1; splits <= kSpanCluster && splits <= nst; ++splits) {
      // (a CTA alone waits for no other: there may be more of them than SMs)
      const int64_t turns = splits == 1 ? (segs + num_sms - 1) / num_sms : 1;
      if (splits > 1 && segs * splits > num_sms) break;
      if (turns > 8) break;
      if (splits > 1 && segs * splits > room[splits]) continue;
      const int64_t stages = (nst + splits - 1) / splits;
      const int64_t busy = turns * (start + stages * stage);
      // (a seventh more in turns, which lengths that differ upset most: 300 sequences of 4
      // stages and fewer, 23.1 us, in shares 17.7)
      const int64_t cost = std::max<int64_t>(turns > 1 ? busy * 8 / 7 : busy, start + hbm) +
                           (splits == 1 ? 0 : hg == 8 ? 150 : 75);
      if (cost < best.cost && ring_stages(pool, head_dim, rows, hg, splits) >= 2) {
        best.hg = hg;
        best.splits = splits;
        best.stages = stages;
        best.cost = cost;
      }
    }
  }
  return best;
}

}  // namespace

// Scratch of the shares: two partials for each CTA.
size_t span_workspace_size(int rows, int num_kv_heads, int head_dim, int num_sms) {
  // (enough for every pool)
  const size_t R = static_cast<size_t>(share_heads(SpanPool::kFp8, num_kv_heads)) * rows;
  return align256(2 * num_sms * R * 4) + align256(2 * num_sms * R * head_dim * 4);
}

cudaError_t launch_span_decode(const SpanArgs& a, cudaStream_t stream) {
  SpanParams p;
  std::memset(&p, 0, sizeof(p));
  const int group = a.num_q_heads / a.num_kv_heads;
  const int rows = a.q_len * group;
  const int tu = span_tile_tokens(a.pool, a.head_dim);
  p.window = a.window > 0 && a.window < kNoWindow ? a.window : kNoWindow;
  p.sinks = a.window > 0 ? std::min(a.sinks, a.max_len) : 0;
  // the longest list of blocks that a sequence can have
  int64_t blocks = (a.max_len + tu - 1) / tu;
  const int64_t unbound = blocks;
  if (p.window < kNoWindow)
    blocks = std::min<int64_t>(blocks, (p.sinks + tu - 1) / tu + (static_cast<int64_t>(p.window) + a.q_len - 1 + tu - 1) / tu + 1);
  blocks = std::max<int64_t>(blocks, 1);
  const Spread sp = choose_spread(a.pool, a.head_dim, rows, a.num_seqs, a.num_kv_heads, blocks,
                                  2 * blocks < unbound, a.num_sms);
  const int hg = sp.hg;
  const bool clusters = sp.splits > 0;
  const int ring_most = ring_stages(a.pool, a.head_dim, rows, hg, sp.splits);

  int grid = 0, ring = ring_most;
  dim3 blocks_of;
  if (clusters) {
    const int splits = sp.splits;
    p.splits = splits;
    p.over_splits = static_cast<uint32_t>(((uint64_t{1} << 32) + splits - 1) / splits);
    blocks_of = dim3(static_cast<unsigned>(splits), static_cast<unsigned>(a.num_kv_heads / hg),
                     static_cast<unsigned>(a.num_seqs));
    ring = static_cast<int>(std::min<int64_t>(ring_most, sp.stages));
  } else {
    grid = a.num_sms;
    blocks_of = dim3(static_cast<unsigned>(grid));
  }
  int hg_log2 = 0;
  while ((1 << hg_log2) < hg) ++hg_log2;

  const int64_t head_pages = static_cast<int64_t>(a.num_blocks) * a.num_kv_heads;
  if (head_pages > INT_MAX) return cudaErrorInvalidValue;
  const int box_tokens = std::min(a.block_size, tu);
  cudaError_t e = make_map(&p.map_k, a.k_cache, a.pool, a.head_dim, a.block_size, head_pages, box_tokens, hg);
  if (e == cudaSuccess)
    e = make_map(&p.map_v, a.v_cache, a.pool, a.head_dim, a.block_size, head_pages, box_tokens, hg);
  if (e != cudaSuccess) return e;
  p.out = a.out;
  p.q = static_cast<const char*>(a.q);
  p.tables = a.tables;
  p.lens = a.lens;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.num_seqs = a.num_seqs;
  p.q_len = a.q_len;
  p.group = group;
  p.group_log2 = group >= 8 ? 3 : group >= 4 ? 2 : group >= 2 ? 1 : 0;
  p.rows = rows;
  p.num_q_heads = a.num_q_heads;
  p.pool_heads = a.num_kv_heads;
  p.hg_log2 = hg_log2;
  p.ngroups = a.num_kv_heads / hg;
  p.block_size = a.block_size;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.max_len = a.max_len;
  p.ring = ring;
  p.device_errors = a.device_errors;
  p.wait_limit = a.wait_limit < 0 ? kMaxPolls : static_cast<uint32_t>(a.wait_limit);
  char* ws = static_cast<char*>(a.workspace);
  const size_t R = static_cast<size_t>(hg) * rows;
  const int64_t segments = static_cast<int64_t>(a.num_seqs) * p.ngroups;
  p.part_lse = reinterpret_cast<float*>(ws);
  p.part_out = p.part_lse + align256(2 * a.num_sms * R * 4) / 4;

  int smem = span_smem(a.pool, a.head_dim, rows, ring).total;
  if (p.splits > 1) {
    p.joint_slots = (static_cast<int>(R) + p.splits - 1) / p.splits * p.splits;
    smem += p.joint_slots * (a.head_dim + 2) * 4;
  }
  smem += 1024;
  if (ring < 1 || smem > kSpanSmem) return cudaErrorInvalidValue;
  e = a.pool == SpanPool::kBf16  ? run_span_bf16(a.head_dim, p, blocks_of, smem, stream)
      : a.pool == SpanPool::kF32 ? run_span_f32(a.head_dim, p, blocks_of, smem, stream)
                                 : run_span_fp8(p, blocks_of, smem, stream);
  if (e != cudaSuccess || clusters) return e;
  switch (a.pool) {
    case SpanPool::kFp8: return launch_join<32, true, 4>(p, segments, grid, stream);
    case SpanPool::kBf16:
      return a.head_dim == 128 ? launch_join<16, true, 4>(p, segments, grid, stream)
                               : launch_join<16, true, 2>(p, segments, grid, stream);
    default:
      return a.head_dim == 128 ? launch_join<8, false, 4>(p, segments, grid, stream)
                               : launch_join<16, false, 2>(p, segments, grid, stream);
  }
}

}  // namespace pa
