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
#include "span_decode.h"

namespace pa {
namespace {

constexpr int kJoinWarps = 8;

template <int CPL>
struct Joined {
  float M = -3.0e38f, S = 0.f, acc[CPL] = {};
  __device__ __forceinline__ void add(float lse, const float* v) {
    const float mn = fmaxf(M, lse);
    const float f = fast_exp2(M - mn), w = fast_exp2(lse - mn);
    S = fmaf(S, f, w);
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = fmaf(acc[k], f, w * v[k]);
    M = mn;
  }
};

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

// A segment whose shares are c1 .. c: out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M)
// over its partials.  Block (c, r): WIDE, the row r by 8 warps that take partials in
// turn (few segments: each spans many shares); else 8 rows, a warp each.
template <bool BF16, int CPL, bool WIDE>
__global__ void __launch_bounds__(kJoinWarps * 32) span_join_kernel(const SpanParams p) {
  constexpr int D = CPL * 32;
  __shared__ float sm[kJoinWarps], ss[kJoinWarps];
  __shared__ float sacc[WIDE ? kJoinWarps : 1][D];
  wait_prior_grids();
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const int4 cut = p.cuts[c];
  if (cut.x < 0) return;
  const int R = p.rows << p.hg_log2;
  const int r = WIDE ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y) * kJoinWarps + warp;
  if (r >= R) return;                                        // (never with WIDE)
  const int n = c - cut.z + 1;
  Joined<CPL> st;
#pragma unroll 4
  for (int i = WIDE ? warp : 0; i < n; i += WIDE ? kJoinWarps : 1) {
    const int64_t slot = 2 * static_cast<int64_t>(cut.z + i) + (i == 0 ? cut.w : 0);
    float v[CPL];
    load_part<CPL>(p.part_out + (slot * R + r) * D + lane * CPL, v);
    st.add(p.part_lse[slot * R + r], v);
  }
  if constexpr (WIDE) {
    if (lane == 0) {
      sm[warp] = st.M;
      ss[warp] = st.S;
    }
#pragma unroll
    for (int k = 0; k < CPL; ++k) sacc[warp][lane * CPL + k] = st.acc[k];
    __syncthreads();
    if (warp != 0) return;
    float M = sm[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) M = fmaxf(M, sm[w]);
    st.S = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) st.acc[k] = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = fast_exp2(sm[w] - M);
      st.S = fmaf(f, ss[w], st.S);
#pragma unroll
      for (int k = 0; k < CPL; ++k) st.acc[k] = fmaf(f, sacc[w][lane * CPL + k], st.acc[k]);
    }
  }
  const float inv = st.S > 0.f || st.S != st.S ? 1.f / st.S : 0.f;
  const int head = (cut.y << p.hg_log2) + r / p.rows, row = r % p.rows;
  const int64_t o = ((static_cast<int64_t>(cut.x) * p.q_len + (row >> p.group_log2)) * p.num_q_heads +
                     head * p.group + (row & (p.group - 1))) * D + lane * CPL;
  if constexpr (BF16) {
    uint32_t w[CPL / 2];
#pragma unroll
    for (int k = 0; k < CPL / 2; ++k) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(st.acc[2 * k] * inv, st.acc[2 * k + 1] * inv);
      w[k] = *reinterpret_cast<const uint32_t*>(&t);
    }
    uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + o);
    if constexpr (CPL == 4) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
    else *d = w[0];
  } else {
    float* d = static_cast<float*>(p.out) + o;
#pragma unroll
    for (int k = 0; k < CPL; ++k) d[k] = st.acc[k] * inv;
  }
}

cudaError_t launch_join(const SpanParams& p, bool bf16, int head_dim, bool wide, int ctas, cudaStream_t stream) {
  const int R = p.rows << p.hg_log2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(wide ? R : (R + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, p); };
  if (bf16) {
    if (head_dim == 128) return wide ? go(span_join_kernel<true, 4, true>) : go(span_join_kernel<true, 4, false>);
    return wide ? go(span_join_kernel<true, 2, true>) : go(span_join_kernel<true, 2, false>);
  }
  if (head_dim == 128) return wide ? go(span_join_kernel<false, 4, true>) : go(span_join_kernel<false, 4, false>);
  return wide ? go(span_join_kernel<false, 2, true>) : go(span_join_kernel<false, 2, false>);
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

// Heads that a CTA can take together: the largest power of two up to 8 that divides them.
int most_heads(int num_kv_heads) {
  int hg = 8;
  while (num_kv_heads % hg) hg /= 2;
  return hg;
}

}  // namespace

// Scratch of the shares: what ends where, and two partials for each CTA.
size_t span_workspace_size(int rows, int num_kv_heads, int head_dim, int num_sms) {
  const size_t R = static_cast<size_t>(most_heads(num_kv_heads)) * rows;
  return align256(static_cast<size_t>(num_sms) * sizeof(int4)) + align256(2 * num_sms * R * 4) +
         align256(2 * num_sms * R * head_dim * 4);
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
  if (p.window < kNoWindow)
    blocks = std::min<int64_t>(blocks, (p.sinks + tu - 1) / tu + (static_cast<int64_t>(p.window) + a.q_len - 1 + tu - 1) / tu + 1);
  blocks = std::max<int64_t>(blocks, 1);
  int hg = most_heads(a.num_kv_heads);
  const int64_t pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  const int64_t stages_all = (pairs * blocks + kSpanWarps - 1) / kSpanWarps;
  const SpanSmem fixed = span_smem(a.pool, a.head_dim, rows, 0);
  const int stage = span_stage_bytes(a.pool, a.head_dim);
  const int ring_most = std::min<int>(kSpanRing, (kSpanSmem - 1024 - fixed.total) / (stage + 160));

  int grid = 0, ring = ring_most;
  const bool clusters = stages_all <= 6 * static_cast<int64_t>(a.num_sms);
  if (clusters) {
    while (hg > 1 && pairs / hg * kSpanCluster < a.num_sms) hg /= 2;
    const int64_t segs = pairs / hg;
    const int wph = kSpanWarps / hg;
    const int64_t nst = (blocks + wph - 1) / wph;
    int splits = 1;
    while (splits < kSpanCluster && segs * splits < a.num_sms && 2 * splits <= nst) splits *= 2;
    p.splits = splits;
    grid = static_cast<int>(segs * splits);
    ring = static_cast<int>(std::min<int64_t>(ring_most, (nst + splits - 1) / splits));
  } else {
    grid = a.num_sms;
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
  p.cuts = reinterpret_cast<int4*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + align256(static_cast<size_t>(a.num_sms) * sizeof(int4)));
  p.part_out = p.part_lse + align256(2 * a.num_sms * R * 4) / 4;

  int smem = span_smem(a.pool, a.head_dim, rows, ring).total;
  // the cluster's joined rows stand where the ring was
  if (p.splits > 1) smem = std::max<int>(smem, static_cast<int>(R * (a.head_dim + 2) * 4));
  smem += 1024;
  if (ring < 1 || smem > kSpanSmem) return cudaErrorInvalidValue;
  e = a.pool == SpanPool::kBf16  ? run_span_bf16(a.head_dim, p, grid, smem, stream)
      : a.pool == SpanPool::kF32 ? run_span_f32(a.head_dim, p, grid, smem, stream)
                                 : run_span_fp8(p, grid, smem, stream);
  if (e != cudaSuccess || clusters) return e;
  // few segments: each is cut into many partials
  const bool wide = static_cast<int64_t>(a.num_seqs) * p.ngroups * 16 <= grid;
  return launch_join(p, a.pool != SpanPool::kF32, a.head_dim, wide, grid, stream);
}

}  // namespace pa
