// Append with rotary positions: q and k rotated on the way, k and v written into
// their slots of the paged pools -- pools of the inputs' own type, e4m3 pools with
// a fixed scale per kv head, and e4m3 pools with a scale for each page and head.
//
// Rotation of a pair (a, b) of a head's row at the token's position, in float32:
//   a' = a cos - b sin,   b' = b cos + a sin
// with the pair (i, i + R/2) or (2 i, 2 i + 1), i < R/2, and cos / sin from the
// position's table row.  The two products of each are rounded before they are
// added (no contraction), so the result does not depend on which one a compiler
// would have fused.
//
// All of it is bound by memory: a token's rows are read once and written once.
// A lane holds the two 16-byte chunks of a row that rotate into each other, and a
// thread takes the same chunks of several heads of one token, so that the table
// row (4 bytes per rotated column, twice what a bf16 row is) is loaded once for
// all of them and their loads are in flight together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_rope.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

// (No load here goes through the read-only path: the kernels start before the one ahead
// of them in the stream has ended, and wait for its writes on the device.)

// 16 bytes of a row as floats and back.  E: float or uint16_t (bf16 bits).
template <typename E>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
  }
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float* x) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

// The two chunks of a row that lane l of the row's D / (2 N) lanes holds.
// Halves: chunk l and its partner R/2 columns on; the lanes behind the rotated
// chunks take the rest of the row two by two.  Neighbours: any two chunks will do.
template <int N, int D, bool INTER>
struct LaneChunks {
  int c0, c1;          // chunk indexes
  bool rot0, rot1;     // rotated (halves: both or neither)
  __device__ __forceinline__ LaneChunks(int l, int rot) {
    if constexpr (INTER) {
      c0 = l;
      c1 = l + D / N / 2;
      rot0 = c0 * N < rot;
      rot1 = c1 * N < rot;
    } else {
      const int half = rot / 2 / N;
      rot0 = rot1 = l < half;
      c0 = rot0 ? l : 2 * l;          // rot / N + 2 (l - half) = 2 l
      c1 = rot0 ? l + half : 2 * l + 1;
    }
  }
};

// This lane's cos and sin values of a table row [cos R/2 | sin R/2].
template <int N, int D, bool INTER>
struct Angles {
  float c[N], s[N];
  __device__ __forceinline__ void load(const float* row, int half, const LaneChunks<N, D, INTER>& lc) {
    if constexpr (INTER) {
      // chunk c holds pairs c N/2 .. + N/2 - 1
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool on = k ? lc.rot1 : lc.rot0;
        const int i = (k ? lc.c1 : lc.c0) * (N / 2);
#pragma unroll
        for (int e = 0; e < N / 2; e += 2) {
          const float2 cc = on ? *reinterpret_cast<const float2*>(row + i + e) : make_float2(1.f, 1.f);
          const float2 ss = on ? *reinterpret_cast<const float2*>(row + half + i + e) : make_float2(0.f, 0.f);
          c[k * N / 2 + e] = cc.x; c[k * N / 2 + e + 1] = cc.y;
          s[k * N / 2 + e] = ss.x; s[k * N / 2 + e + 1] = ss.y;
        }
      }
    } else if (lc.rot0) {
      const int i = lc.c0 * N;
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 cc = *reinterpret_cast<const float4*>(row + i + e);
        const float4 ss = *reinterpret_cast<const float4*>(row + half + i + e);
        c[e] = cc.x; c[e + 1] = cc.y; c[e + 2] = cc.z; c[e + 3] = cc.w;
        s[e] = ss.x; s[e + 1] = ss.y; s[e + 2] = ss.z; s[e + 3] = ss.w;
      }
    }
  }
};

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float a1 = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = a1;
}

// Rotate this lane's two chunks.
template <int N, int D, bool INTER>
__device__ __forceinline__ void rotate(float* x0, float* x1, const LaneChunks<N, D, INTER>& lc,
                                       const Angles<N, D, INTER>& an) {
  if constexpr (INTER) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      if (lc.rot0) turn(x0[2 * e], x0[2 * e + 1], an.c[e], an.s[e]);
      if (lc.rot1) turn(x1[2 * e], x1[2 * e + 1], an.c[N / 2 + e], an.s[N / 2 + e]);
    }
  } else if (lc.rot0) {
#pragma unroll
    for (int e = 0; e < N; ++e) turn(x0[e], x1[e], an.c[e], an.s[e]);
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// Eight floats over s (IEEE division) as e4m3 codes.  A power of two divides by a
// product with its reciprocal, which rounds to the same float.
__device__ __forceinline__ uint2 e4m3x8(const float* x, float s, bool pow2, float inv) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = pow2 ? x[e] * inv : __fdiv_rn(x[e], s);
  return make_uint2(e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16),
                    e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16));
}

// A normal power of two whose reciprocal is normal too.
__device__ __forceinline__ bool is_pow2(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x807fffffu) == 0 && u >= 0x00800000u && u <= 0x7e800000u;
}
__device__ __forceinline__ float pow2_reciprocal(float s) {
  return __uint_as_float(0x7f000000u - __float_as_uint(s));
}

// What becomes of token t: its position is checked against the table and its slot
// against the pool.  pos < 0: a padding token, nothing is read or written.
struct Place {
  int64_t pos, slot;
  bool rotate, write;
};
__device__ __forceinline__ Place place(const RopeArgs& a, int t, bool speak) {
  Place p;
  p.pos = a.positions ? a.positions[t] : 0;
  p.slot = a.slots[t];
  p.rotate = p.pos >= 0;
  p.write = p.rotate && p.slot >= 0;
  if (a.positions && p.pos >= a.max_position) {
    p.rotate = p.write = false;
    if (speak) report(a.device_errors, PA_DEVERR_BAD_POSITION);
  }
  if (p.write && p.slot >= static_cast<int64_t>(a.num_blocks) * a.block_size) {
    p.write = false;
    if (speak) report(a.device_errors, PA_DEVERR_BAD_SLOT);
  }
  return p;
}

// HPT rows (heads h0 .. h0 + HPT - 1, stride D elements) of one kind of one token.
enum Kind { kQ, kK, kV };

template <typename E, int D, bool INTER, bool FP8, int HPT>
__device__ __forceinline__ void rows_of_token(const RopeArgs& a, int t, Kind kind, int h0, int l) {
  constexpr int N = Vec<E>::N;
  constexpr int CPR = D / N;                               // chunks of a row
  const int heads = kind == kQ ? a.num_q_heads : a.num_kv_heads;
  const E* src = static_cast<const E*>(kind == kQ ? a.q : kind == kK ? a.k : a.v) +
                 static_cast<int64_t>(t) * (kind == kQ ? a.q_stride : kind == kK ? a.k_stride : a.v_stride);
  const LaneChunks<N, D, INTER> lc(l, kind == kV ? 0 : a.rot_dim);
  uint4 w0[HPT], w1[HPT];
  const Place p = place(a, t, kind == kK && h0 == 0 && l == 0);
  if (!(kind == kQ ? p.rotate : p.write)) return;
#pragma unroll
  for (int j = 0; j < HPT; ++j)
    if (HPT == 1 || h0 + j < heads) {
      const uint4* r = reinterpret_cast<const uint4*>(src + static_cast<int64_t>(h0 + j) * D);
      w0[j] = r[lc.c0];
      w1[j] = r[lc.c1];
    }
  Angles<N, D, INTER> an;
  const bool turned = kind != kV && a.rot_dim > 0;
  if (turned) an.load(a.cos_sin + p.pos * a.rot_dim, a.rot_dim / 2, lc);
  const int64_t page = p.slot / a.block_size;
  const int64_t off = p.slot - page * a.block_size;
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    if (HPT > 1 && h0 + j >= heads) break;
    const int h = h0 + j;
    if (kind == kV && !FP8) {                              // bytes as they are
      uint4* dst = reinterpret_cast<uint4*>(a.v_cache) +
                   ((page * a.num_kv_heads + h) * a.block_size + off) * CPR;
      dst[lc.c0] = w0[j];
      dst[lc.c1] = w1[j];
      continue;
    }
    float x0[N], x1[N];
    Vec<E>::unpack(w0[j], x0);
    Vec<E>::unpack(w1[j], x1);
    if (turned) rotate<N, D, INTER>(x0, x1, lc, an);
    if (kind == kQ) {
      uint4* dst = reinterpret_cast<uint4*>(a.q_out) +
                   (static_cast<int64_t>(t) * a.num_q_heads + h) * CPR;
      dst[lc.c0] = Vec<E>::pack(x0);
      dst[lc.c1] = Vec<E>::pack(x1);
    } else if constexpr (FP8) {
      const float s = (kind == kK ? a.k_scale : a.v_scale)[h];
      const bool pow2 = is_pow2(s);
      const float inv = pow2 ? pow2_reciprocal(s) : 0.f;
      uint2* dst = reinterpret_cast<uint2*>(kind == kK ? a.k_cache : a.v_cache) +
                   ((page * a.num_kv_heads + h) * a.block_size + off) * CPR;
      dst[lc.c0] = e4m3x8(x0, s, pow2, inv);
      dst[lc.c1] = e4m3x8(x1, s, pow2, inv);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(a.k_cache) +
                   ((page * a.num_kv_heads + h) * a.block_size + off) * CPR;
      dst[lc.c0] = Vec<E>::pack(x0);
      dst[lc.c1] = Vec<E>::pack(x1);
    }
  }
}

// A group of D / (2 N) lanes takes HPT heads of one token and kind.
template <typename E, int D, bool INTER, bool FP8, int HPT>
__global__ void __launch_bounds__(kThreads) rope_and_cache_kernel(const RopeArgs a, int64_t groups,
                                                                  int uq, int uk) {
  wait_prior_grids();
  allow_next_grid();
  constexpr int LPR = D / Vec<E>::N / 2;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
  if (g >= groups) return;
  const int units = uq + 2 * uk;
  const int t = static_cast<int>(g / units);
  const int u = static_cast<int>(g - static_cast<int64_t>(t) * units);
  const int l = threadIdx.x % LPR;
  if (u < uq)
    rows_of_token<E, D, INTER, FP8, HPT>(a, t, kQ, u * HPT, l);
  else if (u < uq + uk)
    rows_of_token<E, D, INTER, FP8, HPT>(a, t, kK, (u - uq) * HPT, l);
  else
    rows_of_token<E, D, INTER, FP8, HPT>(a, t, kV, (u - uq - uk) * HPT, l);
}

// ------------------------------------------------ a scale for each page and head
//
// The tokens that a call puts into one page stand one after another in the batch: a
// run.  One warp takes a run's rows of one head, of K or of V: it rotates them,
// finds their largest magnitude, and from it the page's scale
//   s = 2^k, the least k >= -100 with amax <= 448 2^k
// (a power of two: e4m3 has the same relative steps at every such scale, codes move
// from one scale to another without a second rounding unless they fall below the
// smallest normal code, and dividing is exact).  A run with the page's first slot
// begins the page anew; otherwise the scale only grows, and what the page holds is
// re-encoded when it does.
constexpr int kLanesPerRow = 8;                            // 128 bf16 columns: 2 chunks a lane
constexpr int kRowsPerPass = 32 / kLanesPerRow;

__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // 448 = 1.75 2^8
  int k = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = max(k, -100);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Codes of a word at a new scale: value * ratio, nearest even.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h = static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (16 * i)) & 0xffffu), __NV_E4M3));
    const float2 f = __half22float2(h);
    out |= e4m3x2(f.x * ratio, f.y * ratio) << (16 * i);
  }
  return out;
}

template <bool INTER, int BS>
__device__ __forceinline__ void append_run(const RopeArgs& a, int t0, int n, uint32_t offsets,
                                           int64_t page, bool fresh, int h, bool is_v) {
  constexpr int N = 8, D = 128;
  constexpr int PASSES = BS / kRowsPerPass;
  const int lane = threadIdx.x & 31;
  const int l = lane % kLanesPerRow, row = lane / kLanesPerRow;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) + static_cast<int64_t>(h) * D;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const LaneChunks<N, D, INTER> lc(l, is_v ? 0 : a.rot_dim);
  const bool turned = !is_v && a.rot_dim > 0;
  const float old = fresh ? 0.f : (is_v ? a.v_scales : a.k_scales)[page * a.num_kv_heads + h];

  uint4 w[PASSES][2];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * kRowsPerPass + row;
    if (r < n) {
      const uint4* p = reinterpret_cast<const uint4*>(src + (t0 + static_cast<int64_t>(r)) * stride);
      w[i][0] = p[lc.c0];
      w[i][1] = p[lc.c1];
    }
  }
  uint32_t top = 0;                                        // largest magnitude's bits, finite ones only
  // rotated values replace the raw ones as float32 only while they are coded: the
  // first pass finds the magnitude, the second rotates again (cheaper than twice
  // the registers)
  auto values = [&](int i, float* x0, float* x1) {
    Vec<uint16_t>::unpack(w[i][0], x0);
    Vec<uint16_t>::unpack(w[i][1], x1);
    if (turned) {
      const int r = min(i * kRowsPerPass + row, n - 1);
      Angles<N, D, INTER> an;
      an.load(a.cos_sin + a.positions[t0 + r] * a.rot_dim, a.rot_dim / 2, lc);
      rotate<N, D, INTER>(x0, x1, lc, an);
    }
  };
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    if (i * kRowsPerPass + row < n) {
      float x0[N], x1[N];
      values(i, x0, x1);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t u0 = __float_as_uint(x0[e]) & 0x7fffffffu, u1 = __float_as_uint(x1[e]) & 0x7fffffffu;
        top = max(top, u0 < 0x7f800000u ? u0 : 0u);
        top = max(top, u1 < 0x7f800000u ? u1 : 0u);
      }
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const float need = page_scale(__uint_as_float(top));
  const float s = fmaxf(old, need);
  unsigned char* base = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache) +
                        (page * a.num_kv_heads + h) * BS * static_cast<int64_t>(D);
  if (!fresh && s > old) {
    // what the page holds, rows of this run aside: 16-byte chunk c of row r
    const float ratio = __fdiv_rn(old, s);
#pragma unroll
    for (int i = 0; i < BS * D / 16 / 32; ++i) {
      const int idx = i * 32 + lane;
      if (!((offsets >> (idx / 8)) & 1u)) {
        uint4* p = reinterpret_cast<uint4*>(base) + idx;
        const uint4 c = *p;
        *p = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
      }
    }
  }
  const bool pow2 = is_pow2(s);
  const float inv = pow2 ? pow2_reciprocal(s) : 0.f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * kRowsPerPass + row;
    if (r < n) {
      float x0[N], x1[N];
      values(i, x0, x1);
      const int off = static_cast<int>(a.slots[t0 + r] - page * BS);
      uint2* dst = reinterpret_cast<uint2*>(base + off * D);
      dst[lc.c0] = e4m3x8(x0, s, pow2, inv);
      dst[lc.c1] = e4m3x8(x1, s, pow2, inv);
    }
  }
  if (lane == 0) (is_v ? a.v_scales : a.k_scales)[page * a.num_kv_heads + h] = s;
}

// Page of token t >= 0, or -1 where the token is not written.
__device__ __forceinline__ int64_t page_of(const RopeArgs& a, int t, bool speak) {
  if (t >= a.num_tokens) return -1;
  const Place p = place(a, t, speak);
  return p.write ? p.slot / a.block_size : -1;
}

// Blocks 0 .. kv_blocks - 1 take TILE tokens each: every run that starts among them,
// one warp for each (run, head, K or V).  The blocks behind rotate q.
template <bool INTER, int BS>
__global__ void __launch_bounds__(kThreads) rope_and_cache_page_scale_kernel(
    const RopeArgs a, int tile, int kv_blocks, int warps_per_tile, int64_t q_groups, int uq) {
  wait_prior_grids();
  allow_next_grid();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) >= kv_blocks) {
    constexpr int HPT = 4;
    const int64_t g = static_cast<int64_t>(blockIdx.x - kv_blocks) * (kThreads / kLanesPerRow) +
                      threadIdx.x / kLanesPerRow;
    if (g >= q_groups) return;
    const int t = static_cast<int>(g / uq);
    rows_of_token<uint16_t, 128, INTER, false, HPT>(a, t, kQ, static_cast<int>(g - static_cast<int64_t>(t) * uq) * HPT,
                                                    threadIdx.x % kLanesPerRow);
    return;
  }
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
  const int first = static_cast<int>(gw / warps_per_tile) * tile;
  const int mine = static_cast<int>(gw % warps_per_tile);
  if (first >= a.num_tokens) return;
  // starts among the tile's tokens: the page differs from the token's before
  const int t = first + lane;
  const bool in = lane < tile && t < a.num_tokens;
  const int64_t page = in ? page_of(a, t, mine == 0) : -1;
  const bool start = in && page >= 0 && (t == 0 || page_of(a, t - 1, false) != page);
  uint32_t starts = __ballot_sync(0xffffffffu, start);
  const int items = 2 * a.num_kv_heads;
  int k = mine;                                            // item of the tile: start-major
  while (starts) {
    const int s = first + __ffs(starts) - 1;
    starts &= starts - 1;
    if (k >= items) {
      k -= items;
      continue;
    }
    // the run: up to BS tokens from s on in one page
    const int64_t pg = __shfl_sync(0xffffffffu, page, s - first);
    const int tt = s + lane;
    const bool in_run = tt < a.num_tokens && page_of(a, tt, false) == pg;
    const uint32_t same = __ballot_sync(0xffffffffu, in_run);
    int n = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
    if (n > BS || (n == BS && page_of(a, s + BS, false) == pg)) {
      n = BS;                                              // more tokens than slots: refused
      if (lane == 0) report(a.device_errors, PA_DEVERR_BAD_SLOT);
    }
    const uint32_t bit = lane < n ? 1u << static_cast<uint32_t>(a.slots[tt] - pg * BS) : 0u;
    const uint32_t offsets = __reduce_or_sync(0xffffffffu, bit);
    for (; k < items; k += warps_per_tile)
      append_run<INTER, BS>(a, s, n, offsets, pg, offsets & 1u, k >> 1, k & 1);
    k -= items;
  }
}

// Scale rows of pages that are copied: dst[d] = src[s], one thread per (pair, head).
__global__ void __launch_bounds__(kThreads) copy_scales_kernel(
    const float* __restrict__ src_k, const float* __restrict__ src_v, float* __restrict__ dst_k,
    float* __restrict__ dst_v, const int64_t* __restrict__ pairs, int num_pairs, int heads,
    int num_src, int num_dst, int32_t* device_errors) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t p = i / heads;
  if (p >= num_pairs) return;
  const int64_t h = i - p * heads, s = pairs[2 * p], d = pairs[2 * p + 1];
  if (s < 0 || s >= num_src || d < 0 || d >= num_dst) {
    if (h == 0) report(device_errors, PA_DEVERR_BAD_BLOCK);
    return;
  }
  dst_k[d * heads + h] = src_k[s * heads + h];
  dst_v[d * heads + h] = src_v[s * heads + h];
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t blocks, cudaStream_t stream, A... args) {
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

template <typename E, int D, bool FP8>
cudaError_t run_rope(const RopeArgs& a, cudaStream_t stream) {
  constexpr int per_block = kThreads / (D / Vec<E>::N / 2);
  auto go = [&](auto kernel, int hpt) {
    const int uq = ceil_div(a.num_q_heads, hpt), uk = ceil_div(a.num_kv_heads, hpt);
    const int64_t groups = static_cast<int64_t>(a.num_tokens) * (uq + 2 * uk);
    return launch(kernel, (groups + per_block - 1) / per_block, stream, a, groups, uq, uk);
  };
  // one head a thread while the rows are too few to fill the GPU, four from there on
  const bool few = static_cast<int64_t>(a.num_tokens) * (a.num_q_heads + 2 * a.num_kv_heads) < 8192;
  if (a.interleaved)
    return few ? go(rope_and_cache_kernel<E, D, true, FP8, 1>, 1) : go(rope_and_cache_kernel<E, D, true, FP8, 4>, 4);
  return few ? go(rope_and_cache_kernel<E, D, false, FP8, 1>, 1) : go(rope_and_cache_kernel<E, D, false, FP8, 4>, 4);
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (a.pool == RopePool::kFp8Head) return run_rope<uint16_t, 128, true>(a, stream);
  if (a.pool == RopePool::kBf16)
    return a.head_dim == 128 ? run_rope<uint16_t, 128, false>(a, stream) : run_rope<uint16_t, 64, false>(a, stream);
  if (a.pool == RopePool::kF32)
    return a.head_dim == 128 ? run_rope<float, 128, false>(a, stream) : run_rope<float, 64, false>(a, stream);
  // a scale for each page and head.  Few tokens (decode steps: a run each): a tile of
  // one token, so that every (run, head, K or V) has its warp at once; many: a tile of
  // a page's tokens, which spares the blocks that would find no run of their own.
  const int tile = a.num_tokens <= 1024 ? 1 : a.block_size;
  const int warps_per_tile = 2 * a.num_kv_heads;
  const int64_t kv_warps = static_cast<int64_t>((a.num_tokens + tile - 1) / tile) * warps_per_tile;
  const int64_t kv_blocks = (kv_warps + kThreads / 32 - 1) / (kThreads / 32);
  const int uq = ceil_div(a.num_q_heads, 4);
  const int64_t q_groups = static_cast<int64_t>(a.num_tokens) * uq;
  const int64_t q_blocks = (q_groups + kThreads / kLanesPerRow - 1) / (kThreads / kLanesPerRow);
  if (kv_blocks > 0x3fffffff) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    return launch(kernel, kv_blocks + q_blocks, stream, a, tile, static_cast<int>(kv_blocks), warps_per_tile,
                  q_groups, uq);
  };
  if (a.interleaved)
    return a.block_size == 16 ? go(rope_and_cache_page_scale_kernel<true, 16>)
                              : go(rope_and_cache_page_scale_kernel<true, 32>);
  return a.block_size == 16 ? go(rope_and_cache_page_scale_kernel<false, 16>)
                            : go(rope_and_cache_page_scale_kernel<false, 32>);
}

cudaError_t launch_copy_scales(const float* src_k, const float* src_v, float* dst_k, float* dst_v,
                               const int64_t* pairs, int num_pairs, int num_kv_heads, int num_src,
                               int num_dst, int32_t* device_errors, cudaStream_t stream) {
  if (num_pairs == 0) return cudaSuccess;
  const int64_t n = static_cast<int64_t>(num_pairs) * num_kv_heads;
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  copy_scales_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
      src_k, src_v, dst_k, dst_v, pairs, num_pairs, num_kv_heads, num_src, num_dst, device_errors);
  return cudaGetLastError();
}

}  // namespace pa
