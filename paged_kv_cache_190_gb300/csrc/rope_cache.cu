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
// All of it is bound by memory: a token's rows are read once and written once.  On a GB300
// (6.78 TB/s copied), 32 query and 8 kv heads of 128, bf16: 16384 tokens, 409 MB, in 61.6 us
// (6.64 TB/s); 256 tokens in 2.3 us, one in 1.7 (the kernel's start); into page-scaled e4m3
// pools 8190 tokens, 188 MB, in 31.8 us (5.9 TB/s), 256 single tokens in 3.7 us; into pools
// with a fixed scale per head, 16384 tokens, 378 MB, in 81.7 us (4.6 TB/s): divisions.
// A lane holds the two 16-byte chunks of a row that rotate into each other, and a
// thread takes the same chunks of several heads of one token, so that the table
// row (4 bytes per rotated column, twice what a bf16 row is) is loaded once for
// all of them and their loads are in flight together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_rope.h"

namespace pa {
namespace {

constexpr int kThreads = 128;
// Heads that a thread takes of one token, when there are rows enough to fill the GPU.
// Two: the table row serves two rows, and enough threads are resident to keep HBM busy
// (32 + 8 heads; bf16, 16384 tokens: 61.4 us, one head 73.4, four heads 64.6; float32, 8192:
// 59.3, 60.9, 59.7; e4m3 with a scale per head, 16384: 81.7, 80.2, 164).
constexpr int kHeadsAtOnce = 2;

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

// Four floats as e4m3 codes: nearest even, saturated, NaN kept.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// Division as a call: a scale that is no power of two is rare (one that the append did
// not choose itself), and 16 divisions in line are most of a kernel's code.
__device__ __noinline__ float divide(float x, float s) { return __fdiv_rn(x, s); }

// Eight floats over s (IEEE division) as e4m3 codes.  A power of two divides by a
// product with its reciprocal, which rounds to the same float.
__device__ __forceinline__ uint2 e4m3x8(const float* x, float s, bool pow2, float inv) {
  float y[8];
  if (pow2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * inv;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = divide(x[e], s);
  }
  return make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
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
  const int64_t page = p.slot >> a.block_log2;
  const int off = static_cast<int>(p.slot) & (a.block_size - 1);
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
__global__ void __launch_bounds__(kThreads) rope_and_cache_kernel(const RopeArgs a, unsigned groups,
                                                                  int uq, int uk) {
  wait_prior_grids();
  allow_next_grid();
  constexpr int LPR = D / Vec<E>::N / 2;
  const unsigned g = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;   // under 2^31
  if (g >= groups) return;
  const unsigned units = uq + 2 * uk;
  const int t = g / units, u = g - t * units;
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
// The tokens that a call puts into one page stand one after another in the batch, other
// than tokens that are not written: a run.  A warp takes a head's K and V row of a run of
// one token, a block the rows of up to eight heads of K or of V of a longer one (1 to 8
// warps a head): they rotate the rows, find a head's largest magnitude, and from it the
// page's scale
//   s = 2^k, the least k >= -100 with amax <= 448 2^k
// (a power of two: e4m3 has the same relative steps at every such scale, codes move
// from one scale to another without a second rounding unless they fall below the
// smallest normal code, and dividing is exact).  A run with the page's first slot
// begins the page anew; otherwise the scale only grows, and what the page holds is
// re-encoded when it does.
constexpr int kLanesPerRow = 8;                            // 128 bf16 columns: 2 chunks a lane
constexpr int kRowsPerPass = 32 / kLanesPerRow;
constexpr int kPageThreads = 256;                          // of a block of this kernel
// Heads of q that a thread takes here, where three blocks are resident for the runs' sake
// (8190 tokens: 31.8 us; two heads and four blocks 32.8, one head 44.9).
constexpr int kPageHeadsAtOnce = 4;
constexpr int kKeptRows = 16;                              // tokens that a block holds at a time

__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // 448 = 1.75 2^8
  int k = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = max(k, -100);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// A value's magnitude as ordered bits, 0 for infinities and NaN.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// The largest magnitudes of a chunk's even and odd columns; NaN drops out.
__device__ __forceinline__ __nv_bfloat162 largest(const uint4& w) {
  auto pair = [](uint32_t x) {
    x &= 0x7fff7fffu;
    return *reinterpret_cast<const __nv_bfloat162*>(&x);
  };
  return __hmax2(__hmax2(pair(w.x), pair(w.y)), __hmax2(pair(w.z), pair(w.w)));
}

// Codes of a word at a new scale: value * ratio, nearest even.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  float2 f[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    f[i] = __half22float2(static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (16 * i)) & 0xffffu), __NV_E4M3)));
  return e4m3x4(f[0].x * ratio, f[0].y * ratio, f[1].x * ratio, f[1].y * ratio);
}

// Tokens around a tile, as its block sees them, a thread each: token t0 - kBefore + i is
// entry i.  A run is a page's written tokens with no other page's written token between them,
// the last at most kBehind behind the first; the tile where it starts has it.  Tokens that
// keep to no such run would give a page two owners and are refused: what is more than
// kBehind behind its run's start, and runs of a page that one of the kBefore tokens ahead of
// the tile, or of the tile's, has already begun.  (0.15 us of a decode step.)
constexpr int kTile = 16;
constexpr int kBehind = 48;                               // a page's 32 and 16 more
constexpr int kBefore = kPageThreads - kTile - kBehind;
constexpr int kWords = kPageThreads / 32;
static_assert(kBefore == 192 && kTile + kBehind == 64 && kWords == 8, "the tile and what is behind it: words 6 and 7");
struct Words {                                             // eight words of shared memory, in registers
  uint32_t x[kWords];
  __device__ __forceinline__ explicit Words(const uint32_t* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ uint64_t two(int k) const { return (static_cast<uint64_t>(x[k + 1]) << 32) | x[k]; }
};
struct __align__(16) TileTokens {
  int page_of[kPageThreads];                               // by entry; -1: not written
  uint32_t live[kWords], starts[kWords], again[kWords];
  // the written tokens from t0 on, in order
  int64_t pos[kTile + kBehind];
  int page[kTile + kBehind];
  uint8_t token[kTile + kBehind], off[kTile + kBehind];     // token: behind t0
  // the runs that start in the tile, as their first's place among those: the runs of one
  // token, and those of more with their lengths
  int ones[kTile], more[kTile], length[kTile];
  int num_ones, num_more;
};

// The block looks its tokens up and finds the tile's runs.
__device__ __forceinline__ void find_runs(const RopeArgs& a, TileTokens& seen, int t0, int block_size, bool speak) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, i = threadIdx.x;
  const int64_t t = static_cast<int64_t>(t0) - kBefore + i;
  int page = -1, off = 0;
  int64_t pos = 0;
  if (t >= 0 && t < a.num_tokens) {
    const Place p = place(a, static_cast<int>(t), speak && i >= kBefore && i < kBefore + kTile);
    if (p.write) {
      page = static_cast<int>(p.slot >> a.block_log2);
      off = static_cast<int>(p.slot) & (block_size - 1);
      pos = p.pos;
    }
  }
  seen.page_of[i] = page;
  const uint32_t live = __ballot_sync(0xffffffffu, page >= 0), below = (1u << lane) - 1;
  if (lane == 0) seen.live[warp] = live;
  __syncthreads();
  // a start: the written token before it is another page's
  const Words all(seen.live);
  if (warp >= 4) {                                         // (those of words 0-3 are not needed)
    int w = warp;
    uint32_t earlier = live & below;
#pragma unroll
    for (int k = kWords - 2; k >= 0; --k)
      if (earlier == 0 && k < warp) {
        w = k;
        earlier = all.x[k];
      }
    const bool start = page >= 0 && (earlier == 0 || seen.page_of[32 * w + 31 - __clz(earlier)] != page);
    const uint32_t starts = __ballot_sync(0xffffffffu, start);
    if (lane == 0) seen.starts[warp] = starts;
  }
  // bit j: token t0 + j comes behind this one in the same page
  uint32_t same = 0;
#pragma unroll
  for (int j = 0; j < kTile; j += 4) {
    const int4 q = *reinterpret_cast<const int4*>(seen.page_of + kBefore + j);
    same |= ((q.x == page ? 1u : 0u) | (q.y == page ? 2u : 0u) | (q.z == page ? 4u : 0u) | (q.w == page ? 8u : 0u)) << j;
  }
  if (page < 0 || i >= kBefore + kTile)
    same = 0;
  else if (i >= kBefore)
    same &= ~1u << (i - kBefore);
  same = __reduce_or_sync(0xffffffffu, same);
  if (lane == 0) seen.again[warp] = same;
  if (i >= kBefore && page >= 0) {
    const int c = __popc(live & below) + (warp == 7 ? __popc(all.x[6]) : 0);
    seen.pos[c] = pos;
    seen.token[c] = i - kBefore;
    seen.page[c] = page;
    seen.off[c] = off;
  }
  __syncthreads();
  if (warp == 0) {
    const Words starts(seen.starts), back(seen.again);
    const uint64_t lives = all.two(6), begins = starts.two(6), before = starts.two(4);
    uint32_t agains = 0;
#pragma unroll
    for (int k = 0; k < kWords; ++k) agains |= back.x[k];
    const uint64_t passed = (1ull << lane) - 1;
    int n = 0;
    bool refused = false;
    if (lane < kTile && ((lives >> lane) & 1u)) {
      if ((begins >> lane) & 1u) {
        const uint64_t later = begins >> lane >> 1;        // starts behind this one
        const int most = min(later ? __ffsll(static_cast<long long>(later)) : 64, kBehind + 1);
        n = __popcll((lives >> lane) & ((1ull << most) - 1));
        refused = n > block_size || ((agains >> lane) & 1u);   // more tokens than slots
        n = (agains >> lane) & 1u ? 0 : min(n, block_size);
      } else {
        // its run starts in the tile, or in entry kBefore - 64 + k for bit k of `before`
        refused = (begins & passed) == 0 && before >> (64 - kBehind + lane) == 0;
      }
    }
    if (refused && speak) report(a.device_errors, PA_DEVERR_BAD_SLOT);
    const uint32_t ones = __ballot_sync(0xffffffffu, n == 1), more = __ballot_sync(0xffffffffu, n > 1);
    const int c = __popcll(lives & passed);
    if (n == 1) seen.ones[__popc(ones & below)] = c;
    if (n > 1) {
      seen.more[__popc(more & below)] = c;
      seen.length[__popc(more & below)] = n;
    }
    if (lane == 0) {
      seen.num_ones = __popc(ones);
      seen.num_more = __popc(more);
    }
  }
  __syncthreads();
}

// A copy of 16 bytes to shared memory that nothing waits for until fetched().
__device__ __forceinline__ void fetch16(void* smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A run of several tokens: the block takes its rows of up to kHeadsPerItem heads, of K or
// of V.  The rows and the tokens' table rows come into shared memory all at once, which is
// what has to overlap; the warps go over them there twice, for the magnitude and for the
// codes.  What is left is instructions, 0.54 a cycle of each scheduler over 8190 tokens of
// 32 + 8 heads: hence loops that are not unrolled and no division by a number of heads or
// columns.  Runs of more than kKeptRows tokens come in pieces, the first of them again for
// its codes.
constexpr int kHeadsPerItem = 8;
constexpr int kWarps = kPageThreads / 32;
constexpr int kRunBytes = kKeptRows * (kHeadsPerItem * 256 + 128 * 4);

template <bool INTER, int BS>
__device__ __forceinline__ void append_run(const RopeArgs& a, const TileTokens& seen, unsigned char* buf, float* tops,
                                           int t0, int first, int n, uint32_t offsets, int h0, int heads, bool is_v) {
  constexpr int N = 8, D = 128;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int l = lane % kLanesPerRow, row = lane / kLanesPerRow;
  const int wph_log2 = heads > 4 ? 0 : heads > 2 ? 1 : heads > 1 ? 2 : 3, wph = 1 << wph_log2;   // warps of a head
  static_assert(kWarps == 8 && kHeadsPerItem == 8, "a warp or more for each head");
  const int hh = warp >> wph_log2, sub = warp & (wph - 1);
  const bool active = hh < heads;
  const bool fresh = offsets & 1u;
  const bool turned = !is_v && a.rot_dim > 0;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) + t0 * stride + static_cast<int64_t>(h0) * D;
  float* table = reinterpret_cast<float*>(buf + kKeptRows * kHeadsPerItem * 256);
  const int64_t head_page = static_cast<int64_t>(seen.page[first]) * a.num_kv_heads + h0 + hh;
  float* scale = (is_v ? a.v_scales : a.k_scales) + head_page;
  const LaneChunks<N, D, INTER> lc(l, is_v ? 0 : a.rot_dim);

  auto fetch = [&](int r0, int m) {
    // a token a warp (no divisions: they were most of the instructions here)
    const int cpr = heads * 16, tpr = a.rot_dim / 4;       // 16-byte chunks of a token: rows, table row
    for (int r = warp; r < m; r += kWarps) {
      const uint16_t* from = src + seen.token[first + r0 + r] * stride + lane * N;
      unsigned char* to = buf + (r * cpr + lane) * 16;
      for (int c = lane; c < cpr; c += 32, from += 32 * N, to += 32 * 16) fetch16(to, from);
      if (turned && lane < tpr)
        fetch16(table + r * a.rot_dim + lane * 4, a.cos_sin + seen.pos[first + r0 + r] * a.rot_dim + lane * 4);
    }
    fetched();
    __syncthreads();
  };
  // this lane's two chunks of row r of the piece, rotated
  auto values = [&](int r, float* x0, float* x1) {
    const uint4* p = reinterpret_cast<const uint4*>(buf + (r * heads + hh) * 256);
    Vec<uint16_t>::unpack(p[lc.c0], x0);
    Vec<uint16_t>::unpack(p[lc.c1], x1);
    if (turned) {
      Angles<N, D, INTER> an;
      an.load(table + r * a.rot_dim, a.rot_dim / 2, lc);
      rotate<N, D, INTER>(x0, x1, lc, an);
    }
  };

  const float old = fresh || !active ? 0.f : *scale;
  const int last = (n - 1) / kKeptRows * kKeptRows;
  float top = 0.f;
  __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
  for (int r0 = 0; r0 < n; r0 += kKeptRows) {
    if (r0 > 0) __syncthreads();
    const int m = min(n - r0, kKeptRows);
    fetch(r0, m);
    if (active)
#pragma unroll 1
      for (int r = sub * kRowsPerPass + row; r < m; r += wph * kRowsPerPass) {
        if (!turned) {                                     // bf16 as they are, in pairs
          const uint4* p = reinterpret_cast<const uint4*>(buf + (r * heads + hh) * 256);
          const __nv_bfloat162 t = __hmax2(top2, __hmax2(largest(p[lc.c0]), largest(p[lc.c1])));
          if (!__hisinf(t.x) && !__hisinf(t.y)) {
            top2 = t;
            continue;
          }
        }
        float x0[N], x1[N];
        values(r, x0, x1);
        float t = top;                                     // NaN drops out of fmaxf
#pragma unroll
        for (int e = 0; e < N; ++e) t = fmaxf(t, fmaxf(fabsf(x0[e]), fabsf(x1[e])));
        if (t == INFINITY) {                               // rare: infinities do not count either
          t = top;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            t = fmaxf(t, __uint_as_float(finite_bits(x0[e])));
            t = fmaxf(t, __uint_as_float(finite_bits(x1[e])));
          }
        }
        top = t;
      }
  }
  top = fmaxf(top, fmaxf(__low2float(top2), __high2float(top2)));
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  if (wph > 1) {
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    for (int w = 0; w < wph; ++w) top = fmaxf(top, active ? tops[hh * wph + w] : 0.f);
  }
  const float s = fmaxf(old, page_scale(top));
  unsigned char* base = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache) + head_page * BS * D;
  if (active && !fresh && s > old) {
    // what the page holds, rows of this run aside: 16-byte chunk c of row r
    const float ratio = __fdiv_rn(old, s);
#pragma unroll 2
    for (int idx = sub * 32 + lane; idx < BS * D / 16; idx += wph * 32) {
      if (!((offsets >> (idx / 8)) & 1u)) {
        uint4* p = reinterpret_cast<uint4*>(base) + idx;
        const uint4 c = *p;
        *p = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
      }
    }
  }
  const bool pow2 = is_pow2(s);
  const float inv = pow2 ? pow2_reciprocal(s) : 0.f;
  for (int r0 = last; r0 >= 0; r0 -= kKeptRows) {
    const int m = min(n - r0, kKeptRows);
    if (r0 != last) {
      __syncthreads();
      fetch(r0, m);
    }
    if (active)
#pragma unroll 1
      for (int r = sub * kRowsPerPass + row; r < m; r += wph * kRowsPerPass) {
        float x0[N], x1[N];
        values(r, x0, x1);
        uint2* dst = reinterpret_cast<uint2*>(base + seen.off[first + r0 + r] * D);
        dst[lc.c0] = e4m3x8(x0, s, pow2, inv);
        dst[lc.c1] = e4m3x8(x1, s, pow2, inv);
      }
  }
  if (active && sub == 0 && lane == 0) *scale = s;
  __syncthreads();                                         // the buffer is free
}

// A run of one token, which is what a decode step's are: lanes 0-15 take the head's K
// row, lanes 16-31 its V row, a 16-byte chunk each, and get the chunk that theirs rotates
// with from its lane.
template <bool INTER, int BS>
__device__ __forceinline__ void append_one(const RopeArgs& a, int64_t t, int64_t pos, int off, int64_t page, int h) {
  constexpr int N = 8, D = 128;
  const int lane = threadIdx.x & 31, c = lane & 15;
  const bool is_v = lane >= 16;
  const bool fresh = off == 0;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) + t * (is_v ? a.v_stride : a.k_stride) +
                        static_cast<int64_t>(h) * D;
  const uint4 w = reinterpret_cast<const uint4*>(src)[c];
  float* scale = (is_v ? a.v_scales : a.k_scales) + page * a.num_kv_heads + h;
  const float old = fresh ? 0.f : *scale;
  float x[N];
  Vec<uint16_t>::unpack(w, x);
  if (a.rot_dim > 0) {
    const bool on = !is_v && c * N < a.rot_dim;
    const float* row = a.cos_sin + pos * a.rot_dim;
    const int half = a.rot_dim / 2;
    if constexpr (INTER) {
      if (on) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) turn(x[2 * e], x[2 * e + 1], row[c * 4 + e], row[half + c * 4 + e]);
      }
    } else {
      const int hc = half / N;                             // chunks of a half
      const bool second = c >= hc;
      const int from = on ? (second ? lane - hc : lane + hc) : lane;
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, w.x, from);
      o.y = __shfl_sync(0xffffffffu, w.y, from);
      o.z = __shfl_sync(0xffffffffu, w.z, from);
      o.w = __shfl_sync(0xffffffffu, w.w, from);
      if (on) {
        float y[N];
        Vec<uint16_t>::unpack(o, y);
        const float* cs = row + (second ? c - hc : c) * N;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float xc = __fmul_rn(x[e], cs[e]), ys = __fmul_rn(y[e], cs[half + e]);
          x[e] = second ? __fadd_rn(xc, ys) : __fsub_rn(xc, ys);
        }
      }
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) top = max(top, finite_bits(x[e]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float s = fmaxf(old, page_scale(__uint_as_float(top)));
  unsigned char* base = static_cast<unsigned char*>(is_v ? a.v_cache : a.k_cache) +
                        (page * a.num_kv_heads + h) * BS * static_cast<int64_t>(D);
  if (!fresh && s > old) {
    const float ratio = __fdiv_rn(old, s);
#pragma unroll 4
    for (int idx = c; idx < BS * D / 16; idx += 16)        // 16-byte chunks, 8 a row
      if (idx / 8 != off) {
        uint4* p = reinterpret_cast<uint4*>(base) + idx;
        const uint4 q = *p;
        *p = make_uint4(rescale4(q.x, ratio), rescale4(q.y, ratio), rescale4(q.z, ratio), rescale4(q.w, ratio));
      }
  }
  const bool pow2 = is_pow2(s);
  reinterpret_cast<uint2*>(base + off * D)[c] = e4m3x8(x, s, pow2, pow2 ? pow2_reciprocal(s) : 0.f);
  if (c == 0) *scale = s;
}

// A block of a tile: the runs that start among the tile's kTile tokens, a warp for each
// (token, head) of the runs of one token and the block for each (run, item_heads heads, K
// or V) of the longer ones; the tile's `parts` blocks share these out.  Every block looks
// its tokens up once, into shared memory.  After each of these blocks come `between` that
// rotate q, and the rest of those behind all of them.
template <bool INTER, int BS>
__global__ void __launch_bounds__(kPageThreads, 3) rope_and_cache_page_scale_kernel(
    const RopeArgs a, unsigned parts, unsigned kv_blocks, unsigned between, unsigned q_groups, unsigned uq,
    int item_heads) {
  __shared__ TileTokens seen;
  __shared__ float tops[kWarps];
  // (whole lines: 16 bytes past a sector's border a copy fetches each sector twice, 35.0 us
  // for 8192 tokens instead of 33.6)
  extern __shared__ __align__(128) unsigned char run_buf[];
  wait_prior_grids();
  allow_next_grid();
  unsigned kv = blockIdx.x, qb = blockIdx.x - kv_blocks;
  bool is_q = kv >= kv_blocks;
  if (between > 0 && kv < kv_blocks * (between + 1)) {
    kv = blockIdx.x / (between + 1);
    is_q = kv * (between + 1) != blockIdx.x;
    qb = blockIdx.x - kv - 1;
  }
  if (is_q) {
    const unsigned g = qb * (kPageThreads / kLanesPerRow) + threadIdx.x / kLanesPerRow;
    if (g >= q_groups) return;
    const unsigned t = g / uq;
    rows_of_token<uint16_t, 128, INTER, false, kPageHeadsAtOnce>(a, t, kQ, (g - t * uq) * kPageHeadsAtOnce,
                                                                 threadIdx.x % kLanesPerRow);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int tile = kv / parts, part = kv - tile * parts;
  const int t0 = tile * kTile;
  find_runs(a, seen, t0, BS, part == 0);
  for (int k = part * kWarps + warp; k < seen.num_ones * a.num_kv_heads; k += parts * kWarps) {
    const int j = k / a.num_kv_heads, at = seen.ones[j];
    append_one<INTER, BS>(a, static_cast<int64_t>(t0) + seen.token[at], seen.pos[at], seen.off[at], seen.page[at],
                          k - j * a.num_kv_heads);
  }
  if (seen.num_more == 0) return;                          // (a decode step)
  // a run of few tokens gives its warps a head each, whatever the launch shares out (64
  // sequences of 4 tokens, 8 kv heads: 7.4 us, 10.6 with the launch's)
  auto heads_of = [&](int n) { return n > 8 ? item_heads : kHeadsPerItem; };
  const int few_groups = (a.num_kv_heads + kHeadsPerItem - 1) / kHeadsPerItem;
  const int groups = (a.num_kv_heads + item_heads - 1) / item_heads;
  for (int j = 0, m = part;; m += parts) {
    for (; j < seen.num_more; ++j) {
      const int items = 2 * (seen.length[j] > 8 ? groups : few_groups);
      if (m < items) break;
      m -= items;
    }
    if (j >= seen.num_more) break;
    const int at = seen.more[j], n = seen.length[j], h0 = (m >> 1) * heads_of(n);
    const uint32_t offsets = __reduce_or_sync(0xffffffffu, lane < n ? 1u << seen.off[at + lane] : 0u);
    append_run<INTER, BS>(a, seen, run_buf, tops, t0, at, n, offsets, h0, min(heads_of(n), a.num_kv_heads - h0), m & 1);
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
cudaError_t launch(void (*kernel)(P...), int64_t blocks, int threads, int smem, cudaStream_t stream, A... args) {
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Groups of lanes that a launch may have (their numbers are 32-bit: a 64-bit division each
// costs as much as a head's rotation).
constexpr int64_t kMostGroups = int64_t{1} << 31;

template <typename E, int D, bool FP8>
cudaError_t run_rope(const RopeArgs& a, cudaStream_t stream) {
  constexpr int per_block = kThreads / (D / Vec<E>::N / 2);
  auto go = [&](auto kernel, int hpt) {
    const int uq = ceil_div(a.num_q_heads, hpt), uk = ceil_div(a.num_kv_heads, hpt);
    const int64_t groups = static_cast<int64_t>(a.num_tokens) * (uq + 2 * uk);
    if (groups >= kMostGroups) return cudaErrorInvalidValue;
    return launch(kernel, (groups + per_block - 1) / per_block, kThreads, 0, stream, a, groups, uq, uk);
  };
  // one head a thread while the rows are too few to fill the GPU
  const bool few = static_cast<int64_t>(a.num_tokens) * (a.num_q_heads + 2 * a.num_kv_heads) < 8192;
  constexpr int H = kHeadsAtOnce;
  if (a.interleaved)
    return few ? go(rope_and_cache_kernel<E, D, true, FP8, 1>, 1) : go(rope_and_cache_kernel<E, D, true, FP8, H>, H);
  return few ? go(rope_and_cache_kernel<E, D, false, FP8, 1>, 1) : go(rope_and_cache_kernel<E, D, false, FP8, H>, H);
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (a.pool == RopePool::kFp8Head) return run_rope<uint16_t, 128, true>(a, stream);
  if (a.pool == RopePool::kBf16)
    return a.head_dim == 128 ? run_rope<uint16_t, 128, false>(a, stream) : run_rope<uint16_t, 64, false>(a, stream);
  if (a.pool == RopePool::kF32)
    return a.head_dim == 128 ? run_rope<float, 128, false>(a, stream) : run_rope<float, 64, false>(a, stream);
  // A scale for each page and head.  A tile has a run for each of its tokens (a decode
  // step) or one or two in all (a prompt).  Heads of an item: as many as leave 256 items
  // (512 tokens of 8 kv heads: 6.4 us with 2, 7.6 with 8; 1024: 7.7 with 4, 8.3 with 8).
  // Blocks of a tile: while the tiles are few, as many as give every token and head of a
  // decode step a warp at once, and 16, for as many short runs of a few tokens (333 tokens of
  // 71 sequences, 1 kv head: 5.0 us, 10.0 without; a decode step of 256 tokens, 2 kv heads,
  // 3.4 and 3.0); from there on one for two groups of heads (8190 tokens, 8 kv
  // heads: 31.8 us, 33.2 with a block each for K and V).
  const int64_t tiles = (a.num_tokens + kTile - 1) / kTile;
  int item_heads = 1;
  while (item_heads < kHeadsPerItem &&
         static_cast<int64_t>(a.num_tokens / a.block_size) * a.num_kv_heads >= 256 * item_heads)
    item_heads *= 2;
  const int groups = ceil_div(a.num_kv_heads, item_heads);
  const int most = std::max(ceil_div(kTile * a.num_kv_heads, kWarps), kTile);
  const int parts = static_cast<int>(std::max<int64_t>((groups + 1) / 2, std::min<int64_t>(most, 512 / tiles)));
  const int64_t kv_blocks = tiles * parts;
  const int uq = ceil_div(a.num_q_heads, kPageHeadsAtOnce);
  const int64_t q_groups = static_cast<int64_t>(a.num_tokens) * uq;
  const int64_t q_blocks = (q_groups + kPageThreads / kLanesPerRow - 1) / (kPageThreads / kLanesPerRow);
  // q's blocks between the runs' blocks, where there are rows enough of q: the runs wait and
  // convert while q's rows move (8190 tokens of 32 + 8 heads: 31.8 us; all of q behind 35.0,
  // all between 37.2).  Half of them, which leaves blocks for the end; a page of 32 is two
  // tiles, of which one has the run.
  const int64_t between = a.num_q_heads > 2 * a.num_kv_heads ? q_blocks / kv_blocks * 8 / a.block_size : 0;
  if (kv_blocks >= kMostGroups / 2 || q_groups >= kMostGroups) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    return launch(kernel, kv_blocks + q_blocks, kPageThreads, kRunBytes, stream, a, parts, kv_blocks, between, q_groups, uq, item_heads);
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
