// Decode attention over the visible part of a paged cache -- a sliding window and a
// few first tokens, or all of it -- for pools in float32, bf16, and e4m3 with a scale
// for each page and head.  One kernel, templated on the pool.
//
// Mathematics.  New token j of a sequence of L tokens (q_len of them new) sits at
// p = L - q_len + j and sees the tokens t <= p with p - t < window or t < sinks:
//   out = sum_t e^{s_t} V_t / sum_t e^{s_t},   s_t = scale <q, K_t>,
// one pass with a running maximum (base 2), float32 throughout.
//
// What bounds it: the bytes of K and V.  A token of one kv head is 2 D elements for
// 4 D flops per query row, a flop or a few per byte.
//
// Layout of the work:
//   * The tokens that any row sees are cut into blocks of TU tokens (the tile of one
//     warp); the blocks with sinks and the blocks of the window form one list, so a
//     long context costs what its window costs.  Pages between the two are not
//     touched, their table entries are not read.
//   * A CTA takes hg kv heads (up to 8) of a sequence together.  All heads' rows of a
//     page stand next to each other in the pool, so one tensor-map box brings a page's
//     rows of all hg heads (up to 64 KiB where a box of one head's rows has 4): few
//     copies per byte, which is what a single issuing warp is short of.  Its 8 warps
//     are the hg heads times 8 / hg blocks of a stage.
//   * Two ways to spread (sequence, head group) segments over the GPU.  Shares: one
//     CTA per SM, every CTA takes an equal run of all segments' stages, found by each
//     CTA itself from the lengths (no plan kernel, no counters to reset); a segment
//     that a share's end cuts leaves partials, which a second kernel joins.
//     Clusters, for small calls: a segment's stages go to the CTAs of one cluster,
//     which join their states through distributed shared memory: one launch, no
//     scratch, half the latency.
//   * A producer warp keeps a ring of stages full across segments.  Its lanes are the
//     stage's copies (K and V, block by block); table entries are read three stages
//     ahead, scales one, so no copy waits for a lookup.
//   * Every wait is bounded; on expiry the kernel reports PA_DEVERR_TIMEOUT, waits for
//     its own copies and returns.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <type_traits>

#include "paged_decode.cuh"
#include "span_decode.h"

namespace pa {
namespace span {

// The blocks that a sequence of `len` tokens has to read.
struct Span {
  int len, lo;        // lo: first token that the window of the first new token reaches
  int nblk;           // blocks in the list
  int ns, shift;      // list index v is block v + (v >= ns ? shift : 0)
  int nst;            // stages (at least one, so that empty sequences get their zero rows)
};

template <int TU>
__device__ __forceinline__ Span make_span(const SpanParams& p, int raw_len) {
  Span s;
  s.len = min(max(raw_len, 0), p.max_len);
  s.lo = max(0, s.len - p.q_len + 1 - p.window);
  const int nb = (s.len + TU - 1) / TU;
  const int wb = s.lo / TU;
  s.ns = (min(p.sinks, s.len) + TU - 1) / TU;
  s.shift = wb - s.ns;
  if (s.shift <= 0) s.ns = s.shift = 0;
  s.nblk = nb - s.shift;
  const int wph_log2 = 3 - p.hg_log2;
  s.nst = max(1, (s.nblk + (1 << wph_log2) - 1) >> wph_log2);
  return s;
}

// (Nothing here goes through the read-only path: a kernel ahead in the stream may still
// be writing lengths, tables or q when this one is already resident.)

// Segments (sequence, head group) in order; the lengths of 32 sequences at a time in
// the warp's lanes.
template <int TU>
struct Walk {
  const SpanParams& p;
  int b, grp, base, lens;
  Span sp;
  __device__ __forceinline__ Walk(const SpanParams& p_, int b_, int grp_) : p(p_), b(b_), grp(grp_), base(b_) {
    load();
  }
  __device__ __forceinline__ void load() {
    const int lane = threadIdx.x & 31;
    lens = base + lane < p.num_seqs ? p.lens[base + lane] : 0;
    sp = make_span<TU>(p, __shfl_sync(kFull, lens, 0));
  }
  __device__ __forceinline__ void next() {
    if (++grp < p.ngroups) return;
    grp = 0;
    ++b;
    if (b - base == 32) {
      base = b;
      load();
    } else {
      sp = make_span<TU>(p, __shfl_sync(kFull, lens, b - base));
    }
  }
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void consumer_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSpanWarps * 32) : "memory");
}
// The same, with the answer whether any warp said yes.
__device__ __forceinline__ bool consumer_barrier_any(bool yes) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, 1, %2, q;\n\t"
      "selp.s32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(static_cast<int>(yes)), "n"(kSpanWarps * 32)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Shared address of CTA `rank` of the cluster for a local shared address.
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 peer_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Which tokens of a tile (first token t0) a query row sees.
struct Sight {
  int last, first, sinks;       // of this lane's row, relative to t0: [first, last] or < sinks
  bool all;                     // every row sees every token: no test
  uint32_t bad;                 // bit i: 16 tokens from 16 i on have no page
  __device__ __forceinline__ bool sees(int t) const {
    return t <= last && (t >= first || t < sinks) && !((bad >> (t >> 4)) & 1u);
  }
};

// ------------------------------------------------------------------ one warp's state
// begin: reset, load q's rows of the head;  unit: fold a tile in (release() once its
// bytes are read);  store: hand the state over as (m, l) and the unnormalised sums.

__device__ __forceinline__ int64_t query_row(const SpanParams& p, int b, int head, int r) {
  const int j = r >> p.group_log2;
  return (static_cast<int64_t>(b) * p.q_len + j) * p.num_q_heads + head * p.group + (r & (p.group - 1));
}

// bf16, mma.sync m16n8k16: scores Q K^T with the rows as A (rows past the group are
// zero), O^T = V^T P^T with the rows as columns; the score fragment of a lane is the B
// fragment of the second product, so P stays in registers.  P is rounded to bf16 for
// it, half a step of 2^-8 for each weight; the row's sum l keeps the unrounded ones.
template <int D>
struct Bf16Rows {
  static constexpr int KS = D / 16, MT = D / 16, TU = 16;
  uint32_t qa[KS][2];
  float o[MT][4];
  float m, l;
  int lane, rows;

  __device__ __forceinline__ void init(const SpanParams& p, int lane_, float*) {
    lane = lane_;
    rows = p.rows;
  }
  __device__ __forceinline__ int row() const { return lane >> 2; }

  __device__ __forceinline__ void begin(const SpanParams& p, int b, int head) {
    const int g = lane >> 2, c = lane & 3;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + query_row(p, b, head, g < rows ? g : 0) * (2 * D));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qa[ks][0] = g < rows ? src[8 * ks + c] : 0u;
      qa[ks][1] = g < rows ? src[8 * ks + 4 + c] : 0u;
    }
    m = kNoScore;
    l = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
  }

  // kb, vb: the head's rows of the tile, 128-byte slabs `slab` bytes apart
  template <typename Release>
  __device__ __forceinline__ void unit(uint32_t kb, uint32_t vb, int slab, int, const Sight& see,
                                       float scale_log2, const float2*, int, Release release) {
    const int mi = lane >> 3, r8 = lane & 7, c = lane & 3;
    const int frow = (mi >> 1) * 8 + r8;
    uint32_t kf[KS][4];
    auto at = [&](int chunk) {
      return static_cast<uint32_t>((chunk >> 3) * slab + frow * 128 + (((chunk & 7) ^ r8) << 4));
    };
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      ldsm_x4(kb + at(2 * ks + (mi & 1)), kf[ks][0], kf[ks][1], kf[ks][2], kf[ks][3]);
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      mma_bf16(s0, qa[ks][0], qa[ks][1], kf[ks][0], kf[ks][1]);
      mma_bf16(s1, qa[ks][0], qa[ks][1], kf[ks][2], kf[ks][3]);
    }
    float sv[4] = {s0[0] * scale_log2, s0[1] * scale_log2, s1[0] * scale_log2, s1[1] * scale_log2};
    if (!see.all) {
      const int tk[4] = {2 * c, 2 * c + 1, 8 + 2 * c, 9 + 2 * c};
#pragma unroll
      for (int e = 0; e < 4; ++e) sv[e] = see.sees(tk[e]) ? sv[e] : -INFINITY;
    }
    float mx = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3]));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    const float mn = fmaxf(m, mx);
    const float alpha = fast_exp2(m - mn);
    m = mn;
    float pr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) pr[e] = fast_exp2(sv[e] - mn);
    l = l * alpha + ((pr[0] + pr[1]) + (pr[2] + pr[3]));
    const uint32_t pb0 = pack_bf16x2(pr[0], pr[1]), pb1 = pack_bf16x2(pr[2], pr[3]);
    if (__any_sync(kFull, alpha != 1.f)) {
      const float a_even = __shfl_sync(kFull, alpha, 8 * c), a_odd = __shfl_sync(kFull, alpha, 8 * c + 4);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] *= a_even;
        o[mt][1] *= a_odd;
        o[mt][2] *= a_even;
        o[mt][3] *= a_odd;
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t vf[4];
      ldsm_x4_trans(vb + at(2 * mt + (mi & 1)), vf[0], vf[1], vf[2], vf[3]);
      mma_bf16_full(o[mt], vf[0], vf[1], vf[2], vf[3], pb0, pb1);
    }
    release();
  }

  __device__ __forceinline__ void store(float* macc, float* ml) {
    float lt = l + __shfl_xor_sync(kFull, l, 1);
    lt += __shfl_xor_sync(kFull, lt, 2);
    const int g = lane >> 2, c = lane & 3;
    if (g < rows && c == 0) {
      ml[g * 2] = m;
      ml[g * 2 + 1] = lt;
    }
    const int h0 = 2 * c, h1 = 2 * c + 1;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int d = 16 * mt + g;
      if (h0 < rows) {
        macc[h0 * D + d] = o[mt][0];
        macc[h0 * D + d + 8] = o[mt][2];
      }
      if (h1 < rows) {
        macc[h1 * D + d] = o[mt][1];
        macc[h1 * D + d + 8] = o[mt][3];
      }
    }
  }
};

// e4m3 codes with a scale for each page and head, mma.sync m16n8k32 on the codes as
// they are (Fp8TensorConsumer has the operand layouts).  q's row, scaled by a power of
// two into [128, 256), goes in as two e4m3 parts: a bf16 element has 8 significant bits
// and a part holds 4, so hi + lo is exact down to 2^-10 of the row's largest element.
//
// V's scale differs from page to page, so it goes into the weights, w_t = e^{s_t} vs_t,
// which are what is split into two parts (within 2^-8 of each weight).  They keep a
// running maximum of their own, mo = max(s_t + log2 vs_t): a page of tiny V rows with
// high probability (a first token's, say) would otherwise push the other pages' weights
// below the codes' range, or vanish from the sum.  l sums e^{s_t} under m = max s_t.
template <int G>
struct Fp8Rows {
  static constexpr int D = 128, KS = 4, MT = 8, NT = 4, TU = 32;
  static constexpr float kPScale = 256.f;
  static constexpr bool kPack = G <= 4;      // columns 4..7 of the PV product free for the lo parts
  uint32_t qh[KS][2], ql[KS][2];
  float o[MT][4];
  float m, l, mo, qinv;
  int lane, rows;

  __device__ __forceinline__ void init(const SpanParams& p, int lane_, float*) {
    lane = lane_;
    rows = p.rows;
  }
  __device__ __forceinline__ int row() const { return lane >> 2; }

  __device__ __forceinline__ void begin(const SpanParams& p, int b, int head) {
    const int g = lane >> 2, c = lane & 3;
    const bool on = g < rows;
    const uint2* src = reinterpret_cast<const uint2*>(p.q + query_row(p, b, head, on ? g : 0) * (2 * D));
    uint2 w[KS][2];
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // columns 32 ks + 16 k + 4 c .. + 3
        w[ks][k] = on ? src[8 * ks + 4 * k + c] : make_uint2(0u, 0u);
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(w[ks][k].x)), fabsf(bf16_hi(w[ks][k].x))),
                                 fmaxf(fabsf(bf16_lo(w[ks][k].y)), fabsf(bf16_hi(w[ks][k].y)))));
      }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu);
    const int se = min(max(134 - e, -126), 126);            // amax 2^se in [128, 256)
    const float up = __uint_as_float(static_cast<uint32_t>(se + 127) << 23);
    qinv = __uint_as_float(static_cast<uint32_t>(127 - se) << 23);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x[4] = {bf16_lo(w[ks][k].x) * up, bf16_hi(w[ks][k].x) * up, bf16_lo(w[ks][k].y) * up,
                            bf16_hi(w[ks][k].y) * up};
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __nv_fp8x2_storage_t h =
              __nv_cvt_float2_to_fp8x2(make_float2(x[2 * j], x[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
          const float2 back = __half22float2(static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
          const __nv_fp8x2_storage_t r = __nv_cvt_float2_to_fp8x2(
              make_float2(x[2 * j] - back.x, x[2 * j + 1] - back.y), __NV_SATFINITE, __NV_E4M3);
          hi |= static_cast<uint32_t>(h) << (16 * j);
          lo |= static_cast<uint32_t>(r) << (16 * j);
        }
        qh[ks][k] = hi;
        ql[ks][k] = lo;
      }
    m = mo = kNoScore;
    l = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
  }

  // half: bytes between tokens 0-15 and 16-31;  scales: (k, v) of tokens 0-15 and, at
  // scales[step], of tokens 16-31
  template <typename Release>
  __device__ __forceinline__ void unit(uint32_t kb, uint32_t vb, int, int half, const Sight& see,
                                       float scale_log2, const float2* scales, int step, Release release) {
    const int mi = lane >> 3, r8 = lane & 7, c = lane & 3;
    const float2 sc0 = scales[0], sc1 = scales[step];
    const float qs = qinv * scale_log2;
    const float ks0 = qs * sc0.x, ks1 = qs * sc1.x;
    const float lv0 = __log2f(sc0.y), lv1 = __log2f(sc1.y);
    float sh[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) sh[n][0] = sh[n][1] = sh[n][2] = sh[n][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t kr[NT][2];
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const int row = (mi >> 1) * 8 + r8;
        ldsm_x4(kb + hb * half + row * 128 + (((2 * ks + (mi & 1)) ^ r8) << 4), kr[2 * hb][0], kr[2 * hb][1],
                kr[2 * hb + 1][0], kr[2 * hb + 1][1]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)                          // c0, c1: hi; c2, c3: lo (row g + 8)
        mma_e4m3(sh[n], qh[ks][0], ql[ks][0], qh[ks][1], ql[ks][1], kr[n][0], kr[n][1]);
    }
    // tokens 8 n + 2 c, 8 n + 2 c + 1 of row lane / 4
    float sv[2 * NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) sv[2 * n + e] = (sh[n][e] + sh[n][e + 2]) * (n < 2 ? ks0 : ks1);
    if (!see.all) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!see.sees(8 * n + 2 * c + e)) sv[2 * n + e] = -INFINITY;
    }
    float mx0 = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3]));
    float mx1 = fmaxf(fmaxf(sv[4], sv[5]), fmaxf(sv[6], sv[7]));
    mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, 2));
    const float mn = fmaxf(m, fmaxf(mx0, mx1));
    const float mon = fmaxf(mo, fmaxf(mx0 + lv0, mx1 + lv1));
    const float alpha = fast_exp2(m - mn), beta = fast_exp2(mo - mon);
    m = mn;
    mo = mon;
    float psum = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * NT; ++e) psum += fast_exp2(sv[e] - mn);
    l = l * alpha + psum;
    const float d0 = lv0 - mon, d1 = lv1 - mon;
    uint32_t ph[NT], pl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float d = n < 2 ? d0 : d1;
      split_e4m3x2(fast_exp2(sv[2 * n] + d) * kPScale, fast_exp2(sv[2 * n + 1] + d) * kPScale, ph[n], pl[n]);
    }
    uint32_t bh0 = ph[0] | (ph[1] << 16), bh1 = ph[2] | (ph[3] << 16);
    const uint32_t bl0 = pl[0] | (pl[1] << 16), bl1 = pl[2] | (pl[3] << 16);
    if constexpr (kPack) {
      const uint32_t x0 = __shfl_xor_sync(kFull, bl0, 16), x1 = __shfl_xor_sync(kFull, bl1, 16);
      if (lane >= 16) {
        bh0 = x0;
        bh1 = x1;
      }
    }
    if (__any_sync(kFull, beta != 1.f)) {
      const int hc = kPack ? (c & 1) : c;
      const float a_even = __shfl_sync(kFull, beta, 8 * hc), a_odd = __shfl_sync(kFull, beta, 8 * hc + 4);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] *= a_even;
        o[mt][1] *= a_odd;
        o[mt][2] *= a_even;
        o[mt][3] *= a_odd;
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t vr[4];
      ldsm_x4_trans(vb + (mi >> 1) * half + ((mi & 1) * 8 + r8) * 128 + ((mt ^ r8) << 4), vr[0], vr[1], vr[2],
                    vr[3]);
      const uint32_t a0 = __byte_perm(vr[0], vr[1], 0x6420), a1 = __byte_perm(vr[0], vr[1], 0x7531);
      const uint32_t a2 = __byte_perm(vr[2], vr[3], 0x6420), a3 = __byte_perm(vr[2], vr[3], 0x7531);
      mma_e4m3(o[mt], a0, a1, a2, a3, bh0, bh1);
      if constexpr (!kPack) mma_e4m3(o[mt], a0, a1, a2, a3, bl0, bl1);
    }
    release();
  }

  __device__ __forceinline__ void store(float* macc, float* ml) {
    float lt = l + __shfl_xor_sync(kFull, l, 1);
    lt += __shfl_xor_sync(kFull, lt, 2);
    const int g = lane >> 2, c = lane & 3;
    if (g < rows && c == 0) {
      ml[g * 2] = m;
      ml[g * 2 + 1] = lt;
    }
    // the sums under m instead of mo
    const float back = fast_exp2(mo - m) * (1.f / kPScale);
    const int h0 = 2 * c, h1 = 2 * c + 1;
    const float b0 = __shfl_sync(kFull, back, (8 * c) & 31), b1 = __shfl_sync(kFull, back, (8 * c + 4) & 31);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if constexpr (kPack) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][e] += __shfl_xor_sync(kFull, o[mt][e], 2);
      }
      const int d = 16 * mt + 2 * g;                        // rows g and g + 8: columns 2 g, 2 g + 1
      if (h0 < rows) *reinterpret_cast<float2*>(macc + h0 * D + d) = make_float2(o[mt][0] * b0, o[mt][2] * b0);
      if (h1 < rows) *reinterpret_cast<float2*>(macc + h1 * D + d) = make_float2(o[mt][1] * b1, o[mt][3] * b1);
    }
  }
};

// float32 on the CUDA cores: 8 lanes a token for the scores, each lane D / 32 columns of
// every row for the values (CoreConsumer's arithmetic, with the window's test).
template <int D, int G>
struct F32Rows : CoreConsumer<DecodeTraits<false, D, G>> {
  using Tr = DecodeTraits<false, D, G>;
  using Base = CoreConsumer<Tr>;
  static constexpr int TU = Tr::UT;
  __device__ __forceinline__ void init(const SpanParams&, int lane_, float* ps_) { Base::init(lane_, ps_); }
  __device__ __forceinline__ int row() const { return this->g_lane; }

  __device__ __forceinline__ void begin(const SpanParams& p, int b, int head) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + query_row(p, b, head, g) * (4 * D));
#pragma unroll
      for (int c = 0; c < Tr::NCH; ++c) {
        const uint4 w = src[this->r + 8 * c];
        unpack_chunk<Tr>(w, &this->qf[g][c * 4]);
#pragma unroll
        for (int e = 0; e < 4; ++e) this->qf[g][c * 4 + e] *= p.scale_log2;
      }
      this->m[g] = kNoScore;
#pragma unroll
      for (int c = 0; c < Tr::CPL; ++c) this->acc[g][c] = 0.f;
    }
    this->lsum = 0.f;
  }

  template <typename Release>
  __device__ __forceinline__ void unit(uint32_t kb, uint32_t vb, int, int, const Sight& see, float,
                                       const float2*, int, Release release) {
    const char* kt = static_cast<const char*>(__cvta_shared_to_generic(kb));
    const char* vt = static_cast<const char*>(__cvta_shared_to_generic(vb));
    const int base = this->base, j4 = this->j4, g_lane = this->g_lane, lane = this->lane;
    float* ps = this->ps;
    float part[Tr::N];
#pragma unroll
    for (int pi = 0; pi < Tr::P; ++pi) {
      const int t = 4 * pi + j4;
      float kf[Tr::EPL];
#pragma unroll
      for (int c = 0; c < Tr::NCH; ++c)
        unpack_chunk<Tr>(*reinterpret_cast<const uint4*>(kt + t * Tr::ROW_BYTES + (this->r + 8 * c) * 16),
                         &kf[c * Tr::CE]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < Tr::EPL; ++e) dot = fmaf(this->qf[g][e], kf[e], dot);
        part[g * Tr::P + pi] = dot;
      }
    }
    butterfly_level<Tr::N>(part, lane, 4);
    butterfly_level<(Tr::N >= 4 ? Tr::N / 2 : 1)>(part, lane, 2);
    butterfly_level<(Tr::N >= 8 ? Tr::N / 4 : 1)>(part, lane, 1);
    float umax = -INFINITY;
#pragma unroll
    for (int e = 0; e < Tr::RC; ++e) {
      const int t = 4 * ((base % Tr::P) + e) + j4;
      if (!see.all && !see.sees(t)) part[e] = -INFINITY;
      umax = fmaxf(umax, part[e]);
    }
#pragma unroll
    for (int mask = 1; mask < 8 / G; mask <<= 1) umax = fmaxf(umax, __shfl_xor_sync(kFull, umax, mask));
    umax = fmaxf(umax, __shfl_xor_sync(kFull, umax, 8));
    umax = fmaxf(umax, __shfl_xor_sync(kFull, umax, 16));
    float alpha[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float mu = __shfl_sync(kFull, umax, g * (8 / G));
      const float mn = fmaxf(this->m[g], mu);
      alpha[g] = fast_exp2(this->m[g] - mn);
      this->m[g] = mn;
    }
    float m_lane = this->m[0], a_lane = alpha[0];
#pragma unroll
    for (int g = 1; g < G; ++g)
      if (g_lane == g) {
        m_lane = this->m[g];
        a_lane = alpha[g];
      }
    float psum = 0.f;
#pragma unroll
    for (int e = 0; e < Tr::RC; ++e) {
      const int t = 4 * ((base % Tr::P) + e) + j4;
      const float pr = fast_exp2(part[e] - m_lane);
      psum += pr;
      ps[t * G + g_lane] = pr;                              // lanes with the same sum store the same value
    }
    this->lsum = this->lsum * a_lane + psum;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int c = 0; c < Tr::CPL; ++c) this->acc[g][c] *= alpha[g];
    __syncwarp();
#pragma unroll
    for (int t = 0; t < TU; ++t) {
      float vv[Tr::CPL];
      load_v_cols<Tr>(vt, t, lane, vv);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float w = ps[t * G + g];
#pragma unroll
        for (int c = 0; c < Tr::CPL; ++c) this->acc[g][c] = fmaf(w, vv[c], this->acc[g][c]);
      }
    }
    release();
  }
};

template <int CPL>
struct Cols {
  float v[CPL];
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (CPL == 4) {
      const float4 t = *reinterpret_cast<const float4*>(p);
      v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
      const float2 t = *reinterpret_cast<const float2*>(p);
      v[0] = t.x; v[1] = t.y;
    }
  }
  __device__ __forceinline__ void load_peer(uint32_t a) {
    if constexpr (CPL == 4) {
      const float4 t = peer_f4(a);
      v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
      const float2 t = peer_f2(a);
      v[0] = t.x; v[1] = t.y;
    }
  }
  __device__ __forceinline__ void store(float* p) const {
    if constexpr (CPL == 4)
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  }
  // to element o of out, rounded once
  template <bool BF16>
  __device__ __forceinline__ void store_out(void* out, int64_t o) const {
    if constexpr (BF16) {
      uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + o);
      if constexpr (CPL == 4)
        *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      else
        *d = pack_bf16x2(v[0], v[1]);
    } else {
      store(static_cast<float*>(out) + o);
    }
  }
};

template <SpanPool P, int D, int G>
struct RowsOf;
template <int D, int G>
struct RowsOf<SpanPool::kBf16, D, G> { using type = Bf16Rows<D>; };
template <int G>
struct RowsOf<SpanPool::kFp8, 128, G> { using type = Fp8Rows<G>; };
template <int D, int G>
struct RowsOf<SpanPool::kF32, D, G> { using type = F32Rows<D, G>; };

constexpr int kAhead = 3;               // stages that the table is read ahead

template <SpanPool P, int D, int G>
__global__ void __launch_bounds__(kSpanThreads, 1) span_decode_kernel(const __grid_constant__ SpanParams p) {
  using Rows = typename RowsOf<P, D, G>::type;
  constexpr int TU = span_tile_tokens(P, D);
  constexpr int ROW = span_row_bytes(P, D);
  constexpr int STAGE = span_stage_bytes(P, D);
  constexpr int SLABS = P == SpanPool::kF32 ? 1 : ROW / 128;
  constexpr int CPL = D / 32;
  constexpr bool BF16_OUT = P != SpanPool::kF32;
  constexpr bool FP8 = P == SpanPool::kFp8;
  static_assert(Rows::TU == TU, "tile");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const SpanSmem at = span_smem(P, D, p.rows, p.ring);
  float* macc = reinterpret_cast<float*>(smem + at.macc);
  float* mml = reinterpret_cast<float*>(smem + at.ml);
  float* sc = reinterpret_cast<float*>(smem + at.sc);
  volatile uint32_t* meta = reinterpret_cast<volatile uint32_t*>(smem + at.meta);
  long long* scan = reinterpret_cast<long long*>(smem + at.scan);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + at.bars);
  uint64_t* empty = full + p.ring;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + at.flag);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hg = 1 << p.hg_log2, wph_log2 = 3 - p.hg_log2, wph = 1 << wph_log2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kSpanWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  wait_prior_grids();
  allow_next_grid();
  __syncthreads();

  // ---- this CTA's stages: from stage st0 of segment (b0, grp0), cnt of them
  int b0, grp0, st0, cnt, rank = 0;
  long long share = 0, begin_at = 0;
  if (p.splits) {
    rank = static_cast<int>(blockIdx.x) % p.splits;
    const int seg = static_cast<int>(blockIdx.x) / p.splits;
    b0 = seg / p.ngroups;
    grp0 = seg - b0 * p.ngroups;
    const int len = p.lens[b0];
    if (threadIdx.x == 0 && rank == 0 && grp0 == 0 &&
        (len < 0 || len > p.max_len || (len > 0 && len < p.q_len)))
      report(p.device_errors, PA_DEVERR_BAD_LENGTH);
    const int nst = make_span<TU>(p, len).nst;
    st0 = static_cast<int>(static_cast<long long>(nst) * rank / p.splits);
    cnt = static_cast<int>(static_cast<long long>(nst) * (rank + 1) / p.splits) - st0;
  } else {
    // every CTA adds up the stages of all sequences: thread t a run of them
    const int per = (p.num_seqs + kSpanThreads - 1) / kSpanThreads;
    const int s0 = min(static_cast<int>(threadIdx.x) * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
    long long sum = 0;
    bool bad = false;
    for (int b = s0; b < s1; ++b) {
      const int len = p.lens[b];
      bad |= len < 0 || len > p.max_len || (len > 0 && len < p.q_len);
      sum += make_span<TU>(p, len).nst;
    }
    if (bad && blockIdx.x == 0) report(p.device_errors, PA_DEVERR_BAD_LENGTH);
    long long x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    long long before = x - sum, total = 0;
#pragma unroll
    for (int w = 0; w <= kSpanWarps; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    total *= p.ngroups;
    before *= p.ngroups;
    share = (total + gridDim.x - 1) / gridDim.x;
    begin_at = min(share * blockIdx.x, total);
    cnt = static_cast<int>(min(begin_at + share, total) - begin_at);
    if (cnt > 0 && before <= begin_at && begin_at < before + sum * p.ngroups) {
      for (int b = s0; b < s1; ++b) {
        const int nst = make_span<TU>(p, p.lens[b]).nst;
        const long long n = static_cast<long long>(nst) * p.ngroups;
        if (begin_at < before + n) {
          const int rem = static_cast<int>(begin_at - before);
          int* start = reinterpret_cast<int*>(scan + kSpanWarps + 1);
          start[0] = b;
          start[1] = rem / nst;
          start[2] = rem % nst;
          break;
        }
        before += n;
      }
    }
    __syncthreads();
    const int* start = reinterpret_cast<const int*>(scan + kSpanWarps + 1);
    b0 = start[0];
    grp0 = start[1];
    st0 = start[2];
    if (cnt <= 0) {
      if (threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
      return;
    }
  }

  if (warp == kSpanWarps) {
    // ------------------------------------------------------------ producer
    // Lane (ps, kv) copies the rows of one block (or page of a block) of K or V.
    const int parts = p.block_size < TU ? TU / p.block_size : 1;
    const int t_op = p.block_size < TU ? p.block_size : TU;
    const int op_bytes = hg * t_op * ROW;
    const int kv = lane & 1, ps = lane >> 1;
    const bool mine = ps < wph * parts;
    const int sub = ps / parts, part = ps % parts;
    // fp8: lane (ps, head, kv) brings a scale
    const int s_ps = (lane >> 1) >> p.hg_log2, s_head = (lane >> 1) & (hg - 1);
    const bool s_mine = FP8 && s_ps < wph * parts;
    const float* s_src = kv ? p.v_scales : p.k_scales;

    Walk<TU> wk(p, b0, grp0);
    int st = st0, fetched = 0;
    int q_phys[kAhead], q_off[kAhead], q_head[kAhead];
    bool q_vis[kAhead];
    auto fetch = [&](int& phys, int& off, int& head, bool& vis) {
      phys = 0;
      off = head = 0;
      vis = false;
      if (fetched >= cnt) return;
      const int v = (st << wph_log2) + sub;
      head = wk.grp << p.hg_log2;
      if (mine && v < wk.sp.nblk) {
        const int t = (v + (v >= wk.sp.ns ? wk.sp.shift : 0)) * TU + part * t_op;
        const int page = t / p.block_size, first = page * p.block_size;
        vis = t < wk.sp.len && !(first >= p.sinks && first + p.block_size <= wk.sp.lo);
        off = t - first;
        if (vis) phys = p.tables[static_cast<int64_t>(wk.b) * p.max_blocks + page];
      }
      ++fetched;
      if (++st == wk.sp.nst) {
        st = 0;
        if (fetched < cnt) wk.next();
      }
    };
    auto scale_of = [&](int phys, bool vis, int head) {
      const int src = s_mine ? 2 * s_ps : 0;
      const int ph = __shfl_sync(kFull, phys, src);
      const bool ok = __shfl_sync(kFull, vis ? 1 : 0, src) != 0 && ph >= 0 && ph < p.num_blocks;
      return s_mine && ok ? s_src[static_cast<int64_t>(ph) * p.pool_heads + head + s_head] : 1.f;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(q_phys[k], q_off[k], q_head[k], q_vis[k]);
    float sc_next = 1.f;
    int s = 0, issued = 0;
    uint32_t parity = 1;
    bool ok_all = true;
    for (int i = 0; i < cnt; ++i) {
      if (!mbar_wait(&empty[s], parity, p.wait_limit) || *abort_flag) {
        ok_all = false;
      }
      ok_all = __all_sync(kFull, ok_all);
      if (!ok_all) break;
      const bool valid = q_phys[0] >= 0 && q_phys[0] < p.num_blocks;
      const bool go = q_vis[0] && valid;
      const uint32_t bad = __ballot_sync(kFull, q_vis[0] && !valid);
      const uint32_t ops = __ballot_sync(kFull, go);
      if (lane == 0) {
        if (bad) report(p.device_errors, PA_DEVERR_BAD_BLOCK);
        meta[s] = bad;
        mbar_expect_tx(&full[s], __popc(ops) * op_bytes);
      }
      __syncwarp();
      if (go) {
        unsigned char* dst = smem + s * STAGE + kv * (STAGE / 2) + ps * op_bytes;
        const CUtensorMap* map = kv ? &p.map_v : &p.map_k;
        const int z = q_phys[0] * p.pool_heads + q_head[0];
        if constexpr (SLABS > 1)
          tma_load_4d(dst, map, 0, q_off[0], z, 0, &full[s]);
        else
          tma_load_3d(dst, map, 0, q_off[0], z, &full[s]);
      }
      if constexpr (FP8) {
        const float cur = i == 0 ? scale_of(q_phys[0], q_vis[0], q_head[0]) : sc_next;
        sc_next = scale_of(q_phys[1], q_vis[1], q_head[1]);
        sc[s * 32 + lane] = cur;
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&full[s]);
      ++issued;
      if (++s == p.ring) {
        s = 0;
        parity ^= 1;
      }
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) {
        q_phys[k] = q_phys[k + 1];
        q_off[k] = q_off[k + 1];
        q_head[k] = q_head[k + 1];
        q_vis[k] = q_vis[k + 1];
      }
      fetch(q_phys[kAhead - 1], q_off[kAhead - 1], q_head[kAhead - 1], q_vis[kAhead - 1]);
    }
    if (!ok_all) {
      if (lane == 0) {
        report(p.device_errors, PA_DEVERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
    // copies still in flight, when a wait ran out: at most the last `ring` stages'
    // (with the normal bound; at once when the consumers took them all)
    for (int i = max(0, issued - p.ring); i < issued; ++i)
      mbar_wait(&full[i % p.ring], (i / p.ring) & 1);
  } else {
    // ----------------------------------------------------------- consumers
    const int hl = warp >> wph_log2, sub = warp & (wph - 1);
    const int parts = p.block_size < TU ? TU / p.block_size : 1;
    const int t_op = p.block_size < TU ? p.block_size : TU;
    const int op_bytes = hg * t_op * ROW;
    const int slab = hg * t_op * 128;                        // bytes between 128-byte slabs of a row
    const int half = parts > 1 ? op_bytes : 16 * ROW;        // bytes between 16-token halves (fp8)
    const uint32_t tile_off = sub * parts * op_bytes + hl * t_op * (ROW / SLABS);
    Rows rows;
    rows.init(p, lane, reinterpret_cast<float*>(smem + at.ps) + warp * TU * p.rows);
    Walk<TU> wk(p, b0, grp0);
    int s = 0, left = cnt, st = st0;
    uint32_t parity = 0;
    bool first_seg = true, aborted = false;
    for (;;) {
      const Span& sp = wk.sp;
      const int st_end = min(sp.nst, st + left);
      const int st_begin = st;
      const int head = (wk.grp << p.hg_log2) + hl;
      rows.begin(p, wk.b, head);
      const int q_pos = sp.len - p.q_len + (rows.row() >> p.group_log2);   // of this lane's row
      for (; st < st_end; ++st) {
        if (!mbar_wait(&full[s], parity, p.wait_limit)) {
          report(p.device_errors, PA_DEVERR_TIMEOUT);
          *abort_flag = 1;
          aborted = true;
        }
        aborted = __any_sync(kFull, aborted);
        if (aborted) break;
        const int v = (st << wph_log2) + sub;
        bool wrote = false;
        if (v < sp.nblk) {
          const int t0 = (v + (v >= sp.ns ? sp.shift : 0)) * TU;
          const uint32_t bad_all = meta[s] >> (2 * sub * parts);
          // a bit for each 16 tokens of the tile
          uint32_t bad = bad_all & 1u;
          if (TU == 32) bad |= (parts > 1 ? (bad_all >> 2) & 1u : bad) << 1;
          Sight see;
          see.bad = bad;
          see.all = bad == 0 && t0 + TU <= sp.len - p.q_len + 1 &&
                    (t0 >= sp.len - p.window || t0 + TU <= p.sinks);
          see.last = q_pos - t0;
          see.first = q_pos - p.window + 1 - t0;
          see.sinks = p.sinks - t0;
          const uint32_t kb = smem_addr(smem) + s * STAGE + tile_off, vb = kb + STAGE / 2;
          if (!see.all) {
            // V rows that no row of the sequence sees (stale, never written, of a missing
            // page) must not meet the zero weights as NaN or infinity
            for (int i = lane; i < TU * (ROW / 16); i += 32) {
              const int t = i / (ROW / 16), ch = i % (ROW / 16);
              const int tt = t0 + t;
              if (tt >= sp.len || (tt >= p.sinks && tt < sp.lo) || ((bad >> (t >> 4)) & 1u)) {
                uint32_t a;
                if (P == SpanPool::kF32)
                  a = t * ROW + ch * 16;
                else if (FP8)
                  a = (t >> 4) * half + (t & 15) * 128 + ch * 16;
                else
                  a = (ch >> 3) * slab + t * 128 + (ch & 7) * 16;
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + a), "r"(0u) : "memory");
              }
            }
            wrote = true;
            __syncwarp();
          }
          const float2* scales = reinterpret_cast<const float2*>(sc + s * 32) + ((sub * parts) << p.hg_log2) + hl;
          rows.unit(kb, vb, slab, half, see, p.scale_log2, scales, parts > 1 ? hg : 0, [&] {
            // order the zeroes before the next copy into this stage
            if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
          });
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[s]);
        }
        if (++s == p.ring) {
          s = 0;
          parity ^= 1;
        }
      }
      left -= st_end - st_begin;
      // ---- the segment's part is done: join the head's warps
      float* my_acc = macc + warp * p.rows * D;
      rows.store(my_acc, mml + warp * p.rows * 2);
      // (the warps agree on giving up, so that none waits at a barrier for one that left)
      if (wph > 1 || p.splits) aborted = consumer_barrier_any(aborted); else __syncwarp();
      const int R = hg * p.rows;
      const bool whole = st_begin == 0 && st_end == sp.nst;
      for (int r = sub; r < p.rows; r += wph) {
        const int w0 = hl << wph_log2;
        float M = kNoScore;
        for (int w = 0; w < wph; ++w) M = fmaxf(M, mml[((w0 + w) * p.rows + r) * 2]);
        float lam = 0.f;
        Cols<CPL> acc;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc.v[c] = 0.f;
#pragma unroll 4
        for (int w = 0; w < wph; ++w) {
          const float f = fast_exp2(mml[((w0 + w) * p.rows + r) * 2] - M);
          lam = fmaf(f, mml[((w0 + w) * p.rows + r) * 2 + 1], lam);
          Cols<CPL> x;
          x.load(macc + ((w0 + w) * p.rows + r) * D + lane * CPL);
#pragma unroll
          for (int c = 0; c < CPL; ++c) acc.v[c] = fmaf(f, x.v[c], acc.v[c]);
        }
        if (p.splits > 1) {
          // the cluster's CTAs join later: the ring is free by now (every copy consumed)
          float* cb = reinterpret_cast<float*>(smem);
          acc.store(cb + (hl * p.rows + r) * D + lane * CPL);
          if (lane == 0) {
            cb[R * D + (hl * p.rows + r) * 2] = M;
            cb[R * D + (hl * p.rows + r) * 2 + 1] = lam;
          }
        } else {
          const float inv = lam > 0.f || lam != lam ? 1.f / lam : 0.f;   // no token seen: zeros
#pragma unroll
          for (int c = 0; c < CPL; ++c) acc.v[c] *= inv;
          if (whole) {
            acc.template store_out<BF16_OUT>(p.out, query_row(p, wk.b, head, r) * D + lane * CPL);
          } else {
            const int64_t row = (2 * static_cast<int64_t>(blockIdx.x) + (first_seg ? 0 : 1)) * R + hl * p.rows + r;
            acc.store(p.part_out + row * D + lane * CPL);
            if (lane == 0) p.part_lse[row] = lam > 0.f ? M + __log2f(lam) : (lam != lam ? lam : -INFINITY);
          }
        }
      }
      if (!p.splits && first_seg && warp == 0 && lane == 0) {
        // a segment that began in an earlier share and ends here: that share, and which
        // of its two partials
        int4 cut = make_int4(-1, 0, 0, 0);
        if (st_begin > 0 && st_end == sp.nst) {
          const long long seg_at = begin_at - st_begin;
          const long long c1 = seg_at / share;
          cut = make_int4(wk.b, wk.grp, static_cast<int>(c1), seg_at == c1 * share ? 0 : 1);
        }
        p.cuts[blockIdx.x] = cut;
      }
      if (left <= 0 || aborted) break;
      if (wph > 1) consumer_barrier(); else __syncwarp();      // the states have been read
      first_seg = false;
      st = 0;
      wk.next();
    }
  }

  if (p.splits > 1) {
    // ---- the cluster joins its CTAs' states; rows go round its warps
    cluster_sync();
    if (warp < kSpanWarps) {
      const int R = hg * p.rows;
      const uint32_t cb = smem_addr(smem);
      for (int r = rank * kSpanWarps + warp; r < R; r += p.splits * kSpanWarps) {
        float2 ml[kSpanCluster];
        float M = kNoScore;
#pragma unroll
        for (int c = 0; c < kSpanCluster; ++c)
          if (c < p.splits) {
            ml[c] = peer_f2(peer_addr(cb + (R * D + r * 2) * 4, c));
            M = fmaxf(M, ml[c].x);
          }
        float lam = 0.f;
        Cols<CPL> acc;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc.v[c] = 0.f;
#pragma unroll
        for (int c = 0; c < kSpanCluster; ++c)
          if (c < p.splits) {
            Cols<CPL> x;
            x.load_peer(peer_addr(cb + (r * D + lane * CPL) * 4, c));
            const float f = fast_exp2(ml[c].x - M);
            lam = fmaf(f, ml[c].y, lam);
#pragma unroll
            for (int e = 0; e < CPL; ++e) acc.v[e] = fmaf(f, x.v[e], acc.v[e]);
          }
        const float inv = lam > 0.f || lam != lam ? 1.f / lam : 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc.v[c] *= inv;
        const int h = r / p.rows;
        acc.template store_out<BF16_OUT>(
            p.out, query_row(p, b0, (grp0 << p.hg_log2) + h, r - h * p.rows) * D + lane * CPL);
      }
    }
    cluster_sync();                                          // peers have read this CTA's memory
  }
}

// Launch of one instance: a plain grid of shares, or clusters of p.splits CTAs.
template <SpanPool P, int D, int G>
cudaError_t run_span(const SpanParams& p, int grid, int smem, cudaStream_t stream) {
  // the opt-in to more than 48 KiB of dynamic shared memory is per device
  static std::atomic<uint64_t> configured{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(span_decode_kernel<P, D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpanSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kSpanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits > 1 ? static_cast<unsigned>(p.splits) : 1u;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, span_decode_kernel<P, D, G>, p);
}

}  // namespace span
}  // namespace pa
