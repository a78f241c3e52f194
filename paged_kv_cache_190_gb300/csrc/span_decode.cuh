// Decode attention over the visible part of a paged cache -- a sliding window and a
// few first tokens, or all of it -- for pools in float32, bf16, e4m3 with a scale
// for each page and head, and 4-bit rows.  One kernel, templated on the pool.
//
// Mathematics.  New token j of a sequence of L tokens (q_len of them new) sits at
// p = L - q_len + j and sees the tokens t <= p with p - t < window or t < sinks:
//   out = sum_t e^{s_t} V_t / sum_t e^{s_t},   s_t = scale <q, K_t>,
// one pass with a running maximum (base 2); scores, maxima and sums in float32, the weights
// of the tensor-core pools rounded for the product with V (two bf16 parts, or a half).
//
// What bounds it: the bytes of K and V.  A token of one kv head is 2 D elements for
// 4 D flops per query row, a flop or a few per byte.  On a GB300 (6.78 TB/s copied): 256
// windows of 1028 tokens, bf16, 8 kv heads, 833 MB in 130.6 us (6.38 TB/s); 16 windows of
// 4100 far into contexts of 131072, 8 rows a head, 269 MB in 44.2 us (6.09); e4m3, 256
// ragged sequences, 885 MB in 143.8 us (6.16), 4 of 131072 tokens, 1.07 GB in 163.0 us
// (6.59); a few short sequences 3.7 to 6.2 us, of which half is the chain length -> table
// entry -> page.
//
// Layout of the work:
//   * The tokens that any row sees are cut into blocks of TU tokens (the tile of one
//     warp); the blocks with sinks and the blocks of the window form one list, so a
//     long context costs what its window costs.  Pages between the two are not
//     touched, their table entries are not read.
//   * A CTA takes hg kv heads (up to 8) of a sequence together.  All heads' rows of a
//     page stand next to each other in the pool, so one tensor-map box brings a page's
//     rows of all hg heads (16 to 32 KiB where one head's rows are 2 to 4): the copy
//     engine wants few, large boxes.  Its 8 warps are the hg heads times 8 / hg blocks of
//     a stage; with 8 heads a warp has a head to itself and nothing to join.
//   * Two ways to spread (sequence, head group) segments over the GPU.  Shares: one
//     CTA per SM, every CTA takes an equal run of all segments' stages, found by each
//     CTA itself from the lengths (no plan kernel, no counters to reset); a segment
//     that a share's end cuts leaves partials, which a second kernel joins (it finds the
//     cuts from the lengths too, while this one still runs).
//     Clusters, where all segments fit the GPU at once: a segment's stages go to the CTAs
//     of one cluster, which join their states through distributed shared memory: one
//     launch, no scratch, half the latency (span_launch.cu chooses).
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

#include "fp4.cuh"
#include "paged_decode.cuh"
#include "span_list.cuh"

namespace pa {
namespace span {

// (Nothing here goes through the read-only path: a kernel ahead in the stream may still
// be writing lengths, tables or q when this one is already resident.)

// Segments (sequence, head group) in order; the lengths of 32 sequences at a time in
// the warp's lanes.
template <int TU>
struct Walk {
  const SpanParams& p;
  int b, grp, base, lens;
  Span sp;
  // len: sequence b_'s (known by then; the lanes' lengths are not waited for)
  __device__ __forceinline__ Walk(const SpanParams& p_, int b_, int grp_, int len) : p(p_), b(b_), grp(grp_), base(b_) {
    load();
    sp = make_span<TU>(p, len);
  }
  __device__ __forceinline__ void load() {
    const int lane = threadIdx.x & 31;
    lens = base + lane < p.num_seqs ? p.lens[base + lane] : 0;
  }
  __device__ __forceinline__ void next() {
    if (++grp < p.ngroups) return;
    grp = 0;
    ++b;
    if (b - base == 32) {
      base = b;
      load();
    }
    sp = make_span<TU>(p, __shfl_sync(kFull, lens, b - base));
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

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// Shared address of CTA `rank` of the cluster for a local shared address.
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ void peer_store(uint32_t a, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
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
// load: q's rows of a head on their way (before the last head's state is stored: it does
// not need q any more);  begin: reset, q ready;  unit: fold a tile in (release() once its
// bytes are read);  store: hand the state over as (m, l) and the unnormalised sums.

__device__ __forceinline__ int64_t query_row(const SpanParams& p, int b, int head, int r) {
  const int j = r >> p.group_log2;
  return (static_cast<int64_t>(b) * p.q_len + j) * p.num_q_heads + head * p.group + (r & (p.group - 1));
}

// bf16, mma.sync m16n8k16: scores Q K^T with the rows as A (rows past the group are
// zero), O^T = V^T P^T with the rows as columns; the score fragment of a lane is the B
// fragment of the second product, so P stays in registers.  P goes into it as two bf16
// parts, the rounded weight and what the rounding left (2^-16 of each weight is lost;
// the rounded part alone loses 2^-8, which makes the error 1.25 times the result's own); the
// row's sum l keeps the unrounded ones.
template <int D>
struct Bf16Rows {
  static constexpr int KS = D / 16, MT = D / 16, TU = 16;
  uint32_t qa[KS][2];
  float o[MT][4];
  float m, l;
  int lane, rows;

  __device__ __forceinline__ void init(const SpanParams& p, int lane_, float*, float*) {
    lane = lane_;
    rows = p.rows;
  }
  __device__ __forceinline__ int row() const { return lane >> 2; }

  __device__ __forceinline__ void load(const SpanParams& p, int b, int head) {
    const int g = lane >> 2, c = lane & 3;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + query_row(p, b, head, g < rows ? g : 0) * (2 * D));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qa[ks][0] = g < rows ? src[8 * ks + c] : 0u;
      qa[ks][1] = g < rows ? src[8 * ks + 4 + c] : 0u;
    }
  }
  __device__ __forceinline__ void begin(const SpanParams&) {
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
    // chunk 2 i + (mi & 1) of this lane's row: an XOR with a constant within a slab
    const uint32_t row0 = ((mi >> 1) * 8 + r8) * 128 + (((mi & 1) ^ r8) << 4);
    auto at = [&](uint32_t base, int i) { return (base + row0 + (i >> 2) * slab) ^ ((i & 3) << 5); };
    uint32_t kf[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      ldsm_x4(at(kb, ks), kf[ks][0], kf[ks][1], kf[ks][2], kf[ks][3]);
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
    const uint32_t rb0 = pack_bf16x2(pr[0] - bf16_lo(pb0), pr[1] - bf16_hi(pb0));
    const uint32_t rb1 = pack_bf16x2(pr[2] - bf16_lo(pb1), pr[3] - bf16_hi(pb1));
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
      ldsm_x4_trans(at(vb, mt), vf[0], vf[1], vf[2], vf[3]);
      mma_bf16_full(o[mt], vf[0], vf[1], vf[2], vf[3], pb0, pb1);
      mma_bf16_full(o[mt], vf[0], vf[1], vf[2], vf[3], rb0, rb1);
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

// (Not volatile: products of registers, free to move between the loads around them.)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two pairs of halves, exactly.
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A row of q, spread over four lanes in pairs of bf16, as halves: scaled by a power of two
// into [128, 256); a bf16 element is exact as a half down to 2^-22 of its row's largest.
// Returns the power's inverse.
template <int KS>
__device__ __forceinline__ float halves_of_q(uint32_t (&qa)[KS][2]) {
  float amax = 0.f;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(qa[ks][k])), fabsf(bf16_hi(qa[ks][k]))));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
  const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu);
  const int se = min(max(134 - e, -126), 126);            // amax 2^se in [128, 256)
  const float up = __uint_as_float(static_cast<uint32_t>(se + 127) << 23);
  const float back = __uint_as_float(static_cast<uint32_t>(127 - se) << 23);
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int k = 0; k < 2; ++k) qa[ks][k] = pack_half2(bf16_lo(qa[ks][k]) * up, bf16_hi(qa[ks][k]) * up);
  return back;
}

// e4m3 codes with a scale for each page and head: codes become halves (exactly, two a
// conversion) on the way into mma.sync m16n8k16.  The e4m3 form of the instruction
// converts both operands inside, at every use, and wants q and the weights as sums of two
// e4m3 parts: 650 instructions a tile were 550 this way (161.8 -> 161.0 us for 885 MB
// then), and the weights keep 11 bits instead of 8.
//   * q: halves_of_q.
//   * The codes of a K row that ldmatrix gives a lane are columns 4 c .. 4 c + 3 of a
//     chunk: they become k = 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of a step, for q alike.
//   * V through ldmatrix.trans on code pairs: columns 2 g and 2 g + 1 of tokens 2 c and
//     2 c + 1 of an 8-token block; the columns become rows g and g + 8 of O^T.
//   * V's scale differs from page to page, so it goes into the weights,
//     w_t = e^{s_t} vs_t, which are rounded to halves (2^-11 of each).  They keep a running
//     maximum of their own, mo = max(s_t + log2 vs_t): a page of tiny V rows with high
//     probability (a first token's, say) would otherwise push the other pages' weights
//     below a half's range.  l sums e^{s_t} under m = max s_t.
struct Fp8Rows {
  static constexpr int D = 128, KS = 8, MT = 8, NT = 4, TU = 32;
  static constexpr float kPLog2 = 10.f;      // weights are carried times 2^10
  uint32_t qa[KS][2];
  float o[MT][4];
  float m, l, mo, qinv;
  int lane, rows;

  __device__ __forceinline__ void init(const SpanParams& p, int lane_, float*, float*) {
    lane = lane_;
    rows = p.rows;
  }
  __device__ __forceinline__ int row() const { return lane >> 2; }

  __device__ __forceinline__ void load(const SpanParams& p, int b, int head) {
    const int g = lane >> 2, c = lane & 3;
    const bool on = g < rows;
    const uint2* src = reinterpret_cast<const uint2*>(p.q + query_row(p, b, head, on ? g : 0) * (2 * D));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint2 w = on ? src[4 * ks + c] : make_uint2(0u, 0u);      // columns 16 ks + 4 c .. + 3
      qa[ks][0] = w.x;
      qa[ks][1] = w.y;
    }
  }
  __device__ __forceinline__ void begin(const SpanParams&) {
    qinv = halves_of_q<KS>(qa);
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
    // chunk (2 ks + (mi & 1)) of row r sits at ((2 ks + (mi & 1)) ^ (r & 7)) << 4: an XOR
    // with a constant from step to step
    const uint32_t ka = kb + ((mi >> 1) * 8 + r8) * 128 + (((mi & 1) ^ r8) << 4);
    float sh[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) sh[n][0] = sh[n][1] = sh[n][2] = sh[n][3] = 0.f;
    uint32_t kw[KS / 2][2][4];                              // (tokens 0-7 | 8-15) x chunks 2 k2, 2 k2 + 1
#pragma unroll
    for (int k2 = 0; k2 < KS / 2; ++k2)
#pragma unroll
      for (int hb = 0; hb < 2; ++hb)
        ldsm_x4((ka + hb * half) ^ (k2 << 5), kw[k2][hb][0], kw[k2][hb][1], kw[k2][hb][2], kw[k2][hb][3]);
#pragma unroll
    for (int k2 = 0; k2 < KS / 2; ++k2)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t b0, b1;
          halves_of(kw[k2][n >> 1][2 * (n & 1) + k], b0, b1);
          mma_f16(sh[n], qa[2 * k2 + k][0], 0u, qa[2 * k2 + k][1], 0u, b0, b1);
        }
    // V's codes come in while the scores are worked on: token blocks 0-7, 8-15, 16-23, 24-31
    const uint32_t va = vb + (mi >> 1) * half + ((mi & 1) * 8 + r8) * 128 + (r8 << 4);
    uint32_t vw[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) ldsm_x4_trans(va ^ (mt << 4), vw[mt][0], vw[mt][1], vw[mt][2], vw[mt][3]);
    release();
    // tokens 8 n + 2 c, 8 n + 2 c + 1 of row lane / 4
    const float qs = qinv * scale_log2;
    const float ks0 = qs * sc0.x, ks1 = qs * sc1.x;
    const float lv0 = __log2f(sc0.y), lv1 = __log2f(sc1.y);
    float sv[2 * NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) sv[2 * n + e] = sh[n][e] * (n < 2 ? ks0 : ks1);
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
    // w = p 2^(lv + m - mo): under 1 by mo's choice.  (The bound on the factor leaves out
    // weights only where a page's scale is 2^116 times the others' and its probability 0.)
    const float f0 = fast_exp2(fminf(lv0 + (mn - mon) + kPLog2, 126.f));
    const float f1 = fast_exp2(fminf(lv1 + (mn - mon) + kPLog2, 126.f));
    uint32_t pb[NT];
    float psum = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float p0 = fast_exp2(sv[2 * n] - mn), p1 = fast_exp2(sv[2 * n + 1] - mn);
      psum += p0 + p1;
      pb[n] = pack_half2(p0 * (n < 2 ? f0 : f1), p1 * (n < 2 ? f0 : f1));
    }
    l = l * alpha + psum;
    if (__any_sync(kFull, beta != 1.f)) {
      const float a_even = __shfl_sync(kFull, beta, 8 * c), a_odd = __shfl_sync(kFull, beta, 8 * c + 4);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] *= a_even;
        o[mt][1] *= a_odd;
        o[mt][2] *= a_even;
        o[mt][3] *= a_odd;
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        uint32_t a[4];                                      // column 2 g's pair, column 2 g + 1's
        halves_of(__byte_perm(vw[mt][i], 0u, 0x3120), a[0], a[1]);
        halves_of(__byte_perm(vw[mt][i + 1], 0u, 0x3120), a[2], a[3]);
        mma_f16(o[mt], a[0], a[1], a[2], a[3], pb[i], pb[i + 1]);
      }
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
    const float back = fast_exp2(mo - m - kPLog2);
    const int h0 = 2 * c, h1 = 2 * c + 1;
    const float b0 = __shfl_sync(kFull, back, 8 * c), b1 = __shfl_sync(kFull, back, 8 * c + 4);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int d = 16 * mt + 2 * g;                        // rows g and g + 8: columns 2 g, 2 g + 1
      if (h0 < rows) *reinterpret_cast<float2*>(macc + h0 * D + d) = make_float2(o[mt][0] * b0, o[mt][2] * b0);
      if (h1 < rows) *reinterpret_cast<float2*>(macc + h1 * D + d) = make_float2(o[mt][1] * b1, o[mt][3] * b1);
    }
  }
};

// Loads of shared memory at a constant offset from an address.
__device__ __forceinline__ uint2 lds64(uint32_t a, int off) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a + off));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a, int off) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a + off));
  return v;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// 4-bit rows (fp4.cuh): a code times its scale is exact as a half, so K and V become halves
// on the way into mma.sync m16n8k16, two a conversion, and one product of two of them
// brings the scale in; q and the weights as for e4m3 (the scales differ within a row, so
// they cannot go into the weights; nor need they, for a half holds the values).  256 ragged
// sequences of 8 kv heads, 448 MB, take 107.9 us (66 at the measured copy rate).  What bounds
// them is not known: 52 % of the issue slots are busy, the ALU pipe 40 %, the tensor pipe 22 %;
// an SM takes a stage in about 1.35 us, of which its bytes are 0.83 and the instructions of two
// tiles a scheduler about 0.77.  A small call takes 5.5.
//   * A row of 72 bytes is loaded as it stands, 8 bytes of 16 columns a time.  V: piece p of
//     rows 4 c + i of 16 tokens falls on banks 8 c + 2 p, a half-warp's on all 32.  K: a
//     half-warp has four pieces of rows 0, 1, 4 and 5, on banks 0 to 7, 18 to 25, 8 to 15 and
//     26 to 1, so one pair of banks twice and one not at all (rows 8, 9, 12 and 13 alike).
//   * Scores: a lane has pieces c and c + 4 of its tokens' rows; q's columns go with them.
//   * S^T = K q^T, with the tokens as rows (half the products of Q K^T, which would leave half
//     of its 16 rows empty); movmatrix turns a tile of weights into P^T's fragment.  Tokens 2 j
//     and 2 j + 1 of a tile of 8 are tokens 4 j and 4 j + 1 of their 16 (of the second tile
//     4 j + 2 and 4 j + 3), so that a lane's weights are those of 4 tokens in a row.
//   * Values: lane (g, c) has piece g of those 4 tokens.  The codes of a column of two
//     tokens are put into one byte (two shifts and two selections for 16 codes), which one
//     conversion makes the pair of halves that the product wants; the columns 16 g + 2 t
//     and 16 g + 2 t + 1 become rows g and g + 8 of O^T's tile t, under the scales of one
//     piece.
struct Fp4Rows {
  static constexpr int D = 128, KS = 8, MT = 8, NT = 4, TU = 32;
  static constexpr float kPLog2 = 10.f;      // weights are carried times 2^10
  uint32_t qa[KS][2];
  float o[MT][4];
  float m[2], l[2], qinv[2];                  // of rows 2 (lane & 3) and the next
  int lane, rows, later;                     // later: new tokens between the two

  __device__ __forceinline__ void init(const SpanParams& p, int lane_, float*, float*) {
    lane = lane_;
    rows = p.rows;
    later = p.group == 1 ? 1 : 0;
  }
  __device__ __forceinline__ int row() const { return 2 * (lane & 3); }

  __device__ __forceinline__ void load(const SpanParams& p, int b, int head) {
    const int g = lane >> 2, c = lane & 3;
    const bool on = g < rows;
    const uint2* src = reinterpret_cast<const uint2*>(p.q + query_row(p, b, head, on ? g : 0) * (2 * D));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // columns 4 (ks & 3) .. + 3 of piece c + 4 (ks >> 2)
      const uint2 w = on ? src[4 * (c + 4 * (ks >> 2)) + (ks & 3)] : make_uint2(0u, 0u);
      qa[ks][0] = w.x;
      qa[ks][1] = w.y;
    }
  }
  __device__ __forceinline__ void begin(const SpanParams&) {
    const float back = halves_of_q<KS>(qa);                 // of row lane / 4
    qinv[0] = __shfl_sync(kFull, back, 8 * (lane & 3));
    qinv[1] = __shfl_sync(kFull, back, 8 * (lane & 3) + 4);
    m[0] = m[1] = kNoScore;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
  }

  // half: bytes between tokens 0-15 and 16-31
  template <typename Release>
  __device__ __forceinline__ void unit(uint32_t kb, uint32_t vb, int, int half, const Sight& see,
                                       float scale_log2, const float2*, int, Release release) {
    const int g = lane >> 2, c = lane & 3;
    const uint32_t kt = kb + (4 * (g >> 1) + (g & 1)) * kRow4Bytes;
    const uint32_t vt = vb + 4 * c * kRow4Bytes;
    const uint32_t kp = kt + 8 * c, ks = kt + kRow4Codes + c, vp = vt + 8 * g, vq = vt + kRow4Codes + g;
    float sh[2][4];                                         // [16 tokens]: (token, row) as in O^T
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      sh[hf][0] = sh[hf][1] = sh[hf][2] = sh[hf][3] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t b[2][8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint2 w = lds64(kp + hf * half, 2 * n * kRow4Bytes + 32 * k);
          const uint32_t s = lds8(ks + hf * half, 2 * n * kRow4Bytes + 4 * k) * 0x00800080u;
          halves4_of(w.x, b[n][0], b[n][1], b[n][2], b[n][3]);
          halves4_of(w.y, b[n][4], b[n][5], b[n][6], b[n][7]);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[n][i] = mul_half2(b[n][i], s);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma_f16(sh[hf], b[0][2 * i], b[1][2 * i], b[0][2 * i + 1], b[1][2 * i + 1], qa[4 * k + i][0], qa[4 * k + i][1]);
      }
    }
    const float qs[2] = {qinv[0] * scale_log2, qinv[1] * scale_log2};
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int e = 0; e < 4; ++e) sh[hf][e] *= qs[e & 1];
    if (!see.all) {
      Sight next = see;
      next.last += later;
      next.first += later;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((e & 1) ? next : see).sees(16 * hf + 4 * (g >> 1) + (g & 1) + (e & 2))) sh[hf][e] = -INFINITY;
    }
    float alpha[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(fmaxf(sh[0][h], sh[0][2 + h]), fmaxf(sh[1][h], sh[1][2 + h]));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
      const float mn = fmaxf(m[h], mx);
      alpha[h] = fast_exp2(m[h] - mn);
      m[h] = mn;
      float sum = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          sh[hf][e + h] = fast_exp2(sh[hf][e + h] - mn);
          sum += sh[hf][e + h];
        }
      l[h] = l[h] * alpha[h] + sum;
    }
    // the rows' weights of a token, turned into the tokens' of a row: P^T's fragment
    uint32_t pb[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      pb[n] = transpose8x8(pack_half2(sh[n >> 1][2 * (n & 1)] * 1024.f, sh[n >> 1][2 * (n & 1) + 1] * 1024.f));
    if (__any_sync(kFull, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] *= alpha[0];
        o[mt][1] *= alpha[1];
        o[mt][2] *= alpha[0];
        o[mt][3] *= alpha[1];
      }
    }
    constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint2 vw[4];
      uint32_t vs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vw[i] = lds64(vp + hf * half, i * kRow4Bytes);
        vs[i] = lds8(vq + hf * half, i * kRow4Bytes);
      }
      if (hf == 1) release();
      const uint32_t s01 = (vs[0] << 7) + vs[1] * 0x00800000u;
      const uint32_t s23 = (vs[2] << 7) + vs[3] * 0x00800000u;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = j ? vw[i].y : vw[i].x;
        uint32_t a0[4], a1[4], a2[4], a3[4];                // of tiles 4 j .. 4 j + 3
        halves4_of((x[0] & kLow) | ((x[1] << 4) & ~kLow), a0[0], a0[1], a0[2], a0[3]);
        halves4_of(((x[0] >> 4) & kLow) | (x[1] & ~kLow), a1[0], a1[1], a1[2], a1[3]);
        halves4_of((x[2] & kLow) | ((x[3] << 4) & ~kLow), a2[0], a2[1], a2[2], a2[3]);
        halves4_of(((x[2] >> 4) & kLow) | (x[3] & ~kLow), a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          mma_f16(o[4 * j + t], mul_half2(a0[t], s01), mul_half2(a1[t], s01), mul_half2(a2[t], s23),
                  mul_half2(a3[t], s23), pb[2 * hf], pb[2 * hf + 1]);
      }
    }
  }

  __device__ __forceinline__ void store(float* macc, float* ml) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float lt = l[h] + __shfl_xor_sync(kFull, l[h], 4);
      lt += __shfl_xor_sync(kFull, lt, 8);
      lt += __shfl_xor_sync(kFull, lt, 16);
      if (g == 0 && 2 * c + h < rows) {
        ml[(2 * c + h) * 2] = m[h];
        ml[(2 * c + h) * 2 + 1] = lt;
      }
    }
    constexpr float kBack = 1.f / 1024.f;
#pragma unroll
    for (int mt = 0; mt < MT; mt += 2)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (2 * c + h < rows)
          *reinterpret_cast<float4*>(macc + (2 * c + h) * D + 16 * g + 2 * mt) =
              make_float4(o[mt][h] * kBack, o[mt][2 + h] * kBack, o[mt + 1][h] * kBack, o[mt + 1][2 + h] * kBack);
  }
};

// float32 on the CUDA cores.  Scores: 8 lanes a token, 4 tokens a pass, a lane head_dim / 8
// columns of every row; the butterfly leaves a lane the scores of one row (g_lane), whose
// maximum and sum it keeps.  Values: a lane head_dim / 32 columns of every row.  (One
// maximum a lane, sent round by shuffles, not one of every row and a choice among them:
// the compiler makes that choice an address, and the whole state then lives in local
// memory: 64 sequences of 2000 tokens, 8 kv heads of 8 rows of 128, 221 us instead of 190.)
// q's rows are in registers; 8 rows of 128 would take 128 of them and stand in the warp's
// shared memory.
template <int D, int G>
struct F32Rows {
  using Tr = DecodeTraits<false, D, G>;
  static constexpr int TU = Tr::UT, NCH = Tr::NCH, EPL = Tr::EPL, CPL = Tr::CPL, NP = Tr::P;
  static constexpr bool kShared = span_q_shared(SpanPool::kF32, D, G);
  static constexpr int LANES = 8 / G;   // lanes of 8 that hold a row's scores
  float qf[kShared ? 1 : G][EPL];
  float acc[G][CPL];
  float m, lsum;                        // of row g_lane: its maximum, this lane's share of its sum
  int lane, j4, r, base, g_lane;
  float* ps;                            // this warp's probabilities [TU][G]
  float4* qs;                           // this warp's rows of q [G][D / 4]

  __device__ __forceinline__ void init(const SpanParams&, int lane_, float* ps_, float* qs_) {
    lane = lane_;
    j4 = lane >> 3;
    r = lane & 7;
    // the sums that the butterfly leaves here: base .. base + RC - 1 of [row][pass]
    base = ((r >> 2) & 1) * (Tr::N / 2) + (Tr::N >= 4 ? ((r >> 1) & 1) * (Tr::N / 4) : 0) +
           (Tr::N >= 8 ? (r & 1) * (Tr::N / 8) : 0);
    g_lane = base / NP;
    ps = ps_;
    qs = reinterpret_cast<float4*>(qs_);
  }
  __device__ __forceinline__ int row() const { return g_lane; }

  __device__ __forceinline__ void load(const SpanParams& p, int b, int head) {
    if constexpr (kShared) __syncwarp();                    // (the last segment's reads are done)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float4* src = reinterpret_cast<const float4*>(p.q + query_row(p, b, head, g) * (4 * D));
      if constexpr (kShared) {
        static_assert(!kShared || D == 128, "a chunk a lane");
        const float4 w = src[lane];
        qs[g * (D / 4) + lane] = make_float4(w.x * p.scale_log2, w.y * p.scale_log2, w.z * p.scale_log2,
                                             w.w * p.scale_log2);
      } else {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const float4 w = src[r + 8 * c];
          qf[g][4 * c] = w.x; qf[g][4 * c + 1] = w.y; qf[g][4 * c + 2] = w.z; qf[g][4 * c + 3] = w.w;
        }
      }
    }
  }
  __device__ __forceinline__ void begin(const SpanParams& p) {
    if constexpr (kShared) __syncwarp();
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if constexpr (!kShared) {
#pragma unroll
        for (int e = 0; e < EPL; ++e) qf[g][e] *= p.scale_log2;
      }
#pragma unroll
      for (int c = 0; c < CPL; ++c) acc[g][c] = 0.f;
    }
    m = kNoScore;
    lsum = 0.f;
  }

  template <typename Release>
  __device__ __forceinline__ void unit(uint32_t kb, uint32_t vb, int, int, const Sight& see, float,
                                       const float2*, int, Release release) {
    const char* kt = static_cast<const char*>(__cvta_shared_to_generic(kb));
    const char* vt = static_cast<const char*>(__cvta_shared_to_generic(vb));
    float part[Tr::N], kf[NP][EPL];
#pragma unroll
    for (int pi = 0; pi < NP; ++pi)
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        unpack_chunk<Tr>(*reinterpret_cast<const uint4*>(kt + (4 * pi + j4) * Tr::ROW_BYTES + (r + 8 * c) * 16),
                         &kf[pi][c * Tr::CE]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float q[EPL];
      if constexpr (kShared) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const float4 w = qs[g * (D / 4) + r + 8 * c];
          q[4 * c] = w.x; q[4 * c + 1] = w.y; q[4 * c + 2] = w.z; q[4 * c + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < EPL; ++e) q[e] = qf[g][e];
      }
#pragma unroll
      for (int pi = 0; pi < NP; ++pi) {
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) dot = fmaf(q[e], kf[pi][e], dot);
        part[g * NP + pi] = dot;
      }
    }
    butterfly_level<Tr::N>(part, lane, 4);
    butterfly_level<(Tr::N >= 4 ? Tr::N / 2 : 1)>(part, lane, 2);
    butterfly_level<(Tr::N >= 8 ? Tr::N / 4 : 1)>(part, lane, 1);
    float umax = -INFINITY;
#pragma unroll
    for (int e = 0; e < Tr::RC; ++e) {
      const int t = 4 * ((base % NP) + e) + j4;
      if (!see.all && !see.sees(t)) part[e] = -INFINITY;
      umax = fmaxf(umax, part[e]);
    }
#pragma unroll
    for (int mask = 1; mask < LANES; mask <<= 1) umax = fmaxf(umax, __shfl_xor_sync(kFull, umax, mask));
    umax = fmaxf(umax, __shfl_xor_sync(kFull, umax, 8));
    umax = fmaxf(umax, __shfl_xor_sync(kFull, umax, 16));
    const float mn = fmaxf(m, umax);
    const float alpha = fast_exp2(m - mn);
    m = mn;
    float psum = 0.f;
#pragma unroll
    for (int e = 0; e < Tr::RC; ++e) {
      const int t = 4 * ((base % NP) + e) + j4;
      const float pr = fast_exp2(part[e] - mn);
      psum += pr;
      ps[t * G + g_lane] = pr;                              // lanes with the same sum store the same value
    }
    lsum = lsum * alpha + psum;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float f = __shfl_sync(kFull, alpha, g * LANES);
#pragma unroll
      for (int c = 0; c < CPL; ++c) acc[g][c] *= f;
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < TU; ++t) {
      float vv[CPL], w[G];
      load_v_cols<Tr>(vt, t, lane, vv);
      if constexpr (G >= 4) {
#pragma unroll
        for (int g = 0; g < G; g += 4) {
          const float4 x = *reinterpret_cast<const float4*>(ps + t * G + g);
          w[g] = x.x; w[g + 1] = x.y; w[g + 2] = x.z; w[g + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = ps[t * G + g];
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc[g][c] = fmaf(w[g], vv[c], acc[g][c]);
    }
    release();
  }

  // to macc [G][D] and ml [G][(maximum, sum)]
  __device__ __forceinline__ void store(float* macc, float* ml) {
#pragma unroll
    for (int mask = Tr::DUP_MASK_END; mask < LANES; mask <<= 1) lsum += __shfl_xor_sync(kFull, lsum, mask);
    lsum += __shfl_xor_sync(kFull, lsum, 8);
    lsum += __shfl_xor_sync(kFull, lsum, 16);
    if (j4 == 0 && (r % LANES) == 0) {
      ml[g_lane * 2] = m;
      ml[g_lane * 2 + 1] = lsum;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float* dst = macc + g * D + lane * CPL;
      if constexpr (CPL == 4)
        *reinterpret_cast<float4*>(dst) = make_float4(acc[g][0], acc[g][1], acc[g][2], acc[g][3]);
      else
        *reinterpret_cast<float2*>(dst) = make_float2(acc[g][0], acc[g][1]);
    }
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
  __device__ __forceinline__ void store_peer(uint32_t a) const {
    if constexpr (CPL == 4) peer_store(a, v[0], v[1], v[2], v[3]);
    else peer_store(a, v[0], v[1]);
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

// 1 / l, or 0 where no token was seen (l = 0: the row is zeros); NaN stays.
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }
// Base-2 logarithm of the sum under maximum m.
__device__ __forceinline__ float log_sum(float m, float l) {
  return l > 0.f ? m + __log2f(l) : (l != l ? l : -INFINITY);
}

template <SpanPool P, int D, int G>
struct RowsOf;
template <int D, int G>
struct RowsOf<SpanPool::kBf16, D, G> { using type = Bf16Rows<D>; };
template <int G>
struct RowsOf<SpanPool::kFp8, 128, G> { using type = Fp8Rows; };
template <int G>
struct RowsOf<SpanPool::kFp4, 128, G> { using type = Fp4Rows; };
template <int D, int G>
struct RowsOf<SpanPool::kF32, D, G> { using type = F32Rows<D, G>; };

// Stages that the table is read ahead, and the scales of e4m3 pages (whose addresses the
// table gives).  More (5 and 2, 6 and 3) only lengthen the start: 144.1 us for 256
// sequences of e4m3 pages with these, 144.6 and 145.9; small calls 6.4, 6.6 and 6.8.
constexpr int kAhead = 3, kScaleAhead = 1;

template <SpanPool P, int D, int G>
__global__ void __launch_bounds__(kSpanThreads, 1) span_decode_kernel(const __grid_constant__ SpanParams p) {
  using Rows = typename RowsOf<P, D, G>::type;
  constexpr int TU = span_tile_tokens(P, D);
  constexpr int ROW = span_row_bytes(P, D);
  constexpr int STAGE = span_stage_bytes(P, D);
  constexpr bool FP4 = P == SpanPool::kFp4;
  constexpr int SLABS = P == SpanPool::kF32 || FP4 ? 1 : ROW / 128;
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
  // clusters: [row / splits][CTA] states of the rows that this CTA joins
  float* joint = reinterpret_cast<float*>(smem + at.total);
  float* joint_ml = joint + p.joint_slots * D;

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
  if (p.splits > 1) cluster_arrive();                        // waited for before the first store to a peer
  if (!FP4 && threadIdx.x == 32) {
    prefetch_map(&p.map_k);
    prefetch_map(&p.map_v);
  }
  wait_prior_grids();
  allow_next_grid();
  __syncthreads();

  // ---- this CTA's stages: from stage st0 of segment (b0, grp0), cnt of them
  int b0, grp0, st0, cnt, len0, rank = 0;
  if (p.splits) {
    rank = blockIdx.x;
    grp0 = blockIdx.y;
    b0 = blockIdx.z;
    const int len = p.lens[b0];
    len0 = len;
    if (threadIdx.x == 0 && rank == 0 && grp0 == 0 &&
        (len < 0 || len > p.max_len || (len > 0 && len < p.q_len)))
      report(p.device_errors, PA_DEVERR_BAD_LENGTH);
    const int nst = make_span<TU>(p, len).nst;
    // (exact: nst < 2^28, splits <= 8)
    const int each = p.splits > 1 ? static_cast<int>(__umulhi(static_cast<uint32_t>(nst), p.over_splits)) : nst;
    const int rest = nst - each * p.splits;
    st0 = each * rank + min(rank, rest);
    cnt = each + (rank < rest ? 1 : 0);
  } else {
    // every CTA adds up the stages of all sequences: thread t a run of them
    const int per = (p.num_seqs + kSpanThreads - 1) / kSpanThreads;
    const int s0 = min(static_cast<int>(threadIdx.x) * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
    long long sum = 0;
    bool bad = false;
    int last_len = 0;
    for (int b = s0; b < s1; ++b) {
      const int len = p.lens[b];
      last_len = len;
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
    const long long share = share_of(total, gridDim.x);
    const long long begin_at = min(share * blockIdx.x, total);
    cnt = static_cast<int>(min(begin_at + share, total) - begin_at);
    if (cnt > 0 && before <= begin_at && begin_at < before + sum * p.ngroups) {
      for (int b = s0; b < s1; ++b) {
        const int len = per == 1 ? last_len : p.lens[b];
        const int nst = make_span<TU>(p, len).nst;
        const long long n = static_cast<long long>(nst) * p.ngroups;
        if (begin_at < before + n) {
          const int rem = static_cast<int>(begin_at - before);
          int* start = reinterpret_cast<int*>(scan + kSpanWarps + 1);
          start[0] = b;
          start[1] = rem / nst;
          start[2] = rem % nst;
          start[3] = len;
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
    len0 = start[3];
    if (cnt <= 0) return;
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

    Walk<TU> wk(p, b0, grp0, len0);
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
    float sc_queue[kScaleAhead];
    if constexpr (FP8) {
#pragma unroll
      for (int k = 0; k < kScaleAhead; ++k) sc_queue[k] = scale_of(q_phys[k], q_vis[k], q_head[k]);
    }
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
        if constexpr (FP4)                                   // whole pages, of all the CTA's heads in one piece
          bulk_g2s(dst, (kv ? p.v_pool : p.k_pool) + static_cast<int64_t>(z) * p.block_size * ROW, op_bytes, &full[s]);
        else if constexpr (SLABS > 1)
          tma_load_4d(dst, map, 0, q_off[0], z, 0, &full[s]);
        else
          tma_load_3d(dst, map, 0, q_off[0], z, &full[s]);
      }
      if constexpr (FP8) {
        sc[s * 32 + lane] = sc_queue[0];
#pragma unroll
        for (int k = 0; k + 1 < kScaleAhead; ++k) sc_queue[k] = sc_queue[k + 1];
        sc_queue[kScaleAhead - 1] = scale_of(q_phys[kScaleAhead], q_vis[kScaleAhead], q_head[kScaleAhead]);
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
    rows.init(p, lane, reinterpret_cast<float*>(smem + at.ps) + warp * TU * p.rows,
              reinterpret_cast<float*>(smem + at.qs) + warp * p.rows * D);
    Walk<TU> wk(p, b0, grp0, len0);
    int s = 0, left = cnt, st = st0;
    uint32_t parity = 0;
    bool first_seg = true, aborted = false;
    rows.load(p, wk.b, (wk.grp << p.hg_log2) + hl);
    for (;;) {
      const Span sp = wk.sp;
      const int st_end = min(sp.nst, st + left);
      const int st_begin = st, seg_b = wk.b, seg_grp = wk.grp;
      const int head = (seg_grp << p.hg_log2) + hl;
      rows.begin(p);
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
            if constexpr (FP4) {
              // (a code is always finite: the scales are all there is to clear)
              static_assert(!FP4 || TU == 32, "a token a lane");
              const int tt = t0 + lane;
              if (tt >= sp.len || (tt >= p.sinks && tt < sp.lo) || ((bad >> (lane >> 4)) & 1u))
                asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(vb + (lane >> 4) * half + (lane & 15) * ROW + kRow4Codes),
                             "r"(0u) : "memory");
            }
            for (int i = FP4 ? TU * (ROW / 16) : lane; i < TU * (ROW / 16); i += 32) {
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
      if (left > 0) {
        wk.next();
        rows.load(p, wk.b, (wk.grp << p.hg_log2) + hl);
      }
      // ---- the segment's part is done: join the head's warps.  Rows go round them; the
      // lanes hold the warps' (or, of a warp alone, the rows') maxima and sums, so that no
      // row waits for another's.
      rows.store(macc + warp * p.rows * D, mml + warp * p.rows * 2);
      // (the warps agree on giving up, so that none waits at a barrier for one that left)
      if (wph > 1 || p.splits) aborted = consumer_barrier_any(aborted); else __syncwarp();
      const int R = hg * p.rows;
      const bool whole = st_begin == 0 && st_end == sp.nst;
      const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + (first_seg ? 0 : 1)) * R + hl * p.rows;
      auto put = [&](int r, Cols<CPL>& acc, float inv, float lse) {
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc.v[c] *= inv;
        if (whole) {
          acc.template store_out<BF16_OUT>(p.out, query_row(p, seg_b, head, r) * D + lane * CPL);
        } else {
          acc.store(p.part_out + (part0 + r) * D + lane * CPL);
          if (lane == 0) p.part_lse[part0 + r] = lse;
        }
      };
      if (wph == 1 && p.splits <= 1) {
        const float2 ml = lane < p.rows ? reinterpret_cast<const float2*>(mml + warp * p.rows * 2)[lane]
                                        : make_float2(0.f, 0.f);
        const float inv = inverse_sum(ml.y), lse = log_sum(ml.x, ml.y);
#pragma unroll 4
        for (int r = 0; r < p.rows; ++r) {
          Cols<CPL> acc;
          acc.load(macc + (warp * p.rows + r) * D + lane * CPL);
          put(r, acc, __shfl_sync(kFull, inv, r), __shfl_sync(kFull, lse, r));
        }
      } else {
        const int w0 = hl << wph_log2;
        if (p.splits > 1) cluster_wait();                    // every CTA of the cluster runs
        for (int r = sub; r < p.rows; r += wph) {
          const float2 ml = lane < wph ? reinterpret_cast<const float2*>(mml)[(w0 + lane) * p.rows + r]
                                       : make_float2(kNoScore, 0.f);
          Cols<CPL> x[kSpanWarps];
#pragma unroll
          for (int w = 0; w < kSpanWarps; ++w)               // (a head with fewer warps: its last again, weight 0)
            x[w].load(macc + ((w0 + min(w, wph - 1)) * p.rows + r) * D + lane * CPL);
          float M = ml.x;
#pragma unroll
          for (int o = 1; o < kSpanWarps; o <<= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
          const float f = lane < wph ? fast_exp2(ml.x - M) : 0.f;
          float lam = f * ml.y;
#pragma unroll
          for (int o = 1; o < kSpanWarps; o <<= 1) lam += __shfl_xor_sync(kFull, lam, o);
          M = __shfl_sync(kFull, M, 0);
          lam = __shfl_sync(kFull, lam, 0);
          Cols<CPL> acc;
#pragma unroll
          for (int c = 0; c < CPL; ++c) acc.v[c] = 0.f;
#pragma unroll
          for (int w = 0; w < kSpanWarps; ++w) {
            const float fw = __shfl_sync(kFull, f, w);
#pragma unroll
            for (int c = 0; c < CPL; ++c) acc.v[c] = fmaf(fw, x[w].v[c], acc.v[c]);
          }
          if (p.splits > 1) {
            // to the CTA of the cluster that joins this row
            const int row = hl * p.rows + r;
            const int to = row - static_cast<int>(__umulhi(row, p.over_splits)) * p.splits, slot = row - to + rank;
            acc.store_peer(peer_addr(smem_addr(joint + slot * D + lane * CPL), to));
            if (lane == 0) peer_store(peer_addr(smem_addr(joint_ml + slot * 2), to), M, lam);
          } else {
            put(r, acc, inverse_sum(lam), log_sum(M, lam));
          }
        }
      }
      if (left <= 0 || aborted) break;
      if (wph > 1) consumer_barrier(); else __syncwarp();      // the states have been read
      first_seg = false;
      st = 0;
    }
  }

  if (p.splits > 1) {
    // ---- the cluster joins its CTAs' states: row r in CTA r mod splits, where every CTA
    // has put its own (which nobody has to read across the cluster or wait for to leave)
    if (warp == kSpanWarps) cluster_wait();
    cluster_arrive();
    cluster_wait();
    if (warp < kSpanWarps) {
      const int R = hg * p.rows;
      for (int r = warp * p.splits + rank; r < R; r += kSpanWarps * p.splits) {
        const int slot = r - rank;                           // of CTA 0's state
        const float2 ml = lane < p.splits ? reinterpret_cast<const float2*>(joint_ml)[slot + lane]
                                          : make_float2(kNoScore, 0.f);
        Cols<CPL> x[kSpanCluster];
#pragma unroll
        for (int c = 0; c < kSpanCluster; ++c)
          if (c < p.splits) x[c].load(joint + (slot + c) * D + lane * CPL);
        float M = ml.x;
#pragma unroll
        for (int o = 1; o < kSpanCluster; o <<= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
        M = __shfl_sync(kFull, M, 0);
        const float f = fast_exp2(ml.x - M);
        float lam = f * ml.y;
#pragma unroll
        for (int o = 1; o < kSpanCluster; o <<= 1) lam += __shfl_xor_sync(kFull, lam, o);
        const float inv = inverse_sum(__shfl_sync(kFull, lam, 0));
        Cols<CPL> acc;
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc.v[c] = 0.f;
#pragma unroll
        for (int c = 0; c < kSpanCluster; ++c)
          if (c < p.splits) {
            const float fc = __shfl_sync(kFull, f, c);
#pragma unroll
            for (int e = 0; e < CPL; ++e) acc.v[e] = fmaf(fc, x[c].v[e], acc.v[e]);
          }
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc.v[c] *= inv;
        const int h = r / p.rows;
        acc.template store_out<BF16_OUT>(
            p.out, query_row(p, b0, (grp0 << p.hg_log2) + h, r - h * p.rows) * D + lane * CPL);
      }
    }
  }
}

// The opt-in of an instance to more than 48 KiB of dynamic shared memory, once a device.
template <SpanPool P, int D, int G>
cudaError_t configure_span(int* device) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = cudaGetDevice(device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (*device & 63);
  if (configured.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(span_decode_kernel<P, D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpanSmem);
  if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Launch of one instance: a plain grid of shares, or a grid (splits, head groups,
// sequences) of clusters of p.splits CTAs.
template <SpanPool P, int D, int G>
cudaError_t run_span(const SpanParams& p, dim3 grid, int smem, cudaStream_t stream) {
  int device = 0;
  const cudaError_t e = configure_span<P, D, G>(&device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
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
