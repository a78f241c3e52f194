// Prompt attention over paged bf16 pools on the fifth-generation tensor cores.
//
// Mathematics.  Row (token j, head i of the group) of a tile sees keys t <= p_j (and, with a
// window, p_j - t < window or t < sinks):
//   O = sum_t 2^(s_t - m) V_t / sum_t 2^(s_t - m),   s_t = scale log2(e) <q, K_t>,
// in one pass over the keys, 128 at a time, with a reference m that follows the running
// maximum.  Scores, m and the sums are float32; the weights are rounded to bf16 for the
// product with V (2^-8 of each; a second part of each weight would cost a third product
// beside the two).
//
// What bounds it: the products.  A step of 128 keys for 256 rows of 128 columns is 16.8
// MFLOP (2048 clocks of the tensor cores), 64 KiB of K and V and 32768 exponentials (1024
// clocks).  On a GB300 (1990 TFLOP/s of bf16 products measured, 1738 in a long run), 32 query
// and 8 kv heads of 128, first in a graph of a few calls and then among calls that keep the GPU
// busy for longer: one prompt of 16384 tokens 1327 to 1360 us and 1415 to 1440, 1530 to 1660
// TFLOP/s of what causality leaves; 12 ragged prompts, 17569 tokens, 235 and 243 to 247, 1160 to
// 1220; 6 chunks of 200 to 512 tokens behind up to 15000 253 and 259 to 263, 1220 to 1270; one
// prompt of 37 tokens 6.5.  Heads of 64 have the same exponentials for half the products, and
// their steps take about as long: 4 prompts of 4096 tokens of 16 heads 171 us, 806 TFLOP/s; 4
// prompts, 12802 tokens, in windows of 1024 117.
//
// Layout of the work:
//   * An item is a kv head and a tile of 256 rows: 256 / G consecutive new tokens of a
//     sequence with all G query heads of the head, so K and V are read once for the group.
//     Its rows are two products of 128 (M = 128).  While one half's scores are in softmax
//     the tensor cores work for the other: S0, S1 (128 columns each), O0 and O1 fill the
//     512 columns of tensor memory.
//   * A warp for each half issues its products, in turns, through one of its lanes.  (A warp
//     whose values stay uniform: 1492 us for the prompt of 16384 when a single thread took
//     1588.)
//   * The weights are written back to tensor memory over the scores they came from (bf16, 64
//     columns) and enter the second product from there: shared memory feeds V alone then,
//     while both operands of the first product come from it, which is just its rate.
//   * One warp brings K and V through one ring of tiles, page by page (a page's rows of a
//     head are one box of 128-byte rows for each slab of K, one box for all of V: the copy
//     engine takes 40 ns for a box of 2 KiB and 60 for one of 4, so the 24 boxes of a step
//     of 16-token pages keep ahead of its products).
//   * V rows that no row of the tile sees (past its last key, behind the window) may hold
//     anything; where a tile has such rows beside others a warp clears them before the
//     product.  Their weights are zeros.
//   * The reference is the first step's maximum and moves only when the weights of a row's
//     step come to more than 2^16 (bf16 has float32's range, so they may pass 1), so O is
//     hardly ever rescaled, and the other steps take no maximum: 128 keys of 32 rows cost a
//     warp alone 750 clocks instead of 1030.
//   * Every wait is bounded; on expiry the kernel reports PA_DEVERR_TIMEOUT, waits for its
//     own copies and products, frees its tensor memory and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "paged_decode.cuh"
#include "prefill.h"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kSoftmaxWarps = 8;                           // four for each half of the rows
constexpr int kProducer = 8, kIssuer = 9, kCleaner = 10, kIssuerStep = 2;   // issuers: warps 9 and 11
constexpr int kThreadsPrefill = 12 * 32;
constexpr float kMostSum = 65536.f;                        // of a row's weights in one step
constexpr int kBadRing = 8;
constexpr uint32_t kPatientPolls = 1u << 28;               // a quarter of an hour
constexpr uint32_t kTmemO = 256;                           // column of O0; S0 is column 0

template <int D>
struct PrefillLayout {
  static constexpr int SLABS = D / 64;
  static constexpr int Q_SLAB = 128 * 128;                 // 128 rows of 64 columns
  static constexpr int Q_HALF = SLABS * Q_SLAB;
  static constexpr int TILE = kPrefillKeys * D * 2;
  static constexpr int RING = D == 128 ? 4 : 8;            // (5 of 32 KiB are no faster)
  static constexpr int OFF_RING = 2 * Q_HALF;
  static constexpr int OFF_STAGE = OFF_RING + RING * TILE; // 32 rows of 128 bytes a softmax warp
  static constexpr int OFF_BAD = OFF_STAGE + kSoftmaxWarps * 32 * 128;
  static constexpr int OFF_BARS = OFF_BAD + kBadRing * 4;
  // full, empty, raw [RING]; q_full, q_empty; s_full, p_full, pv_done, o_free, turn [2]; end
  static constexpr int NUM_BARS = 3 * RING + 2 + 10 + 1;
  static constexpr int SMEM = OFF_BARS + NUM_BARS * 8 + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory over budget");
};

__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(kFull, x, 0); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return (static_cast<uint64_t>(hi) << 32) | lo; }

// The wait before tcgen05.ld's registers are used, tied to them.
template <int N>
__device__ __forceinline__ void tmem_landed(float (&v)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// Two floats at once (half the instructions; a warp's scheduler is as busy as its
// exponentials otherwise), and the largest of three.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The lowest n bits of a word, n of any size.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Two kinds of waits may rightly last as long as whole items take: the clearing warp's, and those of
// the second half's softmax behind items that have no rows for it.  They end with the wait of some
// other warp, for nothing stands still without one of the producer's or the issuers' waits, which
// are of one stage, running out and raising the flag.  (In every wait of the softmax this costs 1 to
// 2 % of windows; going along with the ring's steps instead costs up to 5 % of many short chunks.)
__device__ __forceinline__ bool patient_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  for (uint32_t i = 0; i < kPatientPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  return false;
}

template <int D>
__global__ void __launch_bounds__(kThreadsPrefill, 1) prefill_bf16_kernel(const __grid_constant__ PrefillParams p) {
  using Ly = PrefillLayout<D>;
  constexpr int R = Ly::RING;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  volatile uint32_t* bad_ring = reinterpret_cast<volatile uint32_t*>(smem + Ly::OFF_BAD);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly::OFF_BARS);
  uint64_t* empty = full + R;
  uint64_t* raw = empty + R;                               // V landed, rows to be cleared yet
  uint64_t* q_full = raw + R;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* o_free = pv_done + 2;
  uint64_t* turn = o_free + 2;                             // which half's products are next
  uint64_t* end = turn + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(end + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_tokens = kPrefillRows >> p.group_log2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);                             // both halves
      mbar_init(&raw[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&turn[i], 1);
    }
    mbar_init(end, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kIssuer) {
    // (one CTA per SM by its shared memory, so the columns are always free)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_prior_grids();                                      // the plan's list
  allow_next_grid();
  auto fail = [&]() {
    if (!*abort_flag) {
      report(p.device_errors, PA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    // (the flag is not looked at where the first poll says yes, as it nearly always does)
    return mbar_try_wait(bar, parity) || (!*abort_flag && mbar_wait(bar, parity, p.wait_limit));
  };
  PrefillWalk<kPrefillKeys> walk(p, tile_tokens);
  PrefillItem it;
  // keys [x, y) of a step that starts at key t0 are behind the window and no sinks
  auto hidden = [&](const PrefillTile& t, int t0, int hi, int& x, int& y) {
    x = max(t0, p.sinks);
    y = min(t.lo, hi);
    return x < y;
  };

  // A softmax thread holds a row's 128 scores.  The block has 384 * 168 = 64512 registers:
  // 256 * 184 + 128 * 136.  (The compiler allots 168 to all and spills 40 bytes.)
  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
    if (warp == kProducer) {
      // ------------------------------------------------------------ copies
      const int bs = p.block_size, pages_of_step = kPrefillKeys >> p.block_log2;
      const int j = lane / Ly::SLABS, slab = lane % Ly::SLABS;   // of K: page of the step, slab
      uint32_t c = 0, steps = 0, raw_used = 0, raw_parity = 0;   // ring slots filled; raw: a bit a slot
      bool ok = true;
      int items_done = 0;
      while (ok && walk.next(it)) {
        if (it.t.steps <= 0) continue;
        if (lane == 0) {                                     // q, once the last item's is no longer read
          ok = wait(q_empty, (items_done & 1) ^ 1);
          if (ok) {
            const int halves = (it.t.tokens << p.group_log2) > 128 ? 2 : 1;
            mbar_arrive_expect_tx(q_full, halves * Ly::Q_HALF);
            for (int i = 0; i < halves; ++i)
              for (int s = 0; s < Ly::SLABS; ++s)
                tma_load_4d(smem + i * Ly::Q_HALF + s * Ly::Q_SLAB, &p.map_q, 64 * s, 0, it.h,
                            it.t.row0 + i * (tile_tokens / 2), q_full);
          }
        }
        ok = __shfl_sync(kFull, ok, 0);
        if (!ok) break;
        ++items_done;
        const int32_t* table = p.tables + static_cast<int64_t>(it.b) * p.max_blocks;
        // lane l: page l of a step, as a row of the pool's map (-1: not there, reads zeros;
        // -2: nobody sees it, not read); the next step's is looked up ahead
        auto look = [&](int v) {
          if (v >= it.v1 || lane >= pages_of_step) return -2;
          const int first = (v + (v >= it.t.ns ? it.t.shift : 0)) * kPrefillKeys + lane * bs;
          if (first >= it.t.end || (first >= p.sinks && first + bs <= it.t.lo)) return -2;
          const int page = table[first >> p.block_log2];
          return page >= 0 && page < p.num_blocks ? page * p.num_kv_heads + it.h : -1;
        };
        int ahead = look(it.v0);
        // (no polls: given up for certain, behind a step whose copies are in flight.  Asked in the
        // first poll of every wait this would cost 2 to 3 %, and for each step 0.6.)
        const int v_end = p.wait_limit != 0 ? it.v1 : it.v0 + 1;
        for (int v = it.v0; v < v_end; ++v, ++steps) {
          const int z = ahead;
          ahead = look(v + 1);
          const int t0 = (v + (v >= it.t.ns ? it.t.shift : 0)) * kPrefillKeys, hi = min(it.t.end, t0 + kPrefillKeys);
          const uint32_t there = __ballot_sync(kFull, z != -2), gone = __ballot_sync(kFull, z == -1);
          const int bytes = __popc(there) * bs * D * 2;
          // ---- K
          int slot = c % R;
          if (lane == 0) ok = wait(&empty[slot], ((c / R) & 1) ^ 1);
          ok = __shfl_sync(kFull, ok, 0);
          if (!ok) break;
          if (lane == 0) {
            if (gone) report(p.device_errors, PA_DEVERR_BAD_BLOCK);
            uint32_t word = gone;                            // a bit for each 16 keys
            if (bs == 32) {
              word = 0;
              for (int i = 0; i < 4; ++i)
                if ((gone >> i) & 1) word |= 3u << (2 * i);
            }
            bad_ring[steps % kBadRing] = word;
            mbar_arrive_expect_tx(&full[slot], bytes);
          }
          raw_used &= ~(1u << slot);
          __syncwarp();
          const int zk = __shfl_sync(kFull, z, j < pages_of_step ? j : 0);
          if (j < pages_of_step && zk != -2)
            tma_load_4d(smem + Ly::OFF_RING + slot * Ly::TILE + slab * Ly::Q_SLAB + j * bs * 128, &p.map_k, 0, 0, zk,
                        slab, &full[slot]);
          ++c;
          // ---- V
          slot = c % R;
          if (lane == 0) ok = wait(&empty[slot], ((c / R) & 1) ^ 1);
          ok = __shfl_sync(kFull, ok, 0);
          if (!ok) break;
          int x, y;
          const bool clear = (hi & 15) != 0 || hidden(it.t, t0, hi, x, y);
          uint64_t* bar = clear ? &raw[slot] : &full[slot];
          raw_used = clear ? raw_used | 1u << slot : raw_used & ~(1u << slot);
          if (clear) raw_parity ^= 1u << slot;
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (z >= -1)
            tma_load_4d(smem + Ly::OFF_RING + slot * Ly::TILE + lane * bs * D * 2, &p.map_v, 0, 0, z, 0, bar);
          ++c;
        }
        ok = ok && p.wait_limit != 0;
      }
      if (!ok && lane == 0) fail();
      // the copies still in flight must land before the shared memory is released
      if (lane == 0) {
        for (uint32_t i = c > R ? c - R : 0; i < c; ++i) {
          const int slot = i % R;
          if ((raw_used >> slot) & 1) mbar_wait(&raw[slot], ((raw_parity >> slot) & 1) ^ 1);
          else mbar_wait(&full[slot], (i / R) & 1);
        }
        if (items_done > 0) mbar_wait(q_full, (items_done - 1) & 1);
      }
    } else if (warp == kCleaner) {
      // ------------------------------------------------------------ V rows that nobody sees
      uint32_t c = 0, raw_parity = 0;
      bool ok = true;
      while (ok && walk.next(it)) {
        if (it.t.steps <= 0) continue;
        for (int v = it.v0; v < it.v1 && ok; ++v, c += 2) {
          const int slot = (c + 1) % R;
          const int t0 = (v + (v >= it.t.ns ? it.t.shift : 0)) * kPrefillKeys, hi = min(it.t.end, t0 + kPrefillKeys);
          int x, y;
          const bool behind = hidden(it.t, t0, hi, x, y);
          if ((hi & 15) == 0 && !behind) continue;
          ok = patient_wait(&raw[slot], (raw_parity >> slot) & 1, abort_flag);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          raw_parity ^= 1u << slot;
          const uint32_t base = smem_addr(smem + Ly::OFF_RING + slot * Ly::TILE);
          const int bs = p.block_size;
          auto clear = [&](int from, int to) {
            for (int i = lane; i < (to - from) * (D / 8); i += 32) {
              const int t = from + i / (D / 8), ch = i % (D / 8), page = t >> p.block_log2, r = t & (bs - 1);
              const uint32_t a = base + page * bs * D * 2 + (ch >> 3) * bs * 128 + r * 128 + (ch & 7) * 16;
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
            }
          };
          clear(hi - t0, (hi - t0 + 15) & ~15);
          if (behind) clear(x - t0, y - t0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[slot]);
        }
      }
      if (!ok && lane == 0) fail();
    } else if (warp == kIssuer || warp == kIssuer + kIssuerStep) {
      // ------------------------------------------------------------ products: a warp for each half
      // (What is done between two products is not hidden behind them: the queue is short.  So
      // there are two issuers, slots are counted up instead of divided, descriptors differ from
      // ready ones by an addition.  The warp runs as one and a lane of it issues, with values
      // that the compiler knows to be the warp's: they stay in uniform registers.)
      {
        const int half = warp == kIssuer ? 0 : 1;
        const bool issues = elect_lane();
        const uint32_t ring = smem_addr(smem + Ly::OFF_RING);
        constexpr uint32_t kIdS = umma_idesc_bf16(128, kPrefillKeys, false), kIdPV = umma_idesc_bf16(128, D, true);
        const uint64_t qd0 = umma_desc(smem_addr(smem) + half * Ly::Q_HALF, 16, 1024);
        const uint64_t kd0 = umma_desc(ring, 16, 1024), vd0 = umma_desc(ring, p.block_size * 128, 1024);
        const uint32_t q_lo = uniform(static_cast<uint32_t>(qd0)), sbo = static_cast<uint32_t>(kd0 >> 32);
        const uint32_t k_lo0 = uniform(static_cast<uint32_t>(kd0)), v_lo0 = uniform(static_cast<uint32_t>(vd0));
        const uint32_t s_at = uniform(tmem + 128 * half), o_at = uniform(tmem + kTmemO + 128 * half);
        // from 16 keys to the next within V's tile: bs 16, a page; bs 32, 16 rows and then a page
        const uint32_t v_odd = (p.block_size == 16 ? 16 * D * 2 : 16 * 128) >> 4, v_even = (2 * 16 * D * 2) >> 4;
        struct Slot {
          uint32_t i, parity;
          __device__ __forceinline__ void next() {
            if (++i == R) {
              i = 0;
              parity ^= 1;
            }
          }
        } at{0, 0};
        uint32_t p_parity = 0, o_parity = 1, q_parity = 0, t_parity = half ^ 1;
        bool ok = true;
        // (the lanes agree on giving up, once a step: a vote takes as long as the wait before it)
        auto agreed = [&] { return ok = __all_sync(kFull, ok) != 0; };
        // S = this half's rows of q times the K tile in `slot`
        auto scores = [&](uint32_t slot, uint32_t id) {
          const uint32_t k_lo = uniform(k_lo0 + slot * (Ly::TILE >> 4));
          if (issues && ok) {
  #pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = ((ks >> 2) * Ly::Q_SLAB + (ks & 3) * 32) >> 4;
              umma_bf16(s_at, desc_of(q_lo + off, sbo), desc_of(k_lo + off, sbo), id, ks > 0 ? 1u : 0u);
            }
            umma_commit(&s_full[half]);
          }
          __syncwarp();
        };
        // O += the weights times the V tile in `slot`
        auto values = [&](uint32_t v_lo, int keys, uint32_t accumulate) {
          if (issues && ok) {
            if (keys == kPrefillKeys) {
  #pragma unroll
              for (int g = 0; g < kPrefillKeys / 16; ++g)
                umma_bf16_ts(o_at, s_at + 8 * g, desc_of(v_lo + (g >> 1) * v_even + (g & 1) * v_odd, sbo), kIdPV,
                             g > 0 ? 1u : accumulate);
            } else {
              for (int g = 0; 16 * g < keys; ++g)
                umma_bf16_ts(o_at, s_at + 8 * g, desc_of(v_lo + (g >> 1) * v_even + (g & 1) * v_odd, sbo), kIdPV,
                             g > 0 ? 1u : accumulate);
            }
            umma_commit(&pv_done[half]);
          }
          __syncwarp();
        };
        while (ok && walk.next(it)) {
          if (it.t.steps <= 0) continue;
          const int steps = it.v1 - it.v0;
          const bool two = (it.t.tokens << p.group_log2) > 128;
          // Products in turns, a step's of one half and then of the other: both halves' at once
          // would end, and their softmaxes begin, together, with the tensor cores idle meanwhile.
          auto my_turn = [&] {
            if (!two) return true;
            const bool mine = wait(&turn[half], t_parity);
            t_parity ^= 1;
            return mine;
          };
          auto pass_turn = [&] {
            if (two && issues) mbar_arrive(&turn[half ^ 1]);
          };
          if (half == 1 && !two) {
            // no rows for this half: the slots are given back as they come
            for (int i = 0; i < 2 * steps && ok; ++i) {
              ok = wait(&full[at.i], at.parity);
              if (agreed() && issues) mbar_arrive(&empty[at.i]);
              at.next();
            }
            if (ok) {
              ok = wait(q_full, q_parity);
              if (agreed() && issues) mbar_arrive(q_empty);
            }
            q_parity ^= 1;
            continue;
          }
          // (the last step is the only one that may be short)
          const int tail = min(kPrefillKeys, it.t.end - (it.v1 - 1 + (it.v1 - 1 >= it.t.ns ? it.t.shift : 0)) * kPrefillKeys);
          const uint32_t id_tail = umma_idesc_bf16(128, (tail + 15) & ~15, false);
          ok = wait(q_full, q_parity) && wait(&full[at.i], at.parity) && my_turn();
          if (!agreed()) break;
          q_parity ^= 1;
          tmem_fence_after();
          scores(at.i, steps == 1 ? id_tail : kIdS);
          pass_turn();
          if (issues) {
            umma_commit(&empty[at.i]);
            if (steps == 1) umma_commit(q_empty);
          }
          at.next();
          for (int v = 0; v < steps; ++v) {
            Slot kn = at;                                    // V of this step; K of the next
            kn.next();
            const bool next = v + 1 < steps;
            const uint32_t v_lo = uniform(v_lo0 + at.i * (Ly::TILE >> 4));
            ok = wait(&full[at.i], at.parity) && (v > 0 || wait(&o_free[half], o_parity)) && my_turn() &&
                 wait(&p_full[half], p_parity);
            tmem_fence_after();
            values(v_lo, next ? kPrefillKeys : tail, v > 0 ? 1u : 0u);
            if (next) ok = ok && wait(&full[kn.i], kn.parity);
            if (!agreed()) break;
            // (S goes where the weights stand that the product before reads: the tensor cores
            // take one thread's products in their order)
            if (next) scores(kn.i, v + 2 == steps ? id_tail : kIdS);
            pass_turn();
            if (issues) {
              umma_commit(&empty[at.i]);
              if (next) umma_commit(&empty[kn.i]);
              if (v + 2 == steps) umma_commit(q_empty);
            }
            p_parity ^= 1;
            at = kn;
            if (next) at.next();
          }
          o_parity ^= 1;
        }
        if (!ok && issues) fail();
        // nothing may be in flight when the columns are released
        if (issues) {
          umma_commit(end);
          if (!mbar_wait(end, 0)) fail();
        }
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ------------------------------------------------------------ softmax: a row a thread
    const int half = warp >> 2;
    const int r = half * 128 + (warp & 3) * 32 + lane;     // row of the item
    const uint32_t lane_tmem = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_tmem + 128 * half, o_at = lane_tmem + kTmemO + 128 * half;
    const float sc = p.scale_log2;
    uint32_t n = 0, steps = 0;                             // this half's steps; the CTA's
    bool ok = true;
    while (ok && walk.next(it)) {
      const PrefillTile& t = it.t;
      if (half == 1 && (t.tokens << p.group_log2) <= 128) {
        steps += t.steps > 0 ? it.v1 - it.v0 : 0;
        continue;
      }
      const int j = r >> p.group_log2;
      const int pos = t.pos0 + j;
      const int first_pos = t.pos0 + ((r & ~31) >> p.group_log2);
      const int last_pos = t.pos0 + min((r | 31) >> p.group_log2, t.tokens - 1);
      float m = kNoScore, l = 0.f;
      // (behind items that this half had no rows of; if nothing comes, the first step says so)
      if (n != steps && t.steps > 0) patient_wait(&s_full[half], n & 1, abort_flag);
      for (int v = it.v0; v < (t.steps > 0 ? it.v1 : it.v0); ++v, ++n, ++steps) {
        const int t0 = (v + (v >= t.ns ? t.shift : 0)) * kPrefillKeys;
        // does every row of this warp see every key of the step?
        const bool sees_all = t0 + kPrefillKeys <= first_pos + 1 &&
                              (t0 + p.window > last_pos || t0 + kPrefillKeys <= p.sinks);
        const bool got = wait(&s_full[half], n & 1);
        tmem_fence_after();
        float s[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s + 32 * i);
        const uint32_t bad = bad_ring[steps % kBadRing];
        tmem_landed(s);
        if (!sees_all || bad != 0) {
          const int last = pos - t0, first = pos - p.window + 1 - t0, sinks = p.sinks - t0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {                    // a bit for each of 32 keys
            const uint32_t gone = (((bad >> (2 * w)) & 1u) ? 0xffffu : 0u) | (((bad >> (2 * w + 1)) & 1u) ? 0xffff0000u : 0u);
            const uint32_t sees = below(last + 1 - 32 * w) & (~below(first - 32 * w) | below(sinks - 32 * w)) & ~gone;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((sees >> i) & 1u)) s[32 * w + i] = -INFINITY;
          }
        }
        // The reference is the first step's maximum.  Weights need not be below 1 (bf16 has the
        // range of float32), so it is only where a row's weights of a step come to more than
        // 2^16, and so a score has passed it by far, that the reference follows, O is rescaled,
        // and the weights are made again; no maximum is taken otherwise.
        float sum_l = 0.f;
        for (bool refer = v == it.v0;; refer = true) {
          if (refer) {
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i + 8 <= 128; i += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[i + e], s[i + 4 + e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[124 + e]);
            const float x = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * sc;
            float alpha = 1.f;
            if (v == it.v0) {
              m = fmaxf(x, kNoScore);
            } else {
              if (sum_l > kMostSum) {
                alpha = fast_exp2(m - x);
                m = x;
              }
              l *= alpha;
              // (O holds the steps so far: S came after their products)
#pragma unroll 1
              for (int i = 0; i < D / 16; ++i) {
                float o[16];
                tmem_ld16(o_at + 16 * i, o);
                tmem_landed(o);
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
                tmem_st16(o_at + 16 * i, w);
              }
            }
          }
          uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
          const uint64_t sc2 = pair(sc, sc), nm2 = pair(-m, -m);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a, b;
              unpair(fma2(pair(s[32 * i + 2 * e], s[32 * i + 2 * e + 1]), sc2, nm2), a, b);
              a = fast_exp2(a);
              b = fast_exp2(b);
              sum[e & 1] = add2(sum[e & 1], pair(a, b));
              w[e] = pack_bf16x2(a, b);
            }
            tmem_st16(s_at + 16 * i, w);
          }
          float l0, l1;
          unpair(add2(sum[0], sum[1]), l0, l1);
          sum_l = l0 + l1;
          // (the lanes agree on giving up here: one vote a step)
          if (!__any_sync(kFull, !got || (!refer && sum_l > kMostSum))) break;
          ok = __all_sync(kFull, got);
          if (!ok) break;
        }
        if (!ok) break;
        l += sum_l;
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[half]);
      }
      if (!ok) break;
      // ---- the rows, 128 bytes of each at a time: through shared memory, so that a store
      // has whole lines of 4 rows (a lane's own row in 16-byte pieces is 32 lines an
      // instruction: all stores together took a tenth of the kernel's time)
      unsigned char* stage = smem + Ly::OFF_STAGE + warp * (32 * 128);
      const int r0 = r & ~31, line = lane >> 3, chunk = lane & 7;
      auto put = [&](const uint32_t (&w)[32], unsigned char* to, int64_t token_bytes, int64_t head_bytes) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(stage + sw128(lane, c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = r0 + 4 * i + line, jj = rr >> p.group_log2;
          if (jj < t.tokens)
            *reinterpret_cast<uint4*>(to + jj * token_bytes + (rr & (p.group - 1)) * head_bytes + 16 * chunk) =
                *reinterpret_cast<const uint4*>(stage + sw128(4 * i + line, chunk));
        }
      };
      unsigned char* out = static_cast<unsigned char*>(p.out) +
          (static_cast<int64_t>(t.row0) * p.num_q_heads + it.h * p.group) * (2 * D);
      const int64_t out_token = static_cast<int64_t>(p.num_q_heads) * (2 * D);
      if (t.steps <= 0) {                                  // nothing to see
        const uint32_t zeros[32] = {};
        for (int i = 0; i < D / 64; ++i) put(zeros, out + 128 * i, out_token, 2 * D);
        continue;
      }
      ok = wait(&pv_done[half], (n - 1) & 1);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      tmem_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      if (it.slot < 0) {
#pragma unroll 1
        for (int i = 0; i < D / 64; ++i) {
          float o[64];
          tmem_ld32(o_at + 64 * i, o);
          tmem_ld32(o_at + 64 * i + 32, o + 32);
          tmem_landed(o);
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
          put(w, out + 128 * i, out_token, 2 * D);
        }
      } else {
        const int64_t row = static_cast<int64_t>(it.slot) * p.slot_rows;
        if (j < t.tokens) p.part_lse[row + r] = l > 0.f ? m + __log2f(l) : (l != l ? l : -INFINITY);
        unsigned char* part = reinterpret_cast<unsigned char*>(p.part_out + row * D);
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          tmem_ld32(o_at + 32 * i, o);
          tmem_landed(o);
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * inv);
          put(w, part + 128 * i, static_cast<int64_t>(p.group) * (4 * D), 4 * D);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[half]);
    }
    if (!ok) {
      tmem_wait_st();                                      // the weights of a step given up
      if (lane == 0) fail();
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <int D>
cudaError_t run(const PrefillParams& p, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(prefill_bf16_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PrefillLayout<D>::SMEM);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreadsPrefill);
  cfg.dynamicSmemBytes = PrefillLayout<D>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_bf16_kernel<D>, p);
}

}  // namespace

cudaError_t run_prefill_bf16(int head_dim, const PrefillParams& p, int grid, cudaStream_t stream) {
  return head_dim == 128 ? run<128>(p, grid, stream) : run<64>(p, grid, stream);
}

}  // namespace pa
