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
// MFLOP, 64 KiB of K and V and 32768 exponentials.
//
// Layout of the work:
//   * An item is a kv head and a tile of 256 rows: 256 / G consecutive new tokens of a
//     sequence with all G query heads of the head, so K and V are read once for the group.
//     Its rows are two products of 128 (M = 128).  While one half's scores are in softmax
//     the tensor cores work for the other: S0, S1 (128 columns each), O0 and O1 fill the
//     512 columns of tensor memory.
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
//   * The reference maximum moves only when a score passes it by more than 8 (weights then
//     stay below 2^8, and bf16 keeps its relative step), so O is hardly ever rescaled.
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
constexpr int kProducer = 8, kIssuer = 9, kCleaner = 10;   // (warp 11 only fills its warpgroup)
constexpr int kThreadsPrefill = 12 * 32;
constexpr int kBadRing = 8;
constexpr uint32_t kTmemO = 256;                           // column of O0; S0 is column 0

template <int D>
struct PrefillLayout {
  static constexpr int SLABS = D / 64;
  static constexpr int Q_SLAB = 128 * 128;                 // 128 rows of 64 columns
  static constexpr int Q_HALF = SLABS * Q_SLAB;
  static constexpr int TILE = kPrefillKeys * D * 2;
  static constexpr int RING = D == 128 ? 5 : 8;
  static constexpr int OFF_RING = 2 * Q_HALF;
  static constexpr int OFF_BAD = OFF_RING + RING * TILE;
  static constexpr int OFF_BARS = OFF_BAD + kBadRing * 4;
  // full, empty, raw [RING]; q_full, q_empty; s_full, p_full, pv_done, o_free [2]; end
  static constexpr int NUM_BARS = 3 * RING + 2 + 8 + 1;
  static constexpr int SMEM = OFF_BARS + NUM_BARS * 8 + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory over budget");
};

// The wait before tcgen05.ld's registers are used, tied to them.
template <int N>
__device__ __forceinline__ void tmem_landed(float (&v)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// The lowest n bits of a word, n of any size.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

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
  uint64_t* end = o_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(end + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_tokens = kPrefillRows >> p.group_log2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      mbar_init(&raw[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_free[i], 4);
    }
    mbar_init(end, 1);
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
  const int items = p.header[0] * p.num_kv_heads;
  auto fail = [&]() {
    if (!*abort_flag) {
      report(p.device_errors, PA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return !*abort_flag && mbar_wait(bar, parity, p.wait_limit);
  };
  // item k of this CTA: false past the last
  struct Item {
    int b, h;
    PrefillTile t;
  };
  auto take = [&](int k, Item& it) {
    const int i = prefill_item(k, blockIdx.x, gridDim.x);
    if (k * static_cast<int>(gridDim.x) >= items || i >= items) return false;
    const int2 e = p.list[i / p.num_kv_heads];
    it.b = e.x;
    it.h = i % p.num_kv_heads;
    it.t = prefill_tile<kPrefillKeys>(p, prefill_seq(p, e.x), e.y, tile_tokens);
    return true;
  };
  auto more = [&](int k) { return k * static_cast<int>(gridDim.x) < items; };
  // keys [x, y) of a step that starts at key t0 are behind the window and no sinks
  auto hidden = [&](const PrefillTile& t, int t0, int hi, int& x, int& y) {
    x = max(t0, p.sinks);
    y = min(t.lo, hi);
    return x < y;
  };

  if (warp == kProducer) {
    // ------------------------------------------------------------ copies
    const int bs = p.block_size, pages_of_step = kPrefillKeys >> p.block_log2;
    const int j = lane / Ly::SLABS, slab = lane % Ly::SLABS;   // of K: page of the step, slab
    uint32_t c = 0, steps = 0, raw_used = 0, raw_parity = 0;   // ring slots filled; raw: a bit a slot
    bool ok = true;
    int items_done = 0;
    Item it;
    for (int k = 0; ok && more(k); ++k) {
      if (!take(k, it) || it.t.steps <= 0) continue;
      if (lane == 0) {
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
        if (v >= it.t.steps || lane >= pages_of_step) return -2;
        const int first = (v + (v >= it.t.ns ? it.t.shift : 0)) * kPrefillKeys + lane * bs;
        if (first >= it.t.end || (first >= p.sinks && first + bs <= it.t.lo)) return -2;
        const int page = table[first >> p.block_log2];
        return page >= 0 && page < p.num_blocks ? page * p.num_kv_heads + it.h : -1;
      };
      int ahead = look(0);
      for (int v = 0; v < it.t.steps; ++v, ++steps) {
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
    Item it;
    for (int k = 0; ok && more(k); ++k) {
      if (!take(k, it)) continue;
      for (int v = 0; v < it.t.steps && ok; ++v, c += 2) {
        const int slot = (c + 1) % R;
        const int t0 = (v + (v >= it.t.ns ? it.t.shift : 0)) * kPrefillKeys, hi = min(it.t.end, t0 + kPrefillKeys);
        int x, y;
        const bool behind = hidden(it.t, t0, hi, x, y);
        if ((hi & 15) == 0 && !behind) continue;
        ok = wait(&raw[slot], (raw_parity >> slot) & 1);
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
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ products: one thread
    if (lane == 0) {
      const uint32_t ring = smem_addr(smem + Ly::OFF_RING), q_base = smem_addr(smem);
      const int bs = p.block_size;
      constexpr uint32_t kIdPV = umma_idesc_bf16(128, D, true);
      uint32_t c = 0, kp[2] = {0, 0}, ko[2] = {0, 0};      // ring slots taken; weights, items of each half
      bool ok = true;
      int items_done = 0;
      Item it;
      // S of half i = its rows of q times the K tile in `slot`
      auto scores = [&](int i, int slot, int keys) {
        const uint64_t qd = umma_desc(q_base + i * Ly::Q_HALF, 16, 1024);
        const uint64_t kd = umma_desc(ring + slot * Ly::TILE, 16, 1024);
        const uint32_t id = umma_idesc_bf16(128, (keys + 15) & ~15, false);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t off = ((ks >> 2) * Ly::Q_SLAB + (ks & 3) * 32) >> 4;
          umma_bf16(tmem + 128 * i, qd + off, kd + off, id, ks > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[i]);
      };
      for (int k = 0; ok && more(k); ++k) {
        if (!take(k, it) || it.t.steps <= 0) continue;
        const int halves = (it.t.tokens << p.group_log2) > 128 ? 2 : 1;
        auto keys_of = [&](int v) {
          return min(kPrefillKeys, it.t.end - (v + (v >= it.t.ns ? it.t.shift : 0)) * kPrefillKeys);
        };
        ok = wait(q_full, items_done & 1) && wait(&full[c % R], (c / R) & 1);
        if (!ok) break;
        ++items_done;
        tmem_fence_after();
        for (int i = 0; i < halves; ++i) scores(i, c % R, keys_of(0));
        umma_commit(&empty[c % R]);
        if (it.t.steps == 1) umma_commit(q_empty);
        ++c;
        for (int v = 0; v < it.t.steps && ok; ++v) {
          const uint32_t cv = c, ck = c + 1;               // V of this step, K of the next
          const bool next = v + 1 < it.t.steps;
          const int keys = keys_of(v);
          for (int i = 0; i < halves && ok; ++i) {
            if (i == 0) ok = wait(&full[cv % R], (cv / R) & 1);
            ok = ok && wait(&p_full[i], kp[i] & 1);
            if (v == 0) ok = ok && wait(&o_free[i], (ko[i] & 1) ^ 1);
            if (!ok) break;
            ++kp[i];
            tmem_fence_after();
            const uint32_t vt = ring + (cv % R) * Ly::TILE;
            for (int g = 0; 16 * g < keys; ++g) {
              const int page = (16 * g) >> p.block_log2, r = (16 * g) & (bs - 1);
              const uint64_t vd = umma_desc(vt + page * bs * D * 2 + r * 128, bs * 128, 1024);
              umma_bf16_ts(tmem + kTmemO + 128 * i, tmem + 128 * i + 8 * g, vd, kIdPV, v > 0 || g > 0 ? 1u : 0u);
            }
            umma_commit(&pv_done[i]);
            if (next) {
              if (i == 0) {
                ok = wait(&full[ck % R], (ck / R) & 1);
                if (!ok) break;
                tmem_fence_after();
              }
              // (after the product that reads the weights that stand where S goes: the
              // tensor cores take one thread's products in their order)
              scores(i, ck % R, keys_of(v + 1));
            }
          }
          if (!ok) break;
          umma_commit(&empty[cv % R]);
          if (next) umma_commit(&empty[ck % R]);
          if (v + 2 == it.t.steps) umma_commit(q_empty);
          c += next ? 2 : 1;
        }
        ++ko[0];
        if (halves == 2) ++ko[1];
      }
      if (!ok) fail();
      // nothing may be in flight when the columns are released
      umma_commit(end);
      mbar_wait(end, 0);
    }
    __syncwarp();
  } else if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax: a row a thread
    const int half = warp >> 2;
    const int r = half * 128 + (warp & 3) * 32 + lane;     // row of the item
    const uint32_t lane_tmem = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_tmem + 128 * half, o_at = lane_tmem + kTmemO + 128 * half;
    const float sc = p.scale_log2;
    uint32_t n = 0, steps = 0;                             // this half's steps; the CTA's
    bool ok = true;
    Item it;
    for (int k = 0; ok && more(k); ++k) {
      if (!take(k, it)) continue;
      const PrefillTile& t = it.t;
      if (half == 1 && (t.tokens << p.group_log2) <= 128) {
        steps += t.steps;
        continue;
      }
      const int j = r >> p.group_log2;
      const int pos = t.pos0 + j;
      const int first_pos = t.pos0 + ((r & ~31) >> p.group_log2);
      const int last_pos = t.pos0 + min((r | 31) >> p.group_log2, t.tokens - 1);
      float m = kNoScore, l = 0.f;
      for (int v = 0; v < t.steps; ++v, ++n, ++steps) {
        const int t0 = (v + (v >= t.ns ? t.shift : 0)) * kPrefillKeys;
        ok = wait(&s_full[half], n & 1);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tmem_fence_after();
        float s[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s + 32 * i);
        tmem_landed(s);
        const uint32_t bad = bad_ring[steps % kBadRing];
        // does every row of this warp see every key of the step?
        const bool all = bad == 0 && t0 + kPrefillKeys <= first_pos + 1 &&
                         (t0 + p.window > last_pos || t0 + kPrefillKeys <= p.sinks);
        if (!all) {
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
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
        const float x = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        const bool grow = x > m + 8.f;
        float alpha = 1.f;
        if (grow) {
          alpha = fast_exp2(m - x);
          m = x;
        }
        l *= alpha;
        if (v > 0 && __any_sync(kFull, grow)) {
          ok = wait(&pv_done[half], (n - 1) & 1);          // O holds the steps so far
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          tmem_fence_after();
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
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        const float nm = -m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float a = fast_exp2(fmaf(s[32 * i + 2 * e], sc, nm)), b = fast_exp2(fmaf(s[32 * i + 2 * e + 1], sc, nm));
            sum[(2 * e) & 3] += a;
            sum[(2 * e + 1) & 3] += b;
            w[e] = pack_bf16x2(a, b);
          }
          tmem_st16(s_at + 16 * i, w);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[half]);
      }
      if (!ok) break;
      // ---- the rows
      const bool valid = j < t.tokens;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
          ((static_cast<int64_t>(t.row0) + j) * p.num_q_heads + it.h * p.group + (r & (p.group - 1))) * D);
      if (t.steps <= 0) {                                  // nothing to see
        if (valid)
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      ok = wait(&pv_done[half], (n - 1) & 1);
      ok = __all_sync(kFull, ok);
      if (!ok) break;
      tmem_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float o[32];
        tmem_ld32(o_at + 32 * i, o);
        tmem_landed(o);
        if (valid)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[4 * i + e] = make_uint4(pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv),
                                        pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                        pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                        pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[half]);
    }
    if (!ok && lane == 0) fail();
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
