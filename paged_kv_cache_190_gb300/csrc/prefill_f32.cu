// Prompt attention over paged float32 pools, on the CUDA cores: every product and sum in
// float32 (the tensor cores would round the factors).
//
// Mathematics as in prefill_bf16.cu, 64 or 32 rows of a kv head (so many / G new tokens with
// the group's G heads) and 64 keys a step, with the running maximum itself as reference.
//
// What bounds it: multiply-adds, 2 * 64 * 64 * D a step, and the shared-memory reads that
// feed them.  A thread holds 4 (2) rows by 4 keys of the scores and 4 (2) rows by D / 16
// columns of the result, so each 16 bytes read serve 8 to 16 multiply-adds; rows of shared
// memory are 16 bytes longer than D floats, so that 8 keys' 16 bytes fall on all banks.  The
// next step's keys are copied while this one's are worked on.  Tiles of 32 rows where 64 would
// leave SMs without one: a call then ends with its longest sequence (5 prompts of 17 to 200
// tokens behind up to 100, 8 heads of 64: 23.0 us; tiles of 64 rows 31.9, and 32.8 with
// their keys copied when they are needed).
#include <cuda_runtime.h>

#include <atomic>

#include "pa_device.cuh"
#include "prefill.h"

namespace pa {
namespace {

constexpr int kThreadsF32 = 256;
constexpr int kKeysF32 = kPrefillKeysF32;
constexpr float kNoScoreF32 = -3.0e38f;

template <int D, int ROWS>
struct F32Layout {
  static constexpr int ROW = D + 4;                        // floats
  static constexpr int TILE = kKeysF32 * ROW;
  static constexpr int K = ROWS * ROW, V = K + 2 * TILE, P = V + 2 * TILE;
  static constexpr int PROW = kKeysF32 + 4;
  static constexpr int BYTES = (P + ROWS * PROW) * 4;
};

__device__ __forceinline__ void copy16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreadsF32, D == 128 ? 1 : 2) prefill_f32_kernel(const __grid_constant__ PrefillParams p) {
  using Ly = F32Layout<D, ROWS>;
  constexpr int NC = D / 64;                               // 4-column chunks of a thread
  constexpr int RT = ROWS / 16;                            // rows of a thread
  extern __shared__ __align__(16) float smem_f[];
  float* qs = smem_f;
  float* ps = smem_f + Ly::P;
  __shared__ int seen[2][kKeysF32];                        // of a step: may any row see the key?
  wait_prior_grids();
  allow_next_grid();
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int tile_tokens = ROWS >> p.group_log2;
  const float* q = static_cast<const float*>(p.q);
  PrefillWalk<kKeysF32> walk(p, tile_tokens);
  PrefillItem it;
  while (walk.next(it)) {
    const int h = it.h;
    const PrefillTile& t = it.t;
    const int32_t* table = p.tables + static_cast<int64_t>(it.b) * p.max_blocks;
    auto row_of = [&](int r) {                             // of q and out
      return ((static_cast<int64_t>(t.row0) + (r >> p.group_log2)) * p.num_q_heads + h * p.group + (r & (p.group - 1))) * D;
    };
    auto first_key = [&](int v) { return (v + (v >= t.ns ? t.shift : 0)) * kKeysF32; };
    // a step's keys on their way into buffer v & 1; those that no row sees may hold anything:
    // their rows are zeros
    auto fetch = [&](int v) {
      if (v < t.steps) {
        const int t0 = first_key(v);
        float* ks = smem_f + Ly::K + (v & 1) * Ly::TILE;
        float* vs = smem_f + Ly::V + (v & 1) * Ly::TILE;
        for (int i = threadIdx.x; i < kKeysF32 * (D / 4); i += kThreadsF32) {
          const int r = i / (D / 4), c = 4 * (i % (D / 4)), key = t0 + r;
          int z = -1;
          if (key < t.end && (key < p.sinks || key >= t.lo)) {
            z = table[key >> p.block_log2];
            if (z < 0 || z >= p.num_blocks) {
              if (c == 0) report(p.device_errors, PA_DEVERR_BAD_BLOCK);
              z = -1;
            }
          }
          if (c == 0) seen[v & 1][r] = z >= 0;
          if (z >= 0) {
            const int64_t at = ((static_cast<int64_t>(z) * p.num_kv_heads + h) * p.block_size + (key & (p.block_size - 1))) * D + c;
            copy16(ks + r * Ly::ROW + c, static_cast<const float*>(p.k_cache) + at);
            copy16(vs + r * Ly::ROW + c, static_cast<const float*>(p.v_cache) + at);
          } else {
            *reinterpret_cast<float4*>(ks + r * Ly::ROW + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(vs + r * Ly::ROW + c) = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();                                       // the last item's rows and keys have been read
    fetch(0);
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += kThreadsF32) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if ((r >> p.group_log2) < t.tokens) w = *reinterpret_cast<const float4*>(q + row_of(r) + c);
      *reinterpret_cast<float4*>(qs + r * Ly::ROW + c) =
          make_float4(w.x * p.scale_log2, w.y * p.scale_log2, w.z * p.scale_log2, w.w * p.scale_log2);
    }
    float m[RT], l[RT], acc[RT][4 * NC];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      m[i] = kNoScoreF32;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) acc[i][c] = 0.f;
    }
    for (int v = 0; v < t.steps; ++v) {
      const int t0 = first_key(v);
      const float* ks = smem_f + Ly::K + (v & 1) * Ly::TILE;
      const float* vs = smem_f + Ly::V + (v & 1) * Ly::TILE;
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();                                     // this step's keys are there, the last one's read
      fetch(v + 1);
      // ---- scores of rows RT ty + i and keys tx + 16 c
      float s[RT][4] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[RT], b[4];
#pragma unroll
        for (int i = 0; i < RT; ++i) a[i] = *reinterpret_cast<const float4*>(qs + (RT * ty + i) * Ly::ROW + d);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4*>(ks + (tx + 16 * c) * Ly::ROW + d);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s[i][c] = fmaf(a[i].w, b[c].w, fmaf(a[i].z, b[c].z, fmaf(a[i].y, b[c].y, fmaf(a[i].x, b[c].x, s[i][c]))));
      }
      bool there[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) there[c] = seen[v & 1][tx + 16 * c] != 0;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int pos = t.pos0 + ((RT * ty + i) >> p.group_log2);
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int key = t0 + tx + 16 * c;
          if (!(there[c] && key <= pos && (pos - key < p.window || key < p.sinks))) s[i][c] = -INFINITY;
          mx = fmaxf(mx, s[i][c]);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx), alpha = fast_exp2(m[i] - mn);
        m[i] = mn;
        l[i] *= alpha;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float w = fast_exp2(s[i][c] - mn);
          l[i] += w;
          ps[(RT * ty + i) * Ly::PROW + tx + 16 * c] = w;
        }
#pragma unroll
        for (int c = 0; c < 4 * NC; ++c) acc[i][c] *= alpha;
      }
      __syncwarp();                                        // (a warp reads the rows that it wrote)
      // ---- values: columns 4 tx + 64 c
#pragma unroll 2
      for (int t4 = 0; t4 < kKeysF32; t4 += 4) {
        float4 w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = *reinterpret_cast<const float4*>(ps + (RT * ty + i) * Ly::PROW + t4);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(vs + (t4 + n) * Ly::ROW + 4 * tx + 64 * c);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const float f = n == 0 ? w[i].x : n == 1 ? w[i].y : n == 2 ? w[i].z : w[i].w;
              acc[i][4 * c] = fmaf(f, x.x, acc[i][4 * c]);
              acc[i][4 * c + 1] = fmaf(f, x.y, acc[i][4 * c + 1]);
              acc[i][4 * c + 2] = fmaf(f, x.z, acc[i][4 * c + 2]);
              acc[i][4 * c + 3] = fmaf(f, x.w, acc[i][4 * c + 3]);
            }
          }
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float sum = l[i];
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      const int r = RT * ty + i;
      if ((r >> p.group_log2) < t.tokens) {
        float* dst = static_cast<float*>(p.out) + row_of(r);
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float4*>(dst + 4 * tx + 64 * c) =
              make_float4(acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv, acc[i][4 * c + 2] * inv, acc[i][4 * c + 3] * inv);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int ROWS>
cudaError_t run(const PrefillParams& p, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (!(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(prefill_f32_kernel<D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, F32Layout<D, ROWS>::BYTES);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreadsF32);
  cfg.dynamicSmemBytes = F32Layout<D, ROWS>::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_f32_kernel<D, ROWS>, p);
}

}  // namespace

cudaError_t run_prefill_f32(int head_dim, int rows, const PrefillParams& p, int grid, cudaStream_t stream) {
  if (head_dim == 128) return rows == 64 ? run<128, 64>(p, grid, stream) : run<128, 32>(p, grid, stream);
  return rows == 64 ? run<64, 64>(p, grid, stream) : run<64, 32>(p, grid, stream);
}

}  // namespace pa
