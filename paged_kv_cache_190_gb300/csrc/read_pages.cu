// Pages of 4-bit rows read back as bf16: dst[d] = values of src[s] for each pair (s, d).
//
// value = code * scale, exact in bf16 (2 and 4 significant bits).  Bound by memory: 72
// bytes of a row are read and 256 written.  A thread takes the 16 columns of a scale: 8
// bytes of codes, a byte, one 32-byte store; eight threads a row, so that a warp writes whole
// lines (with two 16-byte stores, each in half of every sector, 8 contexts of 1000 to 16384
// tokens, 419 MB, took 84.2 us; so 66.4, 6.3 TB/s, 93 % of the measured copy rate; the pages
// of 256 tokens 6.4 and 3.7; 33 pages 1.9).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp4.cuh"
#include "pa_rope.h"

namespace pa {
namespace {

constexpr int kReadThreads = 128;
constexpr int kReadRows = 2;                               // rows of K and of V that a thread has in flight
constexpr int kBlockRows = kReadThreads / 8 * kReadRows;
static_assert(kBlockRows == kReadPartRows, "what the host's bound counts");

__device__ __forceinline__ uint32_t bf16x2_of(uint32_t halves) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&halves));
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void write16(uint4* dst /* 32-byte aligned */, uint2 codes, uint32_t scale) {
  const uint32_t s = (scale << 7) | (scale << 23);
  uint32_t w[8];
  halves4_of(codes.x, w[0], w[1], w[2], w[3]);
  halves4_of(codes.y, w[4], w[5], w[6], w[7]);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = bf16x2_of(mul_half2(w[i], s));
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Block (pair, part): kBlockRows of the page's rows, of K and of V.
__global__ void __launch_bounds__(kReadThreads) read_pages_fp4_kernel(
    uint4* k_out, uint4* v_out, const unsigned char* k_cache, const unsigned char* v_cache,
    const int64_t* pairs, int page_rows, int num_src, int num_dst, int32_t* device_errors) {
  wait_prior_grids();
  allow_next_grid();
  const int64_t src = pairs[2 * static_cast<int64_t>(blockIdx.x)], dst = pairs[2 * static_cast<int64_t>(blockIdx.x) + 1];
  if (src < 0 || src >= num_src || dst < 0 || dst >= num_dst) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(device_errors, PA_DEVERR_BAD_BLOCK);
    return;
  }
  const int part = threadIdx.x & 7, r0 = blockIdx.y * kBlockRows + (threadIdx.x >> 3);
  uint2 codes[2][kReadRows];
  uint32_t scale[2][kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int r = r0 + i * (kReadThreads / 8);
    if (r >= page_rows) continue;
    const int64_t at = (src * page_rows + r) * kRow4Bytes;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const unsigned char* row = (kv ? v_cache : k_cache) + at;
      codes[kv][i] = *reinterpret_cast<const uint2*>(row + 8 * part);
      scale[kv][i] = row[kRow4Codes + part];
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int r = r0 + i * (kReadThreads / 8);
    if (r >= page_rows) continue;
    const int64_t at = (dst * page_rows + r) * 16 + 2 * part;
    write16(k_out + at, codes[0][i], scale[0][i]);
    write16(v_out + at, codes[1][i], scale[1][i]);
  }
}

}  // namespace

cudaError_t launch_read_pages_fp4(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                                  const int64_t* pairs, int num_pairs, int page_rows, int num_src,
                                  int num_dst, int32_t* device_errors, cudaStream_t stream) {
  if (num_pairs == 0) return cudaSuccess;
  const int parts = (page_rows + kBlockRows - 1) / kBlockRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_pairs), static_cast<unsigned>(parts));
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, read_pages_fp4_kernel, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out),
                            static_cast<const unsigned char*>(k_cache), static_cast<const unsigned char*>(v_cache),
                            pairs, page_rows, num_src, num_dst, device_errors);
}

}  // namespace pa
