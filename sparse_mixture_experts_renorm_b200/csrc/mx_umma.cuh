// mx_umma.cuh — what the kernels of the MXFP4 products share: block-scaled
// tcgen05 instructions (kind::mxf4) and the walk over a grouped product's
// tiles.
#pragma once

#include <atomic>

#include "mx.cuh"
#include "mx_internal.h"
#include "pair.cuh"

namespace moe {
namespace {

// Instruction descriptor for kind::mxf4 (E2M1 x E2M1, E8M0 scales, fp32
// accumulator, both operands K-major): B scale id in bits [4,6), A format 1 =
// E2M1 in [7,10), B format 1 in [10,12), N >> 3 in [17,23), scale format 1 =
// E8M0 in bit 23, M >> 7 in [27,29), A scale id in [29,31).
__device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 7) << 27) | (sf_id << 29);
}

// D[tmem] (+)= A * B^T, 64 columns of K, one scale per 32 of them.
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 512 bytes of scales (128 rows x 4) from both CTAs' shared memory to four
// columns of their own TMEM, repeated in every lane quarter.
__device__ __forceinline__ void tc_cp_scales_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Matrix descriptor of a 32 x 16-byte tile without swizzle: 8-row core
// matrices of 128 bytes one after the other.
__device__ __forceinline__ uint64_t scales_desc(uint32_t smem_addr) {
  uint64_t desc = 0;
  desc |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  desc |= static_cast<uint64_t>(16u >> 4) << 16;
  desc |= static_cast<uint64_t>(128u >> 4) << 32;
  desc |= static_cast<uint64_t>(1u) << 46;
  return desc;
}

// The larger of a and |b|; NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}

// A tile of the grouped product. The rows of A's tiles are the caller's: s_mt
// holds the tiles before each group, s_off its first row; the tiles of one
// weight block follow each other.
struct MxTile {
  int g, m, n, row0, cnt;  // group, its tile of rows, weight block, first row and rows of the group
};

__device__ __forceinline__ MxTile mx_tile(int tile, int n_wb, const int* s_off, const int* s_mt, int G) {
  const int q = tile / n_wb;
  int lo = 0, hi = G;  // s_mt[lo] <= q < s_mt[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_mt[mid] <= q)
      lo = mid;
    else
      hi = mid;
  }
  MxTile t;
  t.g = lo;
  const int mt = s_mt[lo + 1] - s_mt[lo];
  const int local = tile - s_mt[lo] * n_wb;
  t.n = local / mt;
  t.m = local - t.n * mt;
  t.row0 = s_off[lo];
  t.cnt = s_off[lo + 1] - s_off[lo];
  return t;
}

// Resident CTA pairs per GPU, queried once per device and kernel (which is
// given its shared memory then).
inline int max_pairs(const void* kern, int threads, int smem, std::atomic<int>* cache) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int have = cache[dev].load(std::memory_order_acquire);
  if (have > 0) return have;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return 0;
  cache[dev].store(n, std::memory_order_release);
  return n;
}

}  // namespace
}  // namespace moe
