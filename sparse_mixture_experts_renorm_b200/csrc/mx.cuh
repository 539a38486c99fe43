// mx.cuh — MXFP4 (OCP microscaling, E2M1 elements in blocks of 32 with one
// E8M0 scale): the layout of the scales and the rounding of one block.
#pragma once

#include "common.cuh"

namespace moe {

// Scales are stored in tiles of 128 rows x 128 columns, four scales a row in
// 512 bytes, the order in which tcgen05.cp (32x128b.warpx4) brings them to
// TMEM: row r, 32-column block b of the tile at byte (r % 32) * 16 + (r / 32)
// * 4 + b. The two tiles of 256 columns stand side by side (one pipeline stage
// of the product), so 128 rows x 256 columns take 1024 bytes, and the tiles of
// one row of tiles follow one another over the columns. Every group of rows
// (an expert) starts at a new pair of tile rows: 256 rows, one tile of the
// product's CTA pair.
constexpr int kMxBlock = 32;
constexpr int kMxTileRows = 128;
constexpr int kMxStageCols = 256;
constexpr int kMxStageBytes = 1024;  // scales of 128 rows x 256 columns

__host__ __device__ __forceinline__ int mx_stages(int cols) { return (cols + kMxStageCols - 1) / kMxStageCols; }

// Byte of the scale of (tile row, row r < 128 of it, block b of the row).
__host__ __device__ __forceinline__ size_t mx_scale_at(size_t tile_row, int stages, int r, int b) {
  return (tile_row * stages + (b >> 3)) * kMxStageBytes + ((b >> 2) & 1) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
}

// The scale byte of a block from the largest magnitude's bits (as an integer,
// so that NaN > infinity > every finite value): floor(log2 amax) - 2 with bias
// 127, at least 0 (2^-127); 0xFF (NaN) when the block holds a NaN or an
// infinity, which a dequantised block then shows as NaN throughout.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return amax_bits >= 0x7f800000u ? 0xFFu : (uint32_t)max(e - 2, 0);
}

// 2^-(byte - 127), exact and normal for every byte below 0xFF that
// mx_scale_byte gives (0 .. 252); 0 for 0xFF: there the scale alone says that
// the block is NaN, whatever its codes.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return byte == 0xFFu ? 0.f : __uint_as_float((254u - byte) << 23);
}

// The value 2^(byte - 127) (2^-127 is subnormal; 0xFF is NaN).
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return byte == 0xFFu ? __uint_as_float(0x7fffffffu) : byte == 0u ? __uint_as_float(0x00400000u)
                                                                   : __uint_as_float(byte << 23);
}

// Eight values to E2M1 (round to nearest even, saturating at 6), element i in
// bits [4i, 4i + 4).
__device__ __forceinline__ uint32_t mx_pack8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight E2M1 codes as bf16, element i in half i % 2 of w[i / 2].
// Byte permutes look the two bytes of 0, 0.5, 1, 1.5, 2, 3, 4, 6 up, four
// codes at once.
__device__ __forceinline__ void mx_values8(uint32_t code, uint32_t (&w)[4]) {
  const uint32_t even = (code << 4) & 0x80808080u, odd = code & 0x80808080u;  // signs
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t sel = (code >> (16 * i)) & 0x7777u;
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel) | __byte_perm(even, odd, i ? 0x7362 : 0x5140);
    w[2 * i] = __byte_perm(lo, hi, 0x5140);
    w[2 * i + 1] = __byte_perm(lo, hi, 0x7362);
  }
}

}  // namespace moe
