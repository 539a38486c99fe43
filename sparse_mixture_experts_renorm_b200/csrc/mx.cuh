// mx.cuh — MXFP4 (OCP microscaling, E2M1 elements in blocks of 32 with one
// E8M0 scale): the layout of the scales and the rounding of one block.
#pragma once

#include <cuda_fp16.h>

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

__host__ __device__ __forceinline__ int mx_stages(int cols) {
  return (int)(((unsigned)cols + kMxStageCols - 1) / kMxStageCols);
}

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

// 32 bytes to or from memory that is used once, a whole sector at once where
// the address allows (rows are multiples of 32 bytes, so `wide` is a question
// of the first one's).
__device__ __forceinline__ void load_sector(uint32_t (&w)[8], const void* p, bool wide) {
  if (wide) {
    asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldcs(static_cast<const uint4*>(p)), b = __ldcs(static_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store_sector(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(static_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

// A piece in registers: 16 bf16 or 8 fp32, and its codes.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int kCols = 16;
  using Codes = uint2;
  uint32_t w[8];
  // The largest magnitude's bits as those of a float.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
  // Times a power of two: exact where it is not so small that its code is 0.
  __device__ __forceinline__ Codes codes(float inv) const {
    const __nv_bfloat162 s = __float2bfloat162_rn(inv);
    float q[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), s);
      const uint32_t b = *reinterpret_cast<const uint32_t*>(&t);
      q[2 * i] = __uint_as_float(b << 16);
      q[2 * i + 1] = __uint_as_float(b & 0xffff0000u);
    }
    return make_uint2(mx_pack8(q), mx_pack8(q + 8));
  }
  __device__ __forceinline__ void values(const Codes& c, float scale) {
    const __nv_bfloat162 s = __float2bfloat162_rn(scale);
    uint32_t a[4], b[4];
    mx_values8(c.x, a);
    mx_values8(c.y, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(i < 4 ? &a[i] : &b[i - 4]), s);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
  }
};
template <>
struct Piece<float> {
  static constexpr int kCols = 8;
  using Codes = uint32_t;
  uint32_t w[8];
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ Codes codes(float inv) const {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __uint_as_float(w[i]) * inv;
    return mx_pack8(q);
  }
  __device__ __forceinline__ void values(const Codes& c, float s) {
    uint32_t a[4];
    mx_values8(c, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[2 * i] = __float_as_uint(__uint_as_float(a[i] << 16) * s);
      w[2 * i + 1] = __float_as_uint(__uint_as_float(a[i] & 0xffff0000u) * s);
    }
  }
};

// Rows of expert outputs between the down product and the sum over a token's
// experts: fp16 with one exponent byte per 32 columns, by which the largest of
// them lies in [1, 2), or in [2, 4) from 2^127 on (254 would need 2^-127, which
// is no normal number; fp16 holds 4 as well as 2). That leaves 2^-11 of a value
// where bf16 would leave 2^-8, half the error of the whole layer, for the same
// bytes. Exponent byte 0xFF: the block holds a NaN or an infinity, and its
// columns are bf16.
// Exponent bytes stand by 256 columns and rows, eight for each.
__host__ __device__ __forceinline__ size_t y16_exp_at(size_t rows, int col, size_t row) {
  return ((size_t)(col >> 8) * rows + row) * 8 + ((col >> 5) & 7);
}
__device__ __forceinline__ uint32_t y16_exp(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 0xffu ? e : min(max(e, 1u), 253u);
}
// For exponents 1 .. 253: 2^(127 - e) and 2^(e - 127).
__device__ __forceinline__ float y16_inv(uint32_t e) { return __uint_as_float((254u - e) << 23); }
__device__ __forceinline__ float y16_step(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ uint32_t y16_pack(float a, float b, float inv) {
  const __half2 h = __floats2half2_rn(a * inv, b * inv);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The two numbers of a word (times y16_step they are the values).
__device__ __forceinline__ float2 y16_numbers(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

}  // namespace moe
