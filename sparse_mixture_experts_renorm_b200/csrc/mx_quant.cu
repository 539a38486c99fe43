// mx_quant.cu — rows to MXFP4 and back.
//
//   s = max(floor(log2(max |x_i|)) - 2, -127) over a block of 32 columns,
//   code_i = E2M1(x_i / 2^s), round to nearest even, at most 6;   x~_i = code_i 2^s
//
// Both directions only move memory: a row of C columns is C * (2 or 4) bytes
// on one side and C / 2 + C / 32 on the other. A warp takes 256 columns of a
// row at a time, eight consecutive columns a lane (16 or 32 bytes of x, 4 of
// codes), so every access of a warp is one contiguous run; four lanes share a
// block and agree on its scale with two shuffles. Four such pieces are in
// flight per warp.
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQUnits = 4;  // 256-column pieces per warp in flight

// Where the groups of rows lie: group g's rows are [off[g], off[g+1]) and its
// scales start at tile row tile[g].
struct Groups {
  int off[kMaxExperts + 1];
  int tile[kMaxExperts + 1];
};

// Fills s from offsets (G <= kMaxExperts, one thread per group); the block has
// kQThreads threads.
__device__ __forceinline__ void load_groups(Groups& s, const int32_t* __restrict__ offsets, int G) {
  static_assert(kQThreads >= kMaxExperts, "one thread per group");
  __shared__ int s_w[kQThreads / 32];
  const int g = threadIdx.x, lane = g & 31, w = g >> 5;
  const int a = g <= G ? offsets[g] : 0;
  const int b = g < G ? offsets[g + 1] : a;
  const int tiles = b > a ? ((b - a + 255) >> 8) * 2 : 0;
  int incl = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) s_w[w] = incl;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < w; ++i) before += s_w[i];
  if (g < G) {
    s.off[g] = a;
    s.tile[g] = before + incl - tiles;
  }
  if (g == 0) s.off[G] = offsets[G];
  __syncthreads();
}

// The tile row and the row inside it of `row`; false for a row of no group.
__device__ __forceinline__ bool place_row(const Groups& s, int G, int row, size_t* tile_row, int* r) {
  if (row < s.off[0] || row >= s.off[G]) return false;
  int lo = 0, hi = G;  // off[lo] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.off[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  const int in = row - s.off[lo];
  *tile_row = (size_t)(s.tile[lo] + (in >> 7));
  *r = in & 127;
  return true;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// The tile row and row in it of a row of [G, rows] with every group padded.
__device__ __forceinline__ void place_dense(long long row, int rows, int group_tiles, size_t* tile_row, int* r) {
  const long long g = row / rows;
  const int in = (int)(row - g * rows);
  *tile_row = (size_t)g * group_tiles + (size_t)(in >> 7);
  *r = in & 127;
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) mx_quantize_kernel(const T* __restrict__ x, long long n_rows, int rows,
                                                                int cols, const int32_t* __restrict__ offsets, int G,
                                                                int group_tiles, size_t tile_rows,
                                                                uint8_t* __restrict__ data,
                                                                uint8_t* __restrict__ scales) {
  __shared__ Groups s_g;
  pdl_wait();
  if (offsets) load_groups(s_g, offsets, G);
  const int lane = threadIdx.x & 31;
  const int st = mx_stages(cols);
  const long long units = n_rows * st;
  const long long u0 = ((long long)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5)) * kQUnits;
  float v[kQUnits][8];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const long long u = u0 + i, row = u / st;
    const int c = (int)(u - row * st) * kMxStageCols + lane * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (u < units && c < cols) load8(x + row * cols + c, v[i]);
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const long long u = u0 + i;
    if (u >= units) break;
    const long long row = u / st;
    const int kb = (int)(u - row * st);
    const int c = kb * kMxStageCols + lane * 8;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t sb = mx_scale_byte(m);
    const float inv = mx_inv_scale(sb);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = v[i][j] * inv;
    // four blocks' bytes in one word, gathered over 16 lanes
    uint32_t word = sb << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    size_t tile_row = 0;
    int r = 0;
    bool live = true;
    if (offsets)
      live = place_row(s_g, G, (int)row, &tile_row, &r);
    else
      place_dense(row, rows, group_tiles, &tile_row, &r);
    if (!live || tile_row >= tile_rows) continue;
    if (c < cols) *reinterpret_cast<uint32_t*>(data + row * (cols / 2) + c / 2) = mx_pack8(q);
    if ((lane & 15) == 0)
      *reinterpret_cast<uint32_t*>(scales + mx_scale_at(tile_row, st, r, kb * 8 + (lane >> 2))) = word;
  }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) mx_dequantize_kernel(const uint8_t* __restrict__ data,
                                                                  const uint8_t* __restrict__ scales, long long n_rows,
                                                                  int rows, int cols,
                                                                  const int32_t* __restrict__ offsets, int G,
                                                                  int group_tiles, size_t tile_rows,
                                                                  T* __restrict__ out) {
  __shared__ Groups s_g;
  pdl_wait();
  if (offsets) load_groups(s_g, offsets, G);
  const int lane = threadIdx.x & 31;
  const int st = mx_stages(cols);
  const long long units = n_rows * st;
  const long long u0 = ((long long)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5)) * kQUnits;
  uint32_t code[kQUnits], sb[kQUnits];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const long long u = u0 + i, row = u / st;
    const int kb = (int)(u - row * st);
    const int c = kb * kMxStageCols + lane * 8;
    code[i] = sb[i] = 0;
    if (u < units && c < cols) {
      size_t tile_row = 0;
      int r = 0;
      bool live = true;
      if (offsets)
        live = place_row(s_g, G, (int)row, &tile_row, &r);
      else
        place_dense(row, rows, group_tiles, &tile_row, &r);
      if (live && tile_row < tile_rows) {
        code[i] = __ldcs(reinterpret_cast<const uint32_t*>(data + row * (cols / 2) + c / 2));
        sb[i] = 0x100u | __ldg(scales + mx_scale_at(tile_row, st, r, kb * 8 + (lane >> 2)));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const long long u = u0 + i, row = u / st;
    const int c = (int)(u - row * st) * kMxStageCols + lane * 8;
    if (!(sb[i] & 0x100u)) continue;
    const float s = mx_scale_value(sb[i] & 0xffu);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = mx_value(code[i] >> (4 * j)) * s;
    store8(out + row * cols + c, v);
  }
}

}  // namespace

cudaError_t launch_mx_quantize(moe_dtype dtype, const void* x, long long n_rows, int rows, int cols,
                               const int32_t* offsets, int G, int group_tiles, size_t tile_rows, void* data,
                               void* scales, cudaStream_t stream) {
  const long long units = n_rows * mx_stages(cols);
  const int per = (kQThreads / 32) * kQUnits;
  const dim3 grid((unsigned)((units + per - 1) / per));
  uint8_t* d = static_cast<uint8_t*>(data);
  uint8_t* s = static_cast<uint8_t*>(scales);
  if (dtype == MOE_BF16)
    return launch_pdl(mx_quantize_kernel<__nv_bfloat16>, grid, dim3(kQThreads), 0, stream,
                      static_cast<const __nv_bfloat16*>(x), n_rows, rows, cols, offsets, G, group_tiles, tile_rows, d,
                      s);
  return launch_pdl(mx_quantize_kernel<float>, grid, dim3(kQThreads), 0, stream, static_cast<const float*>(x), n_rows,
                    rows, cols, offsets, G, group_tiles, tile_rows, d, s);
}

cudaError_t launch_mx_dequantize(moe_dtype dtype, const void* data, const void* scales, long long n_rows, int rows,
                                 int cols, const int32_t* offsets, int G, int group_tiles, size_t tile_rows, void* out,
                                 cudaStream_t stream) {
  const long long units = n_rows * mx_stages(cols);
  const int per = (kQThreads / 32) * kQUnits;
  const dim3 grid((unsigned)((units + per - 1) / per));
  const uint8_t* d = static_cast<const uint8_t*>(data);
  const uint8_t* s = static_cast<const uint8_t*>(scales);
  if (dtype == MOE_BF16)
    return launch_pdl(mx_dequantize_kernel<__nv_bfloat16>, grid, dim3(kQThreads), 0, stream, d, s, n_rows, rows, cols,
                      offsets, G, group_tiles, tile_rows, static_cast<__nv_bfloat16*>(out));
  return launch_pdl(mx_dequantize_kernel<float>, grid, dim3(kQThreads), 0, stream, d, s, n_rows, rows, cols, offsets, G,
                    group_tiles, tile_rows, static_cast<float*>(out));
}

}  // namespace moe
