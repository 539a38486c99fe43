// mx_quant.cu — rows to MXFP4 and back.
//
//   s = max(floor(log2(max |x_i|)) - 2, -127) over a block of 32 columns,
//   code_i = E2M1(x_i / 2^s), round to nearest even, at most 6;   x~_i = code_i 2^s
//
// Both directions only move memory: a row of C columns is C * (2 or 4) bytes
// on one side and C / 2 + C / 32 on the other. A lane takes 32 bytes of x at a
// time and the lanes of a warp follow one another through the matrix, across
// the ends of rows, so that narrow rows are read as evenly as wide ones; the
// lanes of a block agree on its scale by shuffles. Four such pieces are in
// flight per lane.
//
// Measured, 8 x 14336 x 4096: bf16 183 us to quantise and 186 back (6.5 and 6.4
// TB/s), fp32 323 and 325 us (6.6 and 6.5). With a warp per 256 columns of one
// row and 64-bit divisions the instructions bound it (bf16 266 and 254 us after
// the divisions were gone, 1093 us for both before).
#include "mx.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQUnits = 4;  // pieces per lane in flight

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
  const int tiles = b > a ? (int)(((unsigned)(b - a) + 255u) >> 8) * 2 : 0;
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

// A lane's pieces, 32 apart, with their place among the scales.
// Only the first one takes divisions, unless rows are shorter than a warp's
// step.
struct Pieces {
  uint32_t row, k;          // row, and piece of it
  uint32_t in;              // row in its group (dense)
  size_t group_row;         // first tile row of its group (dense)
  uint32_t per, rows, group_tiles;
  __device__ __forceinline__ Pieces(unsigned long long u, uint32_t per_, uint32_t rows_, uint32_t group_tiles_)
      : per(per_), rows(rows_), group_tiles(group_tiles_) {
    row = u >> 32 ? (uint32_t)(u / per) : (uint32_t)u / per;
    k = (uint32_t)(u - (unsigned long long)row * per);
    const uint32_t g = row / rows;
    in = row - g * rows;
    group_row = (size_t)g * group_tiles;
  }
  __device__ __forceinline__ void next() {
    k += 32;
    if (k < per) return;
    uint32_t n = 1;
    if (per < 32) n = k / per;
    k -= n * per;
    row += n;
    in += n;
    if (in < rows) return;
    const uint32_t g = per < 32 ? in / rows : 1u;
    in -= g * rows;
    group_row += (size_t)g * group_tiles;
  }
  // False for a row of no group, or one whose scales there is no room for.
  __device__ __forceinline__ bool place(const Groups& s, bool ragged, int G, size_t tile_rows, size_t* tile_row,
                                        int* r) const {
    bool live = true;
    if (ragged) {
      live = place_row(s, G, (int)row, tile_row, r);
    } else {
      *tile_row = group_row + (in >> 7);
      *r = (int)(in & 127);
    }
    return live && *tile_row < tile_rows;
  }
};

// The first piece of this lane.
__device__ __forceinline__ unsigned long long first_piece() {
  return ((unsigned long long)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5)) * (kQUnits * 32) + (threadIdx.x & 31);
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) mx_quantize_kernel(const T* __restrict__ x, uint32_t n_rows, int rows,
                                                                int cols, const int32_t* __restrict__ offsets, int G,
                                                                int group_tiles, size_t tile_rows,
                                                                uint8_t* __restrict__ data,
                                                                uint8_t* __restrict__ scales) {
  __shared__ Groups s_g;
  pdl_wait();
  pdl_trigger();
  if (offsets) load_groups(s_g, offsets, G);
  const int st = mx_stages(cols);
  const unsigned long long u = first_piece();
  constexpr int kCols = Piece<T>::kCols, kLanes = 32 / kCols;  // lanes of a block
  Pieces p(u, cols / kCols, rows, group_tiles);
  Pieces q = p;
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0;
  Piece<T> v[kQUnits];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    if (q.row < n_rows) load_sector(v[i].w, x + (u + 32 * i) * kCols, wide);
    q.next();
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const bool have = p.row < n_rows;
    uint32_t m = have ? v[i].amax() : 0u;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    size_t tile_row = 0;
    int r = 0;
    if (have && p.place(s_g, offsets != nullptr, G, tile_rows, &tile_row, &r)) {
      const uint32_t sb = mx_scale_byte(m);
      *reinterpret_cast<typename Piece<T>::Codes*>(data + (u + 32 * i) * (kCols / 2)) = v[i].codes(mx_inv_scale(sb));
      if (p.k % kLanes == 0) {
        const int b = (int)p.k / kLanes;
        scales[mx_scale_at(tile_row, st, r, b)] = (uint8_t)sb;
        if (b == cols / 32 - 1)  // zeros behind the row's last
          for (int z = b + 1; z < 8 * st; ++z) scales[mx_scale_at(tile_row, st, r, z)] = 0;
      }
    }
    p.next();
  }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) mx_dequantize_kernel(const uint8_t* __restrict__ data,
                                                                  const uint8_t* __restrict__ scales, uint32_t n_rows,
                                                                  int rows, int cols,
                                                                  const int32_t* __restrict__ offsets, int G,
                                                                  int group_tiles, size_t tile_rows,
                                                                  T* __restrict__ out) {
  __shared__ Groups s_g;
  pdl_wait();
  pdl_trigger();
  if (offsets) load_groups(s_g, offsets, G);
  const int st = mx_stages(cols);
  const unsigned long long u = first_piece();
  constexpr int kCols = Piece<T>::kCols, kLanes = 32 / kCols;  // lanes of a block
  Pieces p(u, cols / kCols, rows, group_tiles);
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  typename Piece<T>::Codes code[kQUnits];
  uint32_t sb[kQUnits];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    sb[i] = 0;
    size_t tile_row = 0;
    int r = 0;
    if (p.row < n_rows && p.place(s_g, offsets != nullptr, G, tile_rows, &tile_row, &r)) {
      code[i] = __ldcs(reinterpret_cast<const typename Piece<T>::Codes*>(data + (u + 32 * i) * (kCols / 2)));
      sb[i] = 0x100u | __ldg(scales + mx_scale_at(tile_row, st, r, (int)p.k / kLanes));
    }
    p.next();
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i)
    if (sb[i] & 0x100u) {
      Piece<T> v;
      v.values(code[i], mx_scale_value(sb[i] & 0xffu));
      store_sector(out + (u + 32 * i) * kCols, v.w, wide);
    }
}

}  // namespace

cudaError_t launch_mx_quantize(moe_dtype dtype, const void* x, long long total_rows, int rows, int cols,
                               const int32_t* offsets, int G, int group_tiles, size_t tile_rows, void* data,
                               void* scales, cudaStream_t stream) {
  const long long units = total_rows * (cols / (dtype == MOE_BF16 ? Piece<__nv_bfloat16>::kCols : Piece<float>::kCols));
  const uint32_t n_rows = (uint32_t)total_rows;  // below 2^31
  const int per = kQThreads * kQUnits;
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

cudaError_t launch_mx_dequantize(moe_dtype dtype, const void* data, const void* scales, long long total_rows, int rows,
                                 int cols, const int32_t* offsets, int G, int group_tiles, size_t tile_rows, void* out,
                                 cudaStream_t stream) {
  const long long units = total_rows * (cols / (dtype == MOE_BF16 ? Piece<__nv_bfloat16>::kCols : Piece<float>::kCols));
  const uint32_t n_rows = (uint32_t)total_rows;  // below 2^31
  const int per = kQThreads * kQUnits;
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
