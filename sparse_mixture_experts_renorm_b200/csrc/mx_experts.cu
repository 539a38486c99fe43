// mx_experts.cu — around the two MXFP4 products of the experts: the dispatch
// of given choices (the count of every expert's rows and each assignment's
// rank), the quantisation of every token's row on its way into
// expert-contiguous order, and the sum of each token's expert rows.
#include "mx.cuh"
#include "mx_internal.h"

namespace moe {
namespace {

constexpr int kCountThreads = 256;
constexpr int kCountWarps = kCountThreads / 32;
constexpr int kRowThreads = 256;  // 8 warps of 256 columns

// One block per kRouterTokensTc tokens. A warp takes a run of the block's
// assignments in order, 32 at a time: lanes that chose the same expert find
// each other (match) and take ranks in lane order behind the warp's count so
// far; then the warps' counts are summed in order.
__global__ void __launch_bounds__(kCountThreads) mx_count_kernel(const int32_t* __restrict__ idx, int T, int E, int k,
                                                                 int32_t* __restrict__ lrank,
                                                                 int32_t* __restrict__ blk_cnt,
                                                                 float* __restrict__ blk_psum, int32_t* status) {
  __shared__ int s_cnt[kCountWarps][kMaxExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kCountWarps * kMaxExperts; i += kCountThreads) (&s_cnt[0][0])[i] = 0;
  pdl_wait();
  __syncthreads();
  const long long base = (long long)blockIdx.x * kRouterTokensTc * k;
  const int n = (int)min((long long)kRouterTokensTc * k, (long long)T * k - base);
  const int per = kRouterTokensTc / kCountWarps * k;  // assignments of one warp: 16 k
  constexpr int kIt = kRouterTokensTc / kCountWarps * kMaxTopK / 32;
  int rank[kIt], ex[kIt];
#pragma unroll
  for (int it = 0; it < kIt; ++it) {
    const int o = it * 32 + lane, i = warp * per + o;
    ex[it] = -1;
    if (o < per && i < n) {
      ex[it] = idx[base + i];
      if (ex[it] < 0 || ex[it] >= E) {
        atomicOr(status, MOE_DEV_INTERNAL);
        ex[it] = -2;
      }
    }
    const unsigned same = __match_any_sync(0xffffffffu, ex[it]);
    rank[it] = -1;
    if (ex[it] >= 0) rank[it] = s_cnt[warp][ex[it]] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (ex[it] >= 0 && (same >> lane) == 1u) s_cnt[warp][ex[it]] = rank[it] + 1;  // its highest lane
    __syncwarp();
  }
  __syncthreads();
  if ((int)threadIdx.x < E) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kCountWarps; ++w) {
      const int c = s_cnt[w][threadIdx.x];
      s_cnt[w][threadIdx.x] = run;
      run += c;
    }
    blk_cnt[(size_t)blockIdx.x * E + threadIdx.x] = run;
    blk_psum[(size_t)blockIdx.x * E + threadIdx.x] = 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < kIt; ++it) {
    const int o = it * 32 + lane, i = warp * per + o;
    if (o < per && i < n) lrank[base + i] = ex[it] >= 0 ? s_cnt[warp][ex[it]] + rank[it] : -1;
  }
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Block (token t, 2048 columns): a warp rounds 256 columns, eight a lane, and
// writes them k times.
template <typename X>
__global__ void __launch_bounds__(kRowThreads) mx_dispatch_kernel(
    const X* __restrict__ x, int T, int d, int E, int k, int rb, const int32_t* __restrict__ topk_idx,
    const int32_t* __restrict__ lrank, const int32_t* __restrict__ blk_base, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ mtile, const float* __restrict__ gate, int32_t* __restrict__ inv,
    float* __restrict__ rgate, uint8_t* __restrict__ data, uint8_t* __restrict__ scales, int32_t* status) {
  __shared__ int s_row[kMaxTopK];   // dispatched row, -1: none
  __shared__ int s_tile[kMaxTopK];  // tile row of its scales
  __shared__ int s_in[kMaxTopK];    // row in the tile
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  pdl_wait();
  if ((int)threadIdx.x < k) {
    const size_t i = (size_t)t * k + threadIdx.x;
    const int e = topk_idx[i], lr = lrank[i];
    int row = -1;
    if (e >= 0 && e < E && lr >= 0) {
      row = blk_base[(size_t)(t / rb) * E + e] + lr;
      const int in = row - offsets[e];
      if (row < 0 || row >= T * k || in < 0 || row >= offsets[e + 1]) {
        atomicOr(status, MOE_DEV_INTERNAL);
        row = -1;
      } else {
        s_tile[threadIdx.x] = 2 * mtile[e] + (in >> 7);
        s_in[threadIdx.x] = in & 127;
      }
    }
    s_row[threadIdx.x] = row;
    if (blockIdx.y == 0) {
      inv[i] = row;
      if (row >= 0) rgate[row] = gate[i];
    }
  }
  __syncthreads();
  const int st = mx_stages(d);
  const int kb = blockIdx.y * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (kb >= st) return;
  const int c = kb * kMxStageCols + lane * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < d) load8(x + (size_t)t * d + c, v);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t sb = mx_scale_byte(m);
  const float is = mx_inv_scale(sb);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= is;
  const uint32_t code = mx_pack8(v);
  uint32_t word = sb << (8 * ((lane >> 2) & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  word |= __shfl_xor_sync(0xffffffffu, word, 8);
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    if (j >= k || s_row[j] < 0) continue;
    if (c < d) *reinterpret_cast<uint32_t*>(data + (size_t)s_row[j] * (d / 2) + c / 2) = code;
    if ((lane & 15) == 0)
      *reinterpret_cast<uint32_t*>(scales + mx_scale_at((size_t)s_tile[j], st, s_in[j], kb * 8 + (lane >> 2))) = word;
  }
}

// Block (token, 2048 columns): eight columns a thread, the k rows added in
// slot order in fp32 and rounded once.
__global__ void __launch_bounds__(kRowThreads) mx_combine_kernel(const uint4* __restrict__ y,
                                                                 const int32_t* __restrict__ inv, int nvec, int k,
                                                                 int R, uint4* __restrict__ out, int32_t* status) {
  __shared__ int s_row[kMaxTopK];
  const int t = blockIdx.x;
  pdl_wait();
  if ((int)threadIdx.x < k) {
    int row = inv[(size_t)t * k + threadIdx.x];
    if (row >= R) {
      atomicOr(status, MOE_DEV_INTERNAL);
      row = -1;
    }
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  const int i = blockIdx.y * kRowThreads + threadIdx.x;
  if (i >= nvec) return;
  uint4 v[kMaxTopK];
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j)
    if (j < k && s_row[j] >= 0) v[j] = __ldg(y + (size_t)s_row[j] * nvec + i);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    if (j < k && s_row[j] >= 0) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[2 * c] += __uint_as_float(w[c] << 16);
        acc[2 * c + 1] += __uint_as_float(w[c] & 0xffff0000u);
      }
    }
  }
  out[(size_t)t * nvec + i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                         pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

}  // namespace

cudaError_t launch_mx_count(const int32_t* topk_idx, int T, int E, int k, int32_t* lrank, int32_t* blk_cnt,
                            float* blk_psum, int32_t* status, cudaStream_t stream) {
  return launch_pdl(mx_count_kernel, dim3((T + kRouterTokensTc - 1) / kRouterTokensTc), dim3(kCountThreads), 0, stream,
                    topk_idx, T, E, k, lrank, blk_cnt, blk_psum, status);
}

cudaError_t launch_mx_dispatch(moe_dtype dtype, const void* x, int T, int d, int E, int k, int rb,
                               const int32_t* topk_idx, const int32_t* lrank, const int32_t* blk_base,
                               const int32_t* offsets, const int32_t* mtile, const float* topk_gate, int32_t* inv,
                               float* rgate, void* data, void* scales, int32_t* status, cudaStream_t stream) {
  const dim3 grid(T, (mx_stages(d) + 7) / 8);
  uint8_t* q = static_cast<uint8_t*>(data);
  uint8_t* s = static_cast<uint8_t*>(scales);
  if (dtype == MOE_BF16)
    return launch_pdl(mx_dispatch_kernel<__nv_bfloat16>, grid, dim3(kRowThreads), 0, stream,
                      static_cast<const __nv_bfloat16*>(x), T, d, E, k, rb, topk_idx, lrank, blk_base, offsets, mtile,
                      topk_gate, inv, rgate, q, s, status);
  return launch_pdl(mx_dispatch_kernel<float>, grid, dim3(kRowThreads), 0, stream, static_cast<const float*>(x), T, d,
                    E, k, rb, topk_idx, lrank, blk_base, offsets, mtile, topk_gate, inv, rgate, q, s, status);
}

cudaError_t launch_mx_combine(const void* y, const int32_t* inv, int T, int d, int k, void* out, int32_t* status,
                              cudaStream_t stream) {
  const int nvec = d / 8;
  return launch_pdl(mx_combine_kernel, dim3(T, (nvec + kRowThreads - 1) / kRowThreads), dim3(kRowThreads), 0, stream,
                    static_cast<const uint4*>(y), inv, nvec, k, T * k, static_cast<uint4*>(out), status);
}

}  // namespace moe
