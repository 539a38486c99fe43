// mx_experts.cu — around the two MXFP4 products of the experts: the dispatch
// of given choices (the count of every expert's rows and each assignment's
// rank), the quantisation of every token's row on its way into
// expert-contiguous order, and the sum of each token's expert rows.
//
// All of it moves memory. Measured with cold caches, 4096 tokens of the
// fine-grained layer (d 2048, 64 experts, k 6): count 5 us, dispatch 15 us (17 MB
// read, 27 MB written), sum 23 us (102 MB read, 17 MB written: 5.2 TB/s).
#include "mx.cuh"
#include "mx_internal.h"

namespace moe {
namespace {

constexpr int kCountThreads = 256;
constexpr int kCountWarps = kCountThreads / 32;
constexpr int kRowThreads = 256;

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
  pdl_trigger();
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

// The dispatch. A block takes kTok consecutive tokens (of one block of rb) and
// asks for their first pieces of x before it works out where their rows go.
struct DispatchPlan {
  int tot[kMaxExperts];     // rows of every expert
  int before[kMaxExperts];  // and those of earlier tokens, of other blocks
  int off[kMaxExperts + 1];
  int mt[kMaxExperts + 1];
};

// Sums or counts tot and before, and scans them; block 0 writes the results.
__device__ void scan_rows(DispatchPlan& s, const MxDispatch& a, int T, int E, int k, int t0, bool write) {
  const int tid = threadIdx.x;
  if (a.scan == kScanBlocks) {
    const int nb = (T + a.rb - 1) / a.rb, mine = t0 / a.rb;
    for (int e = tid; e < E; e += kRowThreads) s.tot[e] = s.before[e] = 0;
    __syncthreads();
    // a thread per (slice of the blocks, expert)
    const int S = max(1, kRowThreads / E);
    for (int i = tid; i < S * E; i += kRowThreads) {
      const int e = i % E, b0 = i / E * nb / S, b1 = (i / E + 1) * nb / S;
      int tot = 0, before = 0;
#pragma unroll 8
      for (int b = b0; b < b1; ++b) {
        const int c = a.blk[(size_t)b * E + e];
        tot += c;
        before += b < mine ? c : 0;
      }
      if (tot) atomicAdd(&s.tot[e], tot);
      if (before) atomicAdd(&s.before[e], before);
    }
  } else {
    for (int e = tid; e < E; e += kRowThreads) s.tot[e] = s.before[e] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < T * k; i += kRowThreads) {
      const int e = a.topk_idx[i];
      if (e < 0 || e >= E) continue;
      atomicAdd(&s.tot[e], 1);
      if (i < t0 * k) atomicAdd(&s.before[e], 1);
    }
  }
  __syncthreads();
  if (tid < 32) {
    int rows = 0, tiles = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + tid, n = e < E ? s.tot[e] : 0, m = (n + 255) >> 8;
      int ri = n, ti = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ri, o), y = __shfl_up_sync(0xffffffffu, ti, o);
        if (tid >= o) ri += x, ti += y;
      }
      if (e < E) {
        s.off[e] = rows + ri - n;
        s.mt[e] = tiles + ti - m;
      }
      rows += __shfl_sync(0xffffffffu, ri, 31);
      tiles += __shfl_sync(0xffffffffu, ti, 31);
    }
    if (tid == 0) s.off[E] = rows, s.mt[E] = tiles;
  }
  __syncthreads();
  if (write) {
    for (int e = tid; e <= E; e += kRowThreads) {
      if (e < E) a.counts[e] = s.tot[e];
      a.offsets[e] = s.off[e];
      a.mtile[e] = s.mt[e];
    }
  }
}

constexpr int kDispatchPieces = 4;  // pieces of a thread in flight

template <typename X, int kTok>
__global__ void __launch_bounds__(kRowThreads, 4) mx_dispatch_kernel(const X* __restrict__ x, int T, int d, int E, int k,
                                                                  const MxDispatch a, int32_t* __restrict__ inv,
                                                                  float* __restrict__ rgate, uint8_t* __restrict__ data,
                                                                  uint8_t* __restrict__ scales, int32_t* status) {
  constexpr int kCols = Piece<X>::kCols, kLanes = 32 / kCols;  // lanes of a block of 32 columns
  static_assert(kTok == 1 || kTok * kMaxTopK <= kRowThreads, "a thread per choice");
  __shared__ DispatchPlan s_p;
  // where a choice's codes and scales begin; NULL: nowhere
  __shared__ uint8_t* s_data[kTok * kMaxTopK];
  __shared__ uint8_t* s_scale[kTok * kMaxTopK];
  const int st = mx_stages(d);
  const int t0 = blockIdx.x * kTok, nt = min(kTok, T - t0);
  const int per = d / kCols, pieces = nt * per;  // of a token, of the block (whose rows are contiguous)
  pdl_wait();
  pdl_trigger();
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 31) == 0;
  const X* src = x + (size_t)t0 * d;
  Piece<X> v[kDispatchPieces];
#pragma unroll
  for (int i = 0; i < kDispatchPieces; ++i) {
    const int p = i * kRowThreads + (int)threadIdx.x;
    if (p < pieces) load_sector(v[i].w, src + (size_t)p * kCols, wide);
  }
  // this thread's choice
  const int o = threadIdx.x;
  const bool chooses = o < nt * k;
  const size_t oi = (size_t)t0 * k + o;
  const int e = chooses ? a.topk_idx[oi] : 0, lrank = chooses && a.scan != kScanAll ? a.lrank[oi] : 0;
  const float gate = chooses ? a.topk_gate[oi] : 0.f;
  if (a.scan != kScanDone) scan_rows(s_p, a, T, E, k, t0, blockIdx.x == 0);
  if (chooses) {
    int row = -1;
    if (e < 0 || e >= E) {
      atomicOr(status, MOE_DEV_INTERNAL);
    } else {
      int first, end, tile;
      if (a.scan == kScanDone) {
        first = a.offsets[e], end = a.offsets[e + 1], tile = a.mtile[e];
        row = a.blk[(size_t)(t0 / a.rb) * E + e] + lrank;
      } else {
        first = s_p.off[e], end = s_p.off[e + 1], tile = s_p.mt[e];
        row = first + s_p.before[e];
        if (a.scan == kScanBlocks) {
          row += lrank;
        } else {  // the block's own choices of this expert before this one
          for (int q = 0; q < o; ++q) row += a.topk_idx[(size_t)t0 * k + q] == e;
        }
      }
      const int in = row - first;
      if (row < 0 || row >= T * k || in < 0 || row >= end) {
        atomicOr(status, MOE_DEV_INTERNAL);
        row = -1;
      } else {
        s_scale[o] = scales + mx_scale_at((size_t)(2 * tile + (in >> 7)), st, in & 127, 0);
        rgate[row] = gate;
      }
    }
    s_data[o] = row >= 0 ? data + (size_t)row * (d / 2) : nullptr;
    inv[oi] = row;
  }
  __syncthreads();
  const bool words = d % 128 == 0;  // four blocks' bytes are then a word, and 4 kLanes lanes of one row hold them
  for (int p0 = 0; p0 < pieces; p0 += kDispatchPieces * kRowThreads) {
    if (p0 > 0) {
#pragma unroll
      for (int i = 0; i < kDispatchPieces; ++i) {
        const int p = p0 + i * kRowThreads + (int)threadIdx.x;
        if (p < pieces) load_sector(v[i].w, src + (size_t)p * kCols, wide);
      }
    }
#pragma unroll
    for (int i = 0; i < kDispatchPieces; ++i) {
      const int p = p0 + i * kRowThreads + (int)threadIdx.x;
      if (p0 + i * kRowThreads >= pieces) break;
      const bool have = p < pieces;
      uint32_t m = have ? v[i].amax() : 0u;
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t sb = mx_scale_byte(m);
      const int lane = threadIdx.x & 31;
      uint32_t word = sb << (8 * (lane / kLanes & 3));
#pragma unroll
      for (int o = kLanes; o < 4 * kLanes; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
      if (!have) continue;
      const typename Piece<X>::Codes code = v[i].codes(mx_inv_scale(sb));
      const int t = kTok == 1 ? 0 : p / per, q = p - t * per, b = q / kLanes;
      const int at = (b >> 3) * kMxStageBytes + ((b >> 2) & 1) * 512 + (b & 3);  // from the row's first scale
      const bool stores = words ? q % (4 * kLanes) == 0 : q % kLanes == 0;
      const bool ends = b == d / 32 - (words ? 4 : 1);  // zeros follow to the end of the stage
#pragma unroll 2
      for (int o = t * k; o < t * k + k; ++o) {
        uint8_t* to = s_data[o];
        if (!to) continue;
        *reinterpret_cast<typename Piece<X>::Codes*>(to + q * (kCols / 2)) = code;
        if (!stores) continue;
        to = s_scale[o];
        if (words) {
          *reinterpret_cast<uint32_t*>(to + at) = word;
          if (ends && (b & 4) == 0) *reinterpret_cast<uint32_t*>(to + at + 512) = 0;
        } else {
          to[at] = (uint8_t)sb;
          if (ends)
            for (int z = b + 1; z < 8 * st; ++z) to[(z >> 3) * kMxStageBytes + ((z >> 2) & 1) * 512 + (z & 3)] = 0;
        }
      }
    }
  }
}

// Block (token, 2048 columns): eight columns a thread, the k rows added in
// slot order in fp32 and rounded once.
__global__ void __launch_bounds__(kRowThreads) mx_combine_kernel(const uint4* __restrict__ y,
                                                                 const uint8_t* __restrict__ y_exp,
                                                                 const int32_t* __restrict__ inv, int T, int nvec, int k,
                                                                 uint4* __restrict__ out, int32_t* status) {
  __shared__ int row[kMaxTopK];
  const int R = T * k, t = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < kMaxTopK) {
    int r = (int)threadIdx.x < k ? inv[(size_t)t * k + threadIdx.x] : -1;
    if (r >= R) {
      atomicOr(status, MOE_DEV_INTERNAL);
      r = -1;
    }
    row[threadIdx.x] = r;
  }
  __syncthreads();
  const int i = blockIdx.y * kRowThreads + threadIdx.x;
  if (i >= nvec) return;
  const uint8_t* exps = y_exp + y16_exp_at((size_t)R, i * 8, 0);
  constexpr int kAtOnce = 4;  // rows in flight: more take registers that other blocks need
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int j0 = 0; j0 < k; j0 += kAtOnce) {
    uint4 v[kAtOnce];
    uint32_t e[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int r = row[j0 + j];
      if (r >= 0) {
        v[j] = __ldg(y + (size_t)r * nvec + i);
        e[j] = __ldg(exps + (size_t)r * 8);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (row[j0 + j] < 0) continue;
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      if (e[j] == 0xffu) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[2 * c] += __uint_as_float(w[c] << 16);
          acc[2 * c + 1] += __uint_as_float(w[c] & 0xffff0000u);
        }
      } else {
        const float step = y16_step(e[j]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = y16_numbers(w[c]);
          acc[2 * c] = fmaf(f.x, step, acc[2 * c]);
          acc[2 * c + 1] = fmaf(f.y, step, acc[2 * c + 1]);
        }
      }
    }
  }
  out[(size_t)t * nvec + i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                      pack_bf16x2(acc[6], acc[7]));
}

}  // namespace

cudaError_t launch_mx_count(const int32_t* topk_idx, int T, int E, int k, int32_t* lrank, int32_t* blk_cnt,
                            float* blk_psum, int32_t* status, cudaStream_t stream) {
  return launch_pdl(mx_count_kernel, dim3((T + kRouterTokensTc - 1) / kRouterTokensTc), dim3(kCountThreads), 0, stream,
                    topk_idx, T, E, k, lrank, blk_cnt, blk_psum, status);
}

template <typename X>
static cudaError_t dispatch(const void* x, int T, int d, int E, int k, const MxDispatch& a, int32_t* inv, float* rgate,
                            void* data, void* scales, int32_t* status, cudaStream_t stream) {
  const X* src = static_cast<const X*>(x);
  uint8_t *q = static_cast<uint8_t*>(data), *sc = static_cast<uint8_t*>(scales);
  // eight tokens a block where that still fills the SMs: the placing is then
  // done for all of them at once
  if (T >= 2048)
    return launch_pdl(mx_dispatch_kernel<X, 8>, dim3((T + 7) / 8), dim3(kRowThreads), 0, stream, src, T, d, E, k, a, inv,
                      rgate, q, sc, status);
  return launch_pdl(mx_dispatch_kernel<X, 1>, dim3(T), dim3(kRowThreads), 0, stream, src, T, d, E, k, a, inv, rgate, q,
                    sc, status);
}

cudaError_t launch_mx_dispatch(moe_dtype dtype, const void* x, int T, int d, int E, int k, const MxDispatch& a,
                               int32_t* inv, float* rgate, void* data, void* scales, int32_t* status,
                               cudaStream_t stream) {
  return dtype == MOE_BF16 ? dispatch<__nv_bfloat16>(x, T, d, E, k, a, inv, rgate, data, scales, status, stream)
                           : dispatch<float>(x, T, d, E, k, a, inv, rgate, data, scales, status, stream);
}

cudaError_t launch_mx_combine(const void* y, const uint8_t* y_exp, const int32_t* inv, int T, int d, int k, void* out,
                              int32_t* status, cudaStream_t stream) {
  const int nvec = d / 8;
  return launch_pdl(mx_combine_kernel, dim3(T, (nvec + kRowThreads - 1) / kRowThreads), dim3(kRowThreads), 0, stream,
                    static_cast<const uint4*>(y), y_exp, inv, T, nvec, k, static_cast<uint4*>(out), status);
}

}  // namespace moe
