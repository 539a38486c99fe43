// few.cu — the whole layer for at most 16 tokens in two kernels.
//
//   few_up:   p = softmax(x W_r^T + b), the k best experts and their gates;
//             H[row] = SiLU(W_g[e] x_t) * (W_u[e] x_t) for every choice (t, e)
//   few_down: out[t] = sum_j gate[t, j] * W_d[e_j] H[row(t, j)]
//
// Bound by the weights: every chosen expert's 3 d I weights are read once,
// and each takes part in at most 16 products. So both kernels are streams: a
// warp fills a ring in shared memory with rows of weights (bulk copies of 1
// KB a row), a second one with the same columns of the rows that multiply
// them, and eight warps consume 16 weight rows a stage, 64 bytes a row and
// warp at a time, on mma.sync (bf16) or FFMA (fp32). tcgen05 has nothing to
// give here: 16 rows of weights against 8 tokens are one m16n8k16 step, the
// rate of the loads is a tenth of what it takes, and its operand tiles would
// hold 128 rows of one expert where 16 keep the SMs evenly loaded.
//
// Routing has to be known before the first weight can be asked for, and a
// kernel of its own would cost a launch: instead each cluster of few_up
// computes all of it, its CTAs a part of the d columns each, exchanged
// through distributed shared memory. Every cluster adds in the same order,
// so all come to the same choices, and few_down takes them from topk_idx.
//
// A down product's rows of different experts belong to the same output: each
// finished part is written to y, and the last of a block of 16 columns to
// finish adds them up, in slot order whatever the order of arrival.
#include <atomic>
#include <math.h>

#include "few_internal.h"
#include "pair.cuh"

namespace moe {
namespace {

constexpr int kWarps = 10;               // 0: weights, 1: token rows, 2..9: products
constexpr int kThreads = 32 * kWarps;
constexpr int kMathWarps = 8;
constexpr int kMath = 32 * kMathWarps;
constexpr int kRows = 16;                // weight rows of a stage
constexpr int kBox = 512;                // bytes of a row in one tile load
constexpr int kBoxes = 4;                // tile loads side by side in a stage
constexpr int kChunk = kBox * kBoxes;    // bytes of a row in a stage
constexpr int kWeightBytes = kRows * kChunk;
constexpr int kTokPitch = kFewTokPitch;  // bytes between token rows: two rows of a quarter-warp's load on different banks
static_assert(kTokPitch == kChunk + 64, "pitch");
constexpr int kMaxStages = 8;
constexpr int kMaxRows = kFewTokens * kMaxTopK;
constexpr int kCluster = 4;              // CTAs that share one routing
constexpr int kPassE = 64;               // experts whose logits a warp holds at a time
constexpr int kSmemTotal = 227 * 1024;

struct Plan {
  int n_act;                        // experts with tokens
  int most;                         // tokens of the one with most
  int expert[kMaxRows];             // ascending
  int base[kMaxRows + 1];           // first row of each
  int tj[kMaxRows];                 // t * k + j of a row
  float gate[kMaxRows];
  uint32_t mask[kMaxExperts];       // tokens of an expert
  int slot[kMaxExperts];
};

struct Ctrl {
  uint64_t full[kMaxStages];   // both producers' bytes
  uint64_t empty[kMaxStages];  // the math warps
  volatile int abort;
  int last;
  int idx[kMaxRows];
  float gate[kMaxRows];
  float red[kWarps];
  Plan plan;
};

// kParts: partial sums of an item (bf16: every warp has its own columns; fp32:
// two halves of the columns, four groups of rows). kHid: rows that a hidden
// row is stored as. bf16 keeps it in two terms, hi + lo, whose sum is off by
// 2^-17: rounded to one, it would double the error that the output's own
// rounding makes, and the second term costs only shared memory and issue slots
// (both are columns of the same mma.sync while an expert has few tokens).
template <typename X>
struct Traits;
template <>
struct Traits<__nv_bfloat16> {
  static constexpr int kParts = kMathWarps, kHid = 2;
};
template <>
struct Traits<float> {
  static constexpr int kParts = 2, kHid = 1;
};
constexpr int kRedLd = kFewTokens + 1;
template <typename X>
constexpr int red_floats() { return Traits<X>::kParts * kRows * kRedLd; }
template <typename X>
constexpr int fixed_bytes() { return (int)((sizeof(Ctrl) + 127) / 128 * 128 + 2 * red_floats<X>() * 4); }

// The ring's shape follows from the most tokens that an expert got.
struct Ring {
  uint8_t* base;
  int slot, stages;
};
template <typename X, bool kUp>
__device__ __forceinline__ Ring ring_of(uint8_t* base, const Plan& p) {
  int rows = kUp ? p.most : p.most * Traits<X>::kHid;
  if (sizeof(X) == 4) rows = (rows + 3) & ~3;  // fp32 multiplies four token rows at a time
  Ring r;
  r.base = base;
  r.slot = (kWeightBytes + rows * kTokPitch + 127) & ~127;
  r.stages = min(kMaxStages, (kSmemTotal - fixed_bytes<X>()) / r.slot);
  return r;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void math_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kMath) : "memory"); }
// The same, and whether any thread of it said no: all leave together.
__device__ __forceinline__ bool math_sync_all(bool ok) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.eq.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)ok), "n"(kMath)
      : "memory");
  return any == 0;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 columns: a lane holds 8 consecutive ones of a row, and the order of the
// columns inside a product does not matter as long as both sides agree.
__device__ __forceinline__ void mma_block(float (&c)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma_bf16(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma_bf16(c, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// N sums of a warp's lanes: after it, lane l holds sum number l / (32 / N).
template <int N>
__device__ __forceinline__ float reduce_many(float (&v)[N]) {
  static_assert(N == 16, "four steps");
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int off = 16 >> s, n = N >> (s + 1);
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// Groups the choices by expert: idx[T * k] in shared memory, every thread of
// the block. A token names an expert once.
__device__ void make_plan(Plan& p, const int* idx, const float* gate, int T, int E, int k) {
  const int R = T * k;
  for (int e = threadIdx.x; e < E; e += kThreads) p.mask[e] = 0;
  __syncthreads();
  const int i = threadIdx.x;
  if (i < R) atomicOr(&p.mask[idx[i]], 1u << (i / k));
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int act = 0, rows = 0, most = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < E ? __popc(p.mask[e]) : 0;
      const uint32_t live = __ballot_sync(0xffffffffu, n > 0);
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (n > 0) {
        const int s = act + __popc(live & ((1u << lane) - 1u));
        p.expert[s] = e;
        p.base[s] = rows + incl - n;
        p.slot[e] = s;
      }
      most = max(most, (int)__reduce_max_sync(0xffffffffu, (unsigned)n));
      act += __popc(live);
      rows += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      p.n_act = act;
      p.most = most;
      p.base[act] = rows;
    }
  }
  __syncthreads();
  if (i < R) {
    const int e = idx[i], t = i / k;
    const int row = p.base[p.slot[e]] + __popc(p.mask[e] & ((1u << t) - 1u));
    p.tj[row] = i;
    p.gate[row] = gate[i];
  }
  __syncthreads();
}

// ---------------------------------------------------------------- routing --

// Partial logits of all T tokens and E experts over columns [c0, c1): warp
// sums in scratch [kWarps][kPassE][T], added up in warp order into every
// cluster CTA's part[rank][T][E].
template <typename X>
__device__ void logits_part(const X* __restrict__ x, const X* __restrict__ wr, int T, int d, int E, int c0, int c1,
                            float* scratch, float* part, int rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < E; e0 += kPassE) {
    const int ne = min(kPassE, E - e0);
    float* mine = scratch + warp * kPassE * kFewTokens;
    if constexpr (sizeof(X) == 2) {
      float acc[kPassE / 16][2][4];
#pragma unroll
      for (int m = 0; m < kPassE / 16; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
      const int r = lane >> 2;
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
      for (int c = c0 + warp * 32; c < c1; c += kWarps * 32) {
        const int col = c + (lane & 3) * 8;
        const bool in = col < c1;
        uint4 b[2];
#pragma unroll
        for (int n = 0; n < 2; ++n)
          b[n] = in && n * 8 + r < T ? __ldg(reinterpret_cast<const uint4*>(x + (size_t)(n * 8 + r) * d + col)) : zero;
#pragma unroll
        for (int m = 0; m < kPassE / 16; ++m) {
          if (m * 16 < ne) {
            const int e = m * 16 + r;
            const X* w = wr + (size_t)(e0 + e) * d + col;
            const uint4 lo = in && e < ne ? __ldg(reinterpret_cast<const uint4*>(w)) : zero;
            const uint4 hi = in && e + 8 < ne ? __ldg(reinterpret_cast<const uint4*>(w + (size_t)8 * d)) : zero;
            mma_block(acc[m][0], lo, hi, b[0]);
            if (T > 8) mma_block(acc[m][1], lo, hi, b[1]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kPassE / 16; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = m * 16 + r + (i >> 1) * 8, t = n * 8 + (lane & 3) * 2 + (i & 1);
            if (m * 16 < ne) mine[e * kFewTokens + t] = acc[m][n][i];
          }
    } else {
      for (int e = 0; e < ne; e += 4)
        for (int t = 0; t < T; t += 4) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
          for (int col = c0 + warp * 128 + lane * 4; col < c1; col += kWarps * 128) {
            float4 a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] = __ldg(reinterpret_cast<const float4*>(wr + (size_t)(e0 + min(e + i, ne - 1)) * d + col));
              b[i] = __ldg(reinterpret_cast<const float4*>(x + (size_t)min(t + i, T - 1) * d + col));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 &p = a[i >> 2], &q = b[i & 3];
              v[i] = fmaf(p.w, q.w, fmaf(p.z, q.z, fmaf(p.y, q.y, fmaf(p.x, q.x, v[i]))));
            }
          }
          const float s = reduce_many(v);
          if ((lane & 1) == 0) mine[(e + (lane >> 3)) * kFewTokens + t + ((lane >> 1) & 3)] = s;
        }
    }
    __syncthreads();
    const int peers = kCluster;
    for (int i = threadIdx.x; i < ne * T; i += kThreads) {
      const int t = i / ne, e = i - t * ne;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += scratch[(w * kPassE + e) * kFewTokens + t];
      float* dst = part + ((size_t)rank * T + t) * E + e0 + e;
      for (int c = 0; c < peers; ++c) store_cluster(map_to_cta(dst, c), s);
    }
    __syncthreads();
  }
}

// Softmax, the k best (ties to the lower index) and their gates, one warp a
// token. part [kCluster][T][E]; the probabilities replace part[0].
template <typename X>
__device__ void choose(const FewArgs& a, float* part, Ctrl& c, bool write) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kPer = kMaxExperts / 32;
  const int T = a.T, E = a.E, k = a.k;
  for (int t = warp; t < T; t += kWarps) {
    float v[kPer];
    float m = -INFINITY;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      v[i] = -INFINITY;
      if (e < E) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kCluster; ++q) s += part[((size_t)q * T + t) * E + e];
        if (a.br) s += a.br[e];
        finite = finite && isfinite(s);
        v[i] = s;
        m = fmaxf(m, s);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += lane + 32 * i < E ? expf(v[i] - m) : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < E) part[(size_t)t * E + lane + 32 * i] = expf(v[i] - m) / sum;
    if (!__all_sync(0xffffffffu, finite) && lane == 0 && write) atomicOr(a.status, MOE_DEV_NONFINITE);
    // k rounds of an arg-max over the logits, which rank as their exact
    // probabilities do; NaN ranks lowest, so that every token still gets k
    // different experts
    uint32_t taken = 0;
    float mine = 0.f, total = 0.f;
    int mine_e = 0;
    for (int j = 0; j < k; ++j) {
      float bv = -INFINITY;
      int be = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((taken >> i) & 1u)) {
          const float l = v[i] != v[i] ? -INFINITY : v[i];
          if (l > bv || (l == bv && e < be)) bv = l, be = e;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oe = __shfl_xor_sync(0xffffffffu, be, o);
        if (ov > bv || (ov == bv && oe < be)) bv = ov, be = oe;
      }
      if ((be & 31) == lane) taken |= 1u << (be >> 5);
      const float p = expf(bv - m) / sum;
      total += p;
      if (lane == j) mine = p, mine_e = be;
    }
    if (lane < k) {
      const float g = !a.renorm ? mine : total > 0.f ? mine / total : 1.f / (float)k;
      c.idx[t * k + lane] = mine_e;
      c.gate[t * k + lane] = g;
      if (write) {
        a.idx[(size_t)t * k + lane] = mine_e;
        a.gate[(size_t)t * k + lane] = g;
      }
    }
  }
}

// counts and the load-balancing statistic, by one block; prob [T][E].
__device__ void statistics(const FewArgs& a, const float* prob, Ctrl& c) {
  for (int e = threadIdx.x; e < a.E; e += kThreads)
    if (a.counts) a.counts[e] = __popc(c.plan.mask[e]);
  if (!a.aux) return;
  float s = 0.f;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float p = 0.f;
    for (int t = 0; t < a.T; ++t) p += prob[(size_t)t * a.E + e];
    s += (float)__popc(c.plan.mask[e]) * p;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) c.red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.f;
    for (int w = 0; w < kWarps; ++w) sum += c.red[w];
    *a.aux = sum * (float)a.E / ((float)(a.T * a.k) * (float)a.T);
  }
}

// ------------------------------------------------------------------ stream --

// One piece of work: 16 weight rows (of one expert) against that expert's
// token rows over chunks [c0, c1) of their columns.
struct Item {
  int s;       // active expert
  int blk;     // block of rows
  int part;    // of the columns (few_down)
  int c0, c1;  // chunks
  int first, n;  // token rows of the expert
};

template <typename X, bool kUp>
struct Work {
  int n_blk, split, chunks, total;
  __device__ Work(const FewArgs& a, const Plan& p) {
    const int K = kUp ? a.d : a.I;
    chunks = (K * (int)sizeof(X) + kChunk - 1) / kChunk;
    n_blk = kUp ? (a.I + 7) / 8 : (a.d + 15) / 16;
    split = 1;
    const int items = p.n_act * n_blk;
    if (!kUp) {
      // the parts that leave the busiest block the fewest chunks; a finer
      // split has to gain 3 %
      float best = (float)((items + gridDim.x - 1) / gridDim.x) * (float)chunks;
      for (int q = 2; q <= min(a.split, chunks); ++q) {
        const float t = (float)((items * q + gridDim.x - 1) / gridDim.x) * (float)((chunks + q - 1) / q);
        if (t < 0.97f * best) best = t, split = q;
      }
    }
    total = items * split;
  }
  __device__ __forceinline__ Item item(int i, const Plan& p) const {
    Item w;
    const int q = i / split;
    w.part = i - q * split;
    w.s = q / n_blk;
    w.blk = q - w.s * n_blk;
    w.c0 = w.part * chunks / split;
    w.c1 = (w.part + 1) * chunks / split;
    w.first = p.base[w.s];
    w.n = p.base[w.s + 1] - w.first;
    return w;
  }
};

// Ring position.
struct Pos {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) stage = 0, phase ^= 1u;
  }
};

// Where an expert's hidden rows are: chunk after chunk of kChunk bytes, in each
// all its rows (kHid of them for every token) kTokPitch bytes apart, so that a
// stage's part is one contiguous copy.
template <typename X>
__device__ __forceinline__ size_t hidden_at(int first, int n, int chunks, int chunk, int row) {
  constexpr int kHid = Traits<X>::kHid;
  return (((size_t)first * chunks + (size_t)n * chunk) * kHid + row) * kTokPitch;
}

// The weights' producer: one lane. Rows past the last block's are read from
// the next expert, or as zeros, and go into sums that nobody takes.
template <typename X, bool kUp>
__device__ bool produce_weights(const FewMaps& maps, const FewArgs& a, Ctrl& c, const Ring& ring, Pos& pos, int& issued) {
  const Work<X, kUp> work(a, c.plan);
  const int row_bytes = (kUp ? a.d : a.I) * (int)sizeof(X);
  for (int i = blockIdx.x; i < work.total; i += gridDim.x) {
    const Item w = work.item(i, c.plan);
    const int e = c.plan.expert[w.s];
    const int row = kUp ? e * a.I + w.blk * 8 : e * a.d + w.blk * kRows;
    for (int ch = w.c0; ch < w.c1; ++ch) {
      if (!mbar_wait(&c.empty[pos.stage], pos.phase ^ 1u, &c.abort, a.status, a.limit_ns)) return false;
      uint8_t* dst = ring.base + (size_t)pos.stage * ring.slot;
      const int boxes = min(kBoxes, (row_bytes - ch * kChunk + kBox - 1) / kBox);
      mbar_arrive_expect_tx(&c.full[pos.stage], (uint32_t)(boxes * kRows * kBox));
      for (int b = 0; b < boxes; ++b) {
        const int col = (ch * kChunk + b * kBox) / (int)sizeof(X);
        uint8_t* to = dst + b * kRows * kBox;
        if (kUp) {  // rows 0..7: gate rows of 8 hidden units, 8..15: their up rows
          tma_load_2d(to, &maps.wg, &c.full[pos.stage], col, row);
          tma_load_2d(to + 8 * kBox, &maps.wu, &c.full[pos.stage], col, row);
        } else {
          tma_load_2d(to, &maps.wd, &c.full[pos.stage], col, row);
        }
      }
      ++issued;
      pos.next(ring.stages);
    }
  }
  return true;
}

// The token rows' producer: one warp, lane l copies row l of x, or lane 0 all
// hidden rows.
template <typename X, bool kUp>
__device__ bool produce_tokens(const FewArgs& a, Ctrl& c, const Ring& ring, Pos& pos, int& issued) {
  const int lane = threadIdx.x & 31;
  const Work<X, kUp> work(a, c.plan);
  const int row_bytes = (kUp ? a.d : a.I) * (int)sizeof(X);
  for (int i = blockIdx.x; i < work.total; i += gridDim.x) {
    const Item w = work.item(i, c.plan);
    const uint8_t* src = nullptr;
    if (kUp && lane < w.n)
      src = static_cast<const uint8_t*>(a.x) + (size_t)(c.plan.tj[w.first + lane] / a.k) * row_bytes;
    for (int ch = w.c0; ch < w.c1; ++ch) {
      const uint32_t bytes = kUp ? (uint32_t)min(kChunk, row_bytes - ch * kChunk)
                                 : (uint32_t)(w.n * Traits<X>::kHid * kTokPitch);
      bool free = true;
      if (lane == 0) {
        free = mbar_wait(&c.empty[pos.stage], pos.phase ^ 1u, &c.abort, a.status, a.limit_ns);
        if (free) mbar_arrive_expect_tx(&c.full[pos.stage], kUp ? w.n * bytes : bytes);
      }
      if (!__shfl_sync(0xffffffffu, (int)free, 0)) return false;
      uint8_t* dst = ring.base + (size_t)pos.stage * ring.slot + kWeightBytes;
      if (kUp) {
        if (src) bulk_load(dst + lane * kTokPitch, src + (size_t)ch * kChunk, bytes, &c.full[pos.stage]);
      } else if (lane == 0) {
        bulk_load(dst, static_cast<const uint8_t*>(a.h) + hidden_at<X>(w.first, w.n, work.chunks, ch, 0), bytes,
                  &c.full[pos.stage]);
      }
      ++issued;
      pos.next(ring.stages);
    }
  }
  return true;
}

// A block that gives up still waits for the copies it has asked for.
__device__ void drain(const FewArgs& a, Ctrl& c, const Ring& ring, Pos pos, int issued) {
  const int n = min(issued, ring.stages);
  for (int i = 0; i < n; ++i) {
    if (pos.stage == 0) pos.stage = ring.stages, pos.phase ^= 1u;
    --pos.stage;
    if (!mbar_wait(&c.full[pos.stage], pos.phase, nullptr, a.status, a.limit_ns)) return;
  }
}

// Sums of one item into red [parts][kRows][kRedLd]. False: a wait gave up.
//
// bf16: warp w takes bytes 256 w .. 256 w + 255 of the stage's rows, 128 at a
// time. Rows of weights lie 512 bytes apart, so the two rows that a
// quarter-warp reads at once would fall on the same banks: odd rows take the
// two halves of the 128 bytes in the other order.
template <bool kUp>
__device__ bool multiply(const Item& w, const FewArgs& a, Ctrl& c, const Ring& ring, int row_bytes, Pos& pos,
                         float* red, const __nv_bfloat16*) {
  constexpr int kTiles = kUp ? 2 : 4;  // of 8 columns: a token each, or hi and lo of four
  const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
  const int r = lane >> 2, q = lane & 3;
  const bool odd = r & 1;
  const int cols = kUp ? w.n : 2 * w.n;
  float acc[kTiles][4];
#pragma unroll
  for (int j = 0; j < kTiles; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int ch = w.c0; ch < w.c1; ++ch) {
    if (!__all_sync(0xffffffffu, mbar_wait(&c.full[pos.stage], pos.phase, &c.abort, a.status, a.limit_ns))) return false;
    const uint8_t* slot = ring.base + (size_t)pos.stage * ring.slot;
    const int have = row_bytes - ch * kChunk;
    const uint8_t* pw = slot + (warp >> 1) * kRows * kBox + (warp & 1) * 256 + r * kBox + q * 16;
    const uint8_t* pt = slot + kWeightBytes + warp * 256 + q * 16;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int off = warp * 256 + u * 128;
      if (off < have) {
        uint4 lo[2], hi[2];
        lo[0] = *reinterpret_cast<const uint4*>(pw + u * 128 + (odd ? 64 : 0));
        lo[1] = *reinterpret_cast<const uint4*>(pw + u * 128 + (odd ? 0 : 64));
        hi[0] = *reinterpret_cast<const uint4*>(pw + u * 128 + 8 * kBox + (odd ? 64 : 0));
        hi[1] = *reinterpret_cast<const uint4*>(pw + u * 128 + 8 * kBox + (odd ? 0 : 64));
        const uint4 a0 = odd ? lo[1] : lo[0], a1 = odd ? lo[0] : lo[1];
        const uint4 b0 = odd ? hi[1] : hi[0], b1 = odd ? hi[0] : hi[1];
        // the weights end in zeros; the token rows in what was there before
        const bool in0 = off + q * 16 < have, in1 = off + 64 + q * 16 < have;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          if (j * 8 < cols) {
            const uint8_t* p = pt + u * 128 + min(j * 8 + r, cols - 1) * kTokPitch;
            const uint4 t0 = in0 ? *reinterpret_cast<const uint4*>(p) : zero;
            const uint4 t1 = in1 ? *reinterpret_cast<const uint4*>(p + 64) : zero;
            mma_block(acc[j], a0, b0, t0);
            mma_block(acc[j], a1, b1, t1);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.empty[pos.stage]);
    pos.next(ring.stages);
  }
  float* mine = red + warp * kRows * kRedLd;
#pragma unroll
  for (int j = 0; j < kTiles; ++j) {
    if (j * 8 < cols) {
      if (kUp) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(r + (i >> 1) * 8) * kRedLd + j * 8 + q * 2 + (i & 1)] = acc[j][i];
      } else {  // columns 2t and 2t + 1: the two terms of token t
        mine[r * kRedLd + j * 4 + q] = acc[j][0] + acc[j][1];
        mine[(r + 8) * kRedLd + j * 4 + q] = acc[j][2] + acc[j][3];
      }
    }
  }
  return true;
}

// fp32: warp w takes rows 4 (w / 2) .. + 3 and half of the stage's columns.
template <bool kUp>
__device__ bool multiply(const Item& w, const FewArgs& a, Ctrl& c, const Ring& ring, int row_bytes, Pos& pos,
                         float* red, const float*) {
  const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
  const int half = warp & 1, r0 = (warp >> 1) * 4;
  float acc[4][16];  // [four tokens][row * 4 + token]
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[g][i] = 0.f;
  for (int ch = w.c0; ch < w.c1; ++ch) {
    if (!__all_sync(0xffffffffu, mbar_wait(&c.full[pos.stage], pos.phase, &c.abort, a.status, a.limit_ns))) return false;
    const uint8_t* slot = ring.base + (size_t)pos.stage * ring.slot;
    const int have = row_bytes - ch * kChunk;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int box = half * 2 + u, off = box * kBox + lane * 16;
      if (off < have) {
        const uint8_t* pw = slot + box * kRows * kBox + r0 * kBox + lane * 16;
        const uint8_t* pt = slot + kWeightBytes + off;
        float4 wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wv[i] = *reinterpret_cast<const float4*>(pw + i * kBox);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g * 4 < w.n) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const float4 b = *reinterpret_cast<const float4*>(pt + (g * 4 + t) * kTokPitch);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float& s = acc[g][i * 4 + t];
                s = fmaf(wv[i].w, b.w, fmaf(wv[i].z, b.z, fmaf(wv[i].y, b.y, fmaf(wv[i].x, b.x, s))));
              }
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.empty[pos.stage]);
    pos.next(ring.stages);
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (g * 4 < w.n) {
      const float s = reduce_many(acc[g]);
      if ((lane & 1) == 0) red[(half * kRows + r0 + (lane >> 3)) * kRedLd + g * 4 + ((lane >> 1) & 3)] = s;
    }
  }
  return true;
}

__device__ __forceinline__ float silu_of(float z, const __nv_bfloat16*) { return silu_f32(z); }
__device__ __forceinline__ float silu_of(float z, const float*) { return z / (1.f + expf(-z)); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
// A hidden value into its row, and what the row leaves of it into the next.
__device__ __forceinline__ void put_hidden(uint8_t* p, float v, const __nv_bfloat16*) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  *reinterpret_cast<__nv_bfloat16*>(p) = hi;
  *reinterpret_cast<__nv_bfloat16*>(p + kTokPitch) = __float2bfloat16_rn(v - __bfloat162float(hi));
}
__device__ __forceinline__ void put_hidden(uint8_t* p, float v, const float*) { *reinterpret_cast<float*>(p) = v; }

template <typename X>
__device__ __forceinline__ float sum_parts(const float* red, int row, int n) {
  float s = 0.f;
#pragma unroll
  for (int p = 0; p < Traits<X>::kParts; ++p) s += red[(p * kRows + row) * kRedLd + n];
  return s;
}

template <typename X, bool kUp>
__device__ void consume(const FewArgs& a, Ctrl& c, const Ring& ring, float* red2) {
  const Work<X, kUp> work(a, c.plan);
  const int hid_chunks = (a.I * (int)sizeof(X) + kChunk - 1) / kChunk;
  const int K = kUp ? a.d : a.I;
  const int tid = threadIdx.x - 64;
  const int R = a.T * a.k;
  Pos pos;
  int buf = 0;
  for (int i = blockIdx.x; i < work.total; i += gridDim.x) {
    const Item w = work.item(i, c.plan);
    float* red = red2 + buf * red_floats<X>();
    buf ^= 1;
    const bool ok = multiply<kUp>(w, a, c, ring, K * (int)sizeof(X), pos, red, static_cast<const X*>(nullptr));
    if (!math_sync_all(ok)) break;
    if (kUp) {
      const int u = tid & 7, n = tid >> 3, unit = w.blk * 8 + u;
      if (n < w.n && unit < a.I) {
        const float g = sum_parts<X>(red, u, n), up = sum_parts<X>(red, 8 + u, n);
        const int ch = unit * (int)sizeof(X) / kChunk, at = unit * (int)sizeof(X) % kChunk;
        put_hidden(static_cast<uint8_t*>(a.h) + hidden_at<X>(w.first, w.n, hid_chunks, ch, n * Traits<X>::kHid) + at,
                   silu_of(g, static_cast<const X*>(nullptr)) * up, static_cast<const X*>(nullptr));
      }
    } else {
      const int r = tid & 15, n = tid >> 4, col = w.blk * kRows + r;
      if (n < w.n && col < a.d)
        a.y[((size_t)w.part * R + c.plan.tj[w.first + n]) * a.d + col] = c.plan.gate[w.first + n] * sum_parts<X>(red, r, n);
      __threadfence();
      math_sync();
      if (tid == 0) {
        const int before = atomicAdd(&a.done[w.blk], 1);
        c.last = before == c.plan.n_act * work.split - 1;
      }
      math_sync();
      if (c.last) {
        __threadfence();
        if (n < a.T && col < a.d) {
          float s = 0.f;
          for (int j = 0; j < a.k; ++j)
            for (int q = 0; q < work.split; ++q) s += __ldcg(&a.y[((size_t)q * R + n * a.k + j) * a.d + col]);
          put(static_cast<X*>(a.out) + (size_t)n * a.d + col, s);
        }
      }
    }
  }
}

template <typename X, bool kUp>
__device__ void stream(const FewMaps& maps, const FewArgs& a, Ctrl& c, uint8_t* smem_ring, float* red) {
  const Ring ring = ring_of<X, kUp>(smem_ring, c.plan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Pos pos;
  int issued = 0;
  if (warp == 0) {
    if (lane == 0 && (!produce_weights<X, kUp>(maps, a, c, ring, pos, issued) || c.abort))
      drain(a, c, ring, pos, issued);
    __syncwarp();
  } else if (warp == 1) {
    const bool ok = produce_tokens<X, kUp>(a, c, ring, pos, issued);
    if (lane == 0 && (!ok || c.abort)) drain(a, c, ring, pos, issued);
    __syncwarp();
  } else {
    consume<X, kUp>(a, c, ring, red);
  }
}

__device__ __forceinline__ void init_ctrl(Ctrl& c) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&c.full[s], 2);
      mbar_init(&c.empty[s], kMathWarps);
    }
    c.abort = 0;
    fence_mbarrier_init();
  }
}

template <typename X>
__device__ __forceinline__ void carve(uint8_t* smem, Ctrl** c, float** red, uint8_t** ring) {
  *c = reinterpret_cast<Ctrl*>(smem);
  *red = reinterpret_cast<float*>(smem + (sizeof(Ctrl) + 127) / 128 * 128);
  *ring = reinterpret_cast<uint8_t*>(*red + 2 * red_floats<X>());
}

template <typename X>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1) few_up_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  Ctrl* c;
  float* red;
  uint8_t* ring;
  carve<X>(smem, &c, &red, &ring);
  init_ctrl(*c);
  float* part = reinterpret_cast<float*>(ring);                     // [kCluster][T][E]
  float* scratch = part + (size_t)kCluster * a.T * a.E;             // [kWarps][kPassE][16]
  const int rank = (int)cluster_ctarank();
  cluster_sync();  // the peers' shared memory exists
  pdl_wait();
  pdl_trigger();
  // this CTA's columns
  const int unit = 32, units = (a.d + unit - 1) / unit;
  const int c0 = min(a.d, rank * units / kCluster * unit), c1 = min(a.d, (rank + 1) * units / kCluster * unit);
  logits_part(static_cast<const X*>(a.x), static_cast<const X*>(a.wr), a.T, a.d, a.E, c0, c1, scratch, part, rank);
  cluster_sync();  // all parts are here, and no peer writes here any more
  const bool first = blockIdx.x == 0;
  choose<X>(a, part, *c, first);
  __syncthreads();
  make_plan(c->plan, c->idx, c->gate, a.T, a.E, a.k);
  if (first) {
    statistics(a, part, *c);
    for (int i = threadIdx.x; i < (a.d + kRows - 1) / kRows; i += kThreads) a.done[i] = 0;
  }
  fence_async();  // the ring's memory was written above, and is next by the copies
  __syncthreads();
  stream<X, true>(maps, a, *c, ring, red);
}

template <typename X>
__global__ void __launch_bounds__(kThreads, 1) few_down_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  Ctrl* c;
  float* red;
  uint8_t* ring;
  carve<X>(smem, &c, &red, &ring);
  init_ctrl(*c);
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x;
  if (i < a.T * a.k) {
    int e = a.idx[i];
    if (e < 0 || e >= a.E) {  // few_up wrote them: something else has written there since
      atomicOr(a.status, MOE_DEV_INTERNAL);
      e = 0;
    }
    c->idx[i] = e;
    c->gate[i] = a.gate[i];
  }
  __syncthreads();
  make_plan(c->plan, c->idx, c->gate, a.T, a.E, a.k);
  fence_async();  // few_up's hidden rows are read by the copies
  stream<X, false>(maps, a, *c, ring, red);
}

// What a launch needs to know of a device, found once.
struct Device {
  int clusters = 0, sms = 0;
};

template <typename X>
cudaError_t device_info(Device* out) {
  static std::atomic<uint64_t> cache[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const uint64_t have = cache[dev].load(std::memory_order_acquire);
  if (have) {
    out->clusters = (int)(have >> 32);
    out->sms = (int)(have & 0xffffffffu);
    return cudaSuccess;
  }
  err = cudaFuncSetAttribute(few_up_kernel<X>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTotal);
  if (err != cudaSuccess) return err;
  err = cudaFuncSetAttribute(few_down_kernel<X>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTotal);
  if (err != cudaSuccess) return err;
  err = cudaDeviceGetAttribute(&out->sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemTotal;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  err = cudaOccupancyMaxActiveClusters(&out->clusters, few_up_kernel<X>, &cfg);
  if (err != cudaSuccess) return err;
  if (out->clusters <= 0 || out->sms <= 0) return cudaErrorInvalidConfiguration;
  cache[dev].store(((uint64_t)out->clusters << 32) | (uint32_t)out->sms, std::memory_order_release);
  return cudaSuccess;
}

template <typename X>
cudaError_t launch(const FewMaps& m, const FewArgs& a, cudaStream_t stream) {
  // the routing's scratch lies where the ring is, and every ring has two stages
  constexpr int kRing = kSmemTotal - fixed_bytes<X>();
  static_assert(4 * (kCluster * kFewTokens * kMaxExperts + kWarps * kPassE * kFewTokens) <= kRing, "routing scratch");
  static_assert(2 * (kWeightBytes + Traits<X>::kHid * kFewTokens * kTokPitch + 128) <= kRing, "ring");
  Device dev;
  cudaError_t err = device_info<X>(&dev);
  if (err != cudaSuccess) return err;
  err = launch_pdl(few_up_kernel<X>, dim3(dev.clusters * kCluster), dim3(kThreads), kSmemTotal, stream, m, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(few_down_kernel<X>, dim3(dev.sms), dim3(kThreads), kSmemTotal, stream, m, a);
}

}  // namespace

FewWorkspace few_layout(int T, int d, int k, int I, moe_dtype dtype) {
  const size_t R = (size_t)T * k, el = dtype == MOE_BF16 ? 2 : 4;
  FewWorkspace w;
  // room for finer parts where there are few rows: that is where the blocks
  // of 16 columns do not go evenly into the SMs
  w.split = R > 0 && 256 / R < kFewMaxSplit ? (int)(256 / R) : kFewMaxSplit;
  size_t o = 0;
  w.done = o; o = align256(o + 4 * (size_t)((d + kRows - 1) / kRows));
  const size_t chunks = (el * (size_t)I + kChunk - 1) / kChunk;
  w.h = o;    o = align256(o + R * chunks * kTokPitch * (dtype == MOE_BF16 ? Traits<__nv_bfloat16>::kHid : 1));
  w.y = o;    o = align256(o + 4 * (size_t)w.split * R * (size_t)d);
  w.total = o;
  return w;
}

cudaError_t launch_few(moe_dtype dtype, const FewMaps& m, const FewArgs& a, cudaStream_t stream) {
  return dtype == MOE_BF16 ? launch<__nv_bfloat16>(m, a, stream) : launch<float>(m, a, stream);
}

}  // namespace moe
