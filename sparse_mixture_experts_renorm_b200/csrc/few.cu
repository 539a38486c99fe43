// few.cu — the whole layer for at most 16 tokens in two kernels.
//
//   few_up:   p = softmax(x W_r^T + b), the k best experts and their gates;
//             H[row] = SiLU(W_g[e] x_t) * (W_u[e] x_t) for every choice (t, e)
//   few_down: out[t] = sum_j gate[t, j] * W_d[e_j] H[row(t, j)]
//
// Bound by the weights: every chosen expert's 3 d I weights are read once, and
// each takes part in at most 16 products. So both kernels are streams: one
// thread fills a ring in shared memory with stages of 16 weight rows x 1 KB
// (tile loads of 512 bytes x 8 or 16 rows; one bulk copy a row took twice the
// time, as each is issued by itself), the same columns of the rows that
// multiply them come beside, and eight warps consume a stage on mma.sync (bf16)
// or FFMA (fp32). tcgen05 has nothing to give here: 16 rows of weights against
// 8 tokens are one m16n8k16 step, the rate of the loads is a tenth of what it
// takes, and its operand tiles would hold 128 rows of one expert where 16 keep
// the SMs evenly loaded.
//
// Routing has to be known before the first weight can be asked for, and a
// kernel of its own would cost a launch: instead each cluster of few_up
// computes all of it, its CTAs a part of the d columns each, exchanged
// through distributed shared memory. Every cluster adds in the same order,
// so all come to the same choices; few_down takes them from the workspace.
//
// A down product's rows of different experts belong to the same output: each
// finished part is written to y, and the last of a block of 16 columns to
// finish adds them up, in a fixed order whatever the order of arrival.
//
// Measured (bf16, in a graph, us and bytes that it cannot do without over the
// time): 16 tokens of the Mixtral-shaped layer (d 4096, I 14336, 8 experts, k 2)
// 424 to 437 us between boxes, 6.4 to 6.6 TB/s (called one by one 438 to 470 us);
// 5 tokens of the fine-grained one (d 2048, I 1408, 64 experts, k 6) 76 us, 5.7
// TB/s; one token of the small one (d 1024, I 2816, 8 experts, k 2) 20.5 us, 1.7
// TB/s. What is left there: some 8 us from the launch to the first
// weight (3.6 us of logits, 2.5 us of choosing and 1.3 us of grouping for 64
// experts; half of that for 8), 4 us between the kernels, and the last items'
// and joins' tail.
#include <atomic>
#include <math.h>
#include <stddef.h>

#include "few_internal.h"
#include "pair.cuh"

namespace moe {
namespace {

constexpr int kMathWarps = 8;
constexpr int kMath = 32 * kMathWarps;
constexpr int kGroupWarps = 2 + kMathWarps;  // a group: 0: weights, 1: token rows or joins, 2..9: products
constexpr int kMaxGroups = 2;
constexpr int kRows = 16;                // weight rows of a stage
constexpr int kBox = 512;                // bytes of a row in one tile load
constexpr int kBoxes = 2;                // tile loads side by side in a stage: 16 KB of weights; 32 KB leave a ring
                                         // of too few stages for two groups
constexpr int kChunk = kBox * kBoxes;    // bytes of a row in a stage
constexpr int kWeightBytes = kRows * kChunk;
constexpr int kTokPitch = kFewTokPitch;  // bytes between token rows: two rows of a quarter-warp's load on different banks
static_assert(kTokPitch == kChunk + 64, "pitch");
constexpr int kMaxStages = 10;           // of a group
constexpr int kAhead = 5;                // stages of a block brought to L2 ahead of time: 12 MB on 148 SMs
constexpr int kJoinQueue = 256;          // items that the joins may lie behind the products
constexpr int kMaxRows = kFewTokens * kMaxTopK;
constexpr int kCluster = 4;              // CTAs that share one routing
constexpr int kPassE = 64;               // experts whose logits a warp holds at a time
constexpr int kPassLd = kPassE + 4;      // 2 kPassLd % 32 == 8: an mma.sync result's lanes on different banks
constexpr int kSmemTotal = 227 * 1024;

struct Plan {
  int n_act;                        // experts with tokens
  int most;                         // tokens of the one with most
  int down_split;                   // parts of a down product's columns
  int expert[kMaxRows];             // ascending
  int base[kMaxRows + 1];           // first row of each
  int tj[kMaxRows];                 // t * k + j of a row
  int tok[kMaxRows];                // and t
  float gate[kMaxRows];
  // what follows is not for few_down
  uint32_t mask[kMaxExperts];       // tokens of an expert
  int slot[kMaxExperts];
};

constexpr int kPlanWords = (int)(offsetof(Plan, mask) / 4);
static_assert(kPlanWords <= kFewPlanWords && kFewPlanAt + kFewPlanWords <= kFewUpAt, "the workspace's head");

// One group's barriers and lists.
struct Group {
  uint64_t full[kMaxStages];   // the producers' bytes
  uint64_t empty[kMaxStages];  // the math warps
  int4 item[kMaxStages];       // few_down: a stage's item: active expert + 256 x part (-1: there are no more),
                               // block, chunks from and to
  int blk[kJoinQueue];         // few_down: block of output columns of each finished item
  volatile int finished;       // items whose parts are written; negative: ~items, and there are no more
  volatile int joined;         // items that have been counted
};

struct Ctrl {
  Group group[kMaxGroups];
  volatile int abort;
  int idx[kMaxRows];
  float gate[kMaxRows];
  float bias[kMaxExperts];
  float red[kMaxGroups * kGroupWarps];
  Plan plan;
};

// kParts: partial sums of an item (bf16: every warp has its own columns; fp32:
// two halves of the columns, four groups of rows). kHid: rows that a hidden
// row is stored as. bf16 keeps it in two terms, hi + lo, whose sum is off by
// 2^-17: rounded to one, it would double the error that the output's own
// rounding makes, and the second term costs only shared memory and issue slots
// (both are columns of the same mma.sync while an expert has few tokens).
// kGroups: independent pipelines of a block, with half of the ring each: while
// one adds up its partial sums, the other multiplies. The fp32 products hold
// too many sums in registers for a second one.
template <typename X>
struct Traits;
template <>
struct Traits<__nv_bfloat16> {
  static constexpr int kParts = kMathWarps, kHid = 2, kGroups = 2;
};
template <>
struct Traits<float> {
  static constexpr int kParts = 2, kHid = 1, kGroups = 1;
};
constexpr int kRedLd = kFewTokens + 1;
template <typename X>
constexpr int red_floats() { return Traits<X>::kParts * kRows * kRedLd; }
template <typename X>
constexpr int threads() { return Traits<X>::kGroups * kGroupWarps * 32; }
template <typename X>
constexpr int fixed_bytes() {
  return (int)((sizeof(Ctrl) + 127) / 128 * 128 + 2 * Traits<X>::kGroups * red_floats<X>() * 4);
}

// The rings' shape follows from the most tokens that an expert got: two groups
// where each still has three stages.
struct Ring {
  uint8_t* base;
  int slot, stages, groups;
};
template <typename X, bool kUp>
__device__ __forceinline__ int ring_slot(int most) {
  int rows = kUp ? most : most * Traits<X>::kHid;
  if (sizeof(X) == 4) rows = (rows + 3) & ~3;  // fp32 multiplies four token rows at a time
  return (kWeightBytes + rows * kTokPitch + 127) & ~127;
}
template <typename X>
__device__ __forceinline__ int ring_groups(int slot) {
  return Traits<X>::kGroups == 2 && 6 * slot <= kSmemTotal - fixed_bytes<X>() ? 2 : 1;
}
template <typename X, bool kUp>
__device__ __forceinline__ Ring ring_of(uint8_t* base, const Plan& p, int group) {
  Ring r;
  r.slot = ring_slot<X, kUp>(p.most);
  r.groups = ring_groups<X>(r.slot);
  r.stages = min(kMaxStages, (kSmemTotal - fixed_bytes<X>()) / (r.groups * r.slot));
  r.base = base + (size_t)group * r.stages * r.slot;
  return r;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
// A barrier of a group's math warps, and whether any thread said no: all
// leave together.
__device__ __forceinline__ bool math_sync_all(int group, bool ok) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.eq.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %3, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)ok), "n"(kMath), "r"(1 + group)
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
template <typename X>
__device__ void make_plan(const FewArgs& a, Plan& p, const int* idx, const float* gate) {
  const int E = a.E, k = a.k, R = a.T * k;
  for (int e = threadIdx.x; e < E; e += blockDim.x) p.mask[e] = 0;
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
    // lane q - 1: the busiest group's work if columns are split in q parts. An
    // item's own overhead (its sums, its join) is some two chunks; a finer
    // split has to gain 3 %
    const int chunks = (a.I * (int)sizeof(X) + kChunk - 1) / kChunk, q = lane + 1;
    const int units = a.down_blocks * ring_groups<X>(ring_slot<X, false>(most));
    float t = 3.0e38f;
    if (q <= min(a.split, chunks))
      t = (float)((act * ((a.d + kRows - 1) / kRows) * q + units - 1) / units) * (float)((chunks + q - 1) / q + 2);
    float least = t;
#pragma unroll
    for (int o = 16; o; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    const int split = __ffs(__ballot_sync(0xffffffffu, t <= 1.03f * least));
    if (lane == 0) {
      p.n_act = act;
      p.most = most;
      p.base[act] = rows;
      p.down_split = split;
    }
  }
  __syncthreads();
  if (i < R) {
    const int e = idx[i], t = i / k;
    const int row = p.base[p.slot[e]] + __popc(p.mask[e] & ((1u << t) - 1u));
    p.tj[row] = i;
    p.tok[row] = t;
    p.gate[row] = gate[i];
  }
  __syncthreads();
}

// ---------------------------------------------------------------- routing --

// Partial logits of all T tokens and E experts over columns [c0, c1): warp
// sums in scratch [kWarps][T][kPassLd], added up in warp order into every
// cluster CTA's part[rank][T][E]. bias [E] is added to one CTA's.
template <typename X>
__device__ void logits_part(const X* __restrict__ x, const X* __restrict__ wr, int T, int d, int E, int c0, int c1,
                            const float* bias, float* scratch, float* part, int rank) {
  constexpr int kWarps = threads<X>() / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < E; e0 += kPassE) {
    const int ne = min(kPassE, E - e0);
    float* mine = scratch + warp * kFewTokens * kPassLd;
    int parts = kWarps;  // partial sums of a logit in this CTA
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
#pragma unroll 1
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
            if (m * 16 < ne) mine[t * kPassLd + e] = acc[m][n][i];
          }
    } else {
      // blocks of 4 experts x 4 tokens over the warps; where there are fewer
      // than warps, the columns too
      const int pe = (ne + 3) / 4, pairs = pe * ((T + 3) / 4);
      parts = max(1, kWarps / pairs);
      const int slice = parts > 1 ? warp / pairs : 0;
      mine = scratch + slice * kFewTokens * kPassLd;
      for (int p = parts > 1 ? (slice < parts ? warp % pairs : pairs) : warp; p < pairs; p += parts > 1 ? pairs : kWarps) {
        const int t = p / pe * 4, e = p % pe * 4;
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
#pragma unroll 2
        for (int col = c0 + slice * 128 + lane * 4; col < c1; col += parts * 128) {
          float4 a[4], b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = __ldg(reinterpret_cast<const float4*>(wr + (size_t)(e0 + min(e + i, ne - 1)) * d + col));
            b[i] = __ldg(reinterpret_cast<const float4*>(x + (size_t)min(t + i, T - 1) * d + col));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float4 &q = a[i >> 2], &r = b[i & 3];
            v[i] = fmaf(q.w, r.w, fmaf(q.z, r.z, fmaf(q.y, r.y, fmaf(q.x, r.x, v[i]))));
          }
        }
        const float s = reduce_many(v);
        if ((lane & 1) == 0) mine[(t + ((lane >> 1) & 3)) * kPassLd + e + (lane >> 3)] = s;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ne * T; i += blockDim.x) {
      const int t = i / ne, e = i - t * ne;
      float s = rank == 0 ? bias[e0 + e] : 0.f;
#pragma unroll 4
      for (int w = 0; w < parts; ++w) s += scratch[(w * kFewTokens + t) * kPassLd + e];
      float* dst = part + ((size_t)rank * T + t) * E + e0 + e;
      for (int c = 0; c < kCluster; ++c) store_cluster(map_to_cta(dst, c), s);
    }
    __syncthreads();
  }
}

// A float's bits in an order that integers have: -inf < ... < inf, NaN below
// them all, 0 for none.
__device__ __forceinline__ uint32_t rank_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return v != v ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Softmax, the k best (ties to the lower index) and their gates. part
// [kCluster][T][E]; the logits replace part[0], and then the probabilities if
// the statistic is wanted. An expert's place is the number of those before it
// in its token's row, counted by a thread per (token, expert): k rounds of an
// arg-max by a warp per token took 2.0 us for 64 experts and k = 6, this 0.6.
// Experts rank by their logits, as their exact probabilities do; NaN ranks
// lowest, so that every token still gets k different experts. keys [T][E
// rounded to 4].
__device__ void choose(const FewArgs& a, float* part, uint32_t* keys, Ctrl& c, bool write) {
  const int T = a.T, E = a.E, k = a.k, ld = (E + 3) & ~3;
  for (int i = threadIdx.x; i < T * ld; i += blockDim.x) {
    const int t = i / ld, e = i - t * ld;
    uint32_t key = 0;
    if (e < E) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < kCluster; ++q) s += part[((size_t)q * T + t) * E + e];
      part[(size_t)t * E + e] = s;
      if (write && !isfinite(s)) atomicOr(a.status, MOE_DEV_NONFINITE);
      key = rank_key(s);
    }
    keys[i] = key;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * E; i += blockDim.x) {
    const int t = i / E, e = i - t * E;
    const uint32_t mine = keys[t * ld + e];
    const uint4* row = reinterpret_cast<const uint4*>(keys + t * ld);
    int place = 0;
    for (int j = 0; j < ld; j += 4) {
      const uint4 v = row[j >> 2];
      place += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
      place += (v.x == mine && j < e) + (v.y == mine && j + 1 < e) + (v.z == mine && j + 2 < e) +
               (v.w == mine && j + 3 < e);
    }
    if (place < k) c.idx[t * k + place] = e;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int t = warp; t < T; t += blockDim.x / 32) {
    float* row = part + (size_t)t * E;
    const int mine = lane < k ? c.idx[t * k + lane] : 0;
    const float l = key_value(keys[t * ld + mine]);
    const float m = __shfl_sync(0xffffffffu, l, 0);
    float sum = 0.f;
    if (!a.renorm || (write && a.aux)) {
      for (int e = lane; e < E; e += 32) sum += expf(row[e] - m);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    // renormalised, the softmax's own sum cancels
    const float p = lane < k ? expf(l - m) : 0.f;
    float total = p;
#pragma unroll
    for (int o = 4; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane < k) {
      const float g = !a.renorm ? p / sum : total > 0.f ? p / total : 1.f / (float)k;
      c.gate[t * k + lane] = g;
      if (write) {
        a.idx[(size_t)t * k + lane] = mine;
        a.gate[(size_t)t * k + lane] = g;
      }
    }
    if (write && a.aux)
      for (int e = lane; e < E; e += 32) row[e] = expf(row[e] - m) / sum;
  }
}

// counts and the load-balancing statistic, by one block; prob [T][E].
__device__ void statistics(const FewArgs& a, const float* prob, Ctrl& c) {
  for (int e = threadIdx.x; e < a.E; e += blockDim.x)
    if (a.counts) a.counts[e] = __popc(c.plan.mask[e]);
  if (!a.aux) return;
  float s = 0.f;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
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
    for (int w = 0; w < (int)blockDim.x / 32; ++w) sum += c.red[w];
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
  __device__ __forceinline__ Work(const FewArgs& a, int n_act, int parts) {
    chunks = ((kUp ? a.d : a.I) * (int)sizeof(X) + kChunk - 1) / kChunk;
    n_blk = kUp ? (a.I + 7) / 8 : (a.d + kRows - 1) / kRows;
    split = parts;
    total = n_act * n_blk * split;
  }
  __device__ __forceinline__ Item item(int i) const {
    Item w;
    const int q = i / split;
    w.part = i - q * split;
    w.s = q / n_blk;
    w.blk = q - w.s * n_blk;
    w.c0 = w.part * chunks / split;
    w.c1 = (w.part + 1) * chunks / split;
    return w;
  }
  __device__ __forceinline__ Item item(int i, const Plan& p) const {
    Item w = item(i);
    w.first = p.base[w.s];
    w.n = p.base[w.s + 1] - w.first;
    return w;
  }
};

// few_up's items of one group, one after the other without divisions: `step`
// items further each time.
struct Walk {
  int s, blk, step_s, step_blk, n_blk;
  __device__ __forceinline__ Walk(int first, int step, int blocks) : n_blk(blocks) {
    s = first / blocks, blk = first - s * blocks;
    step_s = step / blocks, step_blk = step - step_s * blocks;
  }
  __device__ __forceinline__ void next() {
    s += step_s;
    blk += step_blk;
    if (blk >= n_blk) blk -= n_blk, ++s;
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

// Asks for the weights of block `block`'s first stages to be brought to L2.
template <typename X, bool kUp>
__device__ void prefetch_weights(const FewMaps& maps, const FewArgs& a, const int* expert, int n_act, int split,
                                 int block, int grid) {
  const Work<X, kUp> work(a, n_act, split);
  const int row_bytes = (kUp ? a.d : a.I) * (int)sizeof(X);
  int n = 0;
  for (int i = block; i < work.total; i += grid) {
    const Item w = work.item(i);
    const int e = expert ? expert[w.s] : w.s;
    const int row = kUp ? e * a.I + w.blk * 8 : e * a.d + w.blk * kRows;
    for (int ch = w.c0; ch < w.c1; ++ch) {
      if (n++ == kAhead) return;
      for (int at = ch * kChunk; at < min(row_bytes, (ch + 1) * kChunk); at += kBox) {
        const int col = at / (int)sizeof(X);
        if (kUp) {
          tma_prefetch_2d(&maps.wg, col, row);
          tma_prefetch_2d(&maps.wu, col, row);
        } else {
          tma_prefetch_2d(&maps.wd, col, row);
        }
      }
    }
  }
}

// Asks for a stage of weights. Rows past the last block's are read from the
// next expert, or as zeros, and go into sums that nobody takes. Returns bytes.
template <typename X, bool kUp>
__device__ __forceinline__ uint32_t weight_bytes(int chunk, int row_bytes) {
  return (uint32_t)(min(kBoxes, (row_bytes - chunk * kChunk + kBox - 1) / kBox) * kRows * kBox);
}
template <typename X, bool kUp>
__device__ __forceinline__ void load_weights(const FewMaps& maps, uint8_t* dst, uint64_t* bar, int chunk, int row,
                                             int row_bytes) {
#pragma unroll
  for (int b = 0; b < kBoxes; ++b) {
    const int at = chunk * kChunk + b * kBox, col = at / (int)sizeof(X);
    uint8_t* to = dst + b * kRows * kBox;
    if (at < row_bytes) {
      if (kUp) {  // rows 0..7: gate rows of 8 hidden units, 8..15: their up rows
        tma_load_2d(to, &maps.wg, bar, col, row);
        tma_load_2d(to + 8 * kBox, &maps.wu, bar, col, row);
      } else {
        tma_load_2d(to, &maps.wd, bar, col, row);
      }
    }
  }
}

// few_up's weights: one lane. Items go round the groups of all blocks.
template <typename X>
__device__ bool produce_up_weights(const FewMaps& maps, const FewArgs& a, Ctrl& c, Group& g, const Ring& ring, int first,
                                   int step, Pos& pos, int& issued) {
  const Work<X, true> work(a, c.plan.n_act, 1);
  const int row_bytes = a.d * (int)sizeof(X);
  for (Walk w(first, step, work.n_blk); w.s < c.plan.n_act; w.next()) {
    const int row = c.plan.expert[w.s] * a.I + w.blk * 8;
    for (int ch = 0; ch < work.chunks; ++ch) {
      if (!mbar_wait(&g.empty[pos.stage], pos.phase ^ 1u, &c.abort, a.status, a.limit_ns)) return false;
      mbar_arrive_expect_tx(&g.full[pos.stage], weight_bytes<X, true>(ch, row_bytes));
      load_weights<X, true>(maps, ring.base + (size_t)pos.stage * ring.slot, &g.full[pos.stage], ch, row, row_bytes);
      ++issued;
      pos.next(ring.stages);
    }
  }
  return true;
}

// few_up's token rows: one warp, lane l copies row l.
template <typename X>
__device__ bool produce_up_tokens(const FewArgs& a, Ctrl& c, Group& g, const Ring& ring, int first, int step, Pos& pos,
                                  int& issued) {
  const int lane = threadIdx.x & 31;
  const Work<X, true> work(a, c.plan.n_act, 1);
  const int row_bytes = a.d * (int)sizeof(X);
  for (Walk w(first, step, work.n_blk); w.s < c.plan.n_act; w.next()) {
    const int n0 = c.plan.base[w.s], n = c.plan.base[w.s + 1] - n0;
    const uint8_t* src = nullptr;
    if (lane < n) src = static_cast<const uint8_t*>(a.x) + (size_t)c.plan.tok[n0 + lane] * row_bytes;
    for (int ch = 0; ch < work.chunks; ++ch) {
      const uint32_t bytes = (uint32_t)min(kChunk, row_bytes - ch * kChunk);
      bool free = true;
      if (lane == 0) {
        free = mbar_wait(&g.empty[pos.stage], pos.phase ^ 1u, &c.abort, a.status, a.limit_ns);
        if (free) mbar_arrive_expect_tx(&g.full[pos.stage], n * bytes);
      }
      if (!__shfl_sync(0xffffffffu, (int)free, 0)) return false;
      if (src)
        bulk_load(ring.base + (size_t)pos.stage * ring.slot + kWeightBytes + lane * kTokPitch, src + (size_t)ch * kChunk,
                  bytes, &g.full[pos.stage]);
      ++issued;
      pos.next(ring.stages);
    }
  }
  return true;
}

// few_down's weights and hidden rows: one lane. The items that fill a group's
// ring at the start are its own; then it takes the next that nobody has (SMs
// reach the memory at rates some 10 % apart), asked for an item ahead.
template <typename X>
__device__ bool produce_down(const FewMaps& maps, const FewArgs& a, Ctrl& c, Group& g, const Ring& ring, int first,
                             int step, Pos& pos, int& issued) {
  const Work<X, false> work(a, c.plan.n_act, c.plan.down_split);
  const int row_bytes = a.I * (int)sizeof(X);
  const int own = 1 + ring.stages * work.split / work.chunks;
  int i = first;
  for (int n = 1;; ++n) {
    const bool more = i < work.total;
    int next = i + step;
    if (n >= own && more) next = own * step + atomicAdd(a.next, 1);
    Item w = {};
    if (more) w = work.item(i, c.plan);
    for (int ch = w.c0; ch < (more ? w.c1 : w.c0 + 1); ++ch) {
      if (!mbar_wait(&g.empty[pos.stage], pos.phase ^ 1u, &c.abort, a.status, a.limit_ns)) return false;
      g.item[pos.stage] = make_int4(more ? w.s | w.part << 8 : -1, w.blk, w.c0, w.c1);
      const uint32_t bytes = (uint32_t)(w.n * Traits<X>::kHid * kTokPitch);
      if (more) {
        mbar_arrive_expect_tx(&g.full[pos.stage], weight_bytes<X, false>(ch, row_bytes) + bytes);
        uint8_t* dst = ring.base + (size_t)pos.stage * ring.slot;
        load_weights<X, false>(maps, dst, &g.full[pos.stage], ch, c.plan.expert[w.s] * a.d + w.blk * kRows, row_bytes);
        bulk_load(dst + kWeightBytes,
                  static_cast<const uint8_t*>(a.h) + hidden_at<X>(w.first, w.n, work.chunks, ch, 0), bytes,
                  &g.full[pos.stage]);
      } else {
        mbar_arrive(&g.full[pos.stage]);
      }
      ++issued;
      pos.next(ring.stages);
    }
    if (!more) return true;
    i = next;
  }
}

// A block that gives up still waits for the copies it has asked for.
__device__ void drain(const FewArgs& a, Group& g, const Ring& ring, Pos pos, int issued) {
  const int n = min(issued, ring.stages);
  for (int i = 0; i < n; ++i) {
    if (pos.stage == 0) pos.stage = ring.stages, pos.phase ^= 1u;
    --pos.stage;
    if (!mbar_wait(&g.full[pos.stage], pos.phase, nullptr, a.status, a.limit_ns)) return;
  }
}

// Sums of one item into red [parts][kRows][kRedLd]. False: a wait gave up.
//
// bf16: warp w takes bytes 128 w .. 128 w + 127 of the stage's rows. Rows of
// weights lie 512 bytes apart, so the two rows that a quarter-warp reads at
// once would fall on the same banks: odd rows take the two halves of the 128
// bytes in the other order. The halves have sums of their own, which keeps
// the chains of dependent products short.
template <bool kUp>
__device__ bool multiply(const Item& w, const FewArgs& a, Ctrl& c, Group& g, const Ring& ring, int warp, int row_bytes,
                         Pos& pos, float* red, const __nv_bfloat16*) {
  constexpr int kTiles = kUp ? 2 : 4;  // of 8 columns: a token each, or hi and lo of four
  const int lane = threadIdx.x & 31;
  const int r = lane >> 2, q = lane & 3;
  const bool odd = r & 1;
  const int cols = kUp ? w.n : 2 * w.n;
  float acc[2][kTiles][4];
#pragma unroll
  for (int j = 0; j < kTiles; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[0][j][i] = acc[1][j][i] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int wo = (warp >> 2) * kRows * kBox + (warp & 3) * 128 + r * kBox + q * 16;
  const int to = kWeightBytes + warp * 128 + q * 16;
  for (int ch = w.c0; ch < w.c1; ++ch) {
    if (!__all_sync(0xffffffffu, mbar_wait(&g.full[pos.stage], pos.phase, &c.abort, a.status, a.limit_ns))) return false;
    const uint8_t* slot = ring.base + (size_t)pos.stage * ring.slot;
    const int have = row_bytes - ch * kChunk, off = warp * 128;
    if (off < have) {
      const uint8_t* pw = slot + wo;
      const uint4 l0 = *reinterpret_cast<const uint4*>(pw + (odd ? 64 : 0));
      const uint4 l1 = *reinterpret_cast<const uint4*>(pw + (odd ? 0 : 64));
      const uint4 h0 = *reinterpret_cast<const uint4*>(pw + 8 * kBox + (odd ? 64 : 0));
      const uint4 h1 = *reinterpret_cast<const uint4*>(pw + 8 * kBox + (odd ? 0 : 64));
      const uint4 a0 = odd ? l1 : l0, a1 = odd ? l0 : l1;
      const uint4 b0 = odd ? h1 : h0, b1 = odd ? h0 : h1;
      // the weights end in zeros; the token rows in what was there before
      const bool in0 = off + q * 16 < have, in1 = off + 64 + q * 16 < have;
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        if (j * 8 < cols) {
          const uint8_t* p = slot + to + min(j * 8 + r, cols - 1) * kTokPitch;
          const uint4 t0 = in0 ? *reinterpret_cast<const uint4*>(p) : zero;
          const uint4 t1 = in1 ? *reinterpret_cast<const uint4*>(p + 64) : zero;
          mma_block(acc[0][j], a0, b0, t0);
          mma_block(acc[1][j], a1, b1, t1);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&g.empty[pos.stage]);
    pos.next(ring.stages);
  }
  float* mine = red + warp * kRows * kRedLd;
#pragma unroll
  for (int j = 0; j < kTiles; ++j) {
    if (j * 8 < cols) {
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = acc[0][j][i] + acc[1][j][i];
      if (kUp) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(r + (i >> 1) * 8) * kRedLd + j * 8 + q * 2 + (i & 1)] = s[i];
      } else {  // columns 2t and 2t + 1: the two terms of token t
        mine[r * kRedLd + j * 4 + q] = s[0] + s[1];
        mine[(r + 8) * kRedLd + j * 4 + q] = s[2] + s[3];
      }
    }
  }
  return true;
}

// fp32: warp w takes rows 4 (w / 2) .. + 3 and half of the stage's columns.
template <bool kUp>
__device__ bool multiply(const Item& w, const FewArgs& a, Ctrl& c, Group& g, const Ring& ring, int warp, int row_bytes,
                         Pos& pos, float* red, const float*) {
  const int lane = threadIdx.x & 31;
  const int half = warp & 1, r0 = (warp >> 1) * 4;
  float acc[4][16];  // [four tokens][row * 4 + token]
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[q][i] = 0.f;
  for (int ch = w.c0; ch < w.c1; ++ch) {
    if (!__all_sync(0xffffffffu, mbar_wait(&g.full[pos.stage], pos.phase, &c.abort, a.status, a.limit_ns))) return false;
    const uint8_t* slot = ring.base + (size_t)pos.stage * ring.slot;
    const int off = half * kBox + lane * 16;
    if (off < row_bytes - ch * kChunk) {
      const uint8_t* pw = slot + half * kRows * kBox + r0 * kBox + lane * 16;
      const uint8_t* pt = slot + kWeightBytes + off;
      float4 wv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wv[i] = *reinterpret_cast<const float4*>(pw + i * kBox);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q * 4 < w.n) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float4 b = *reinterpret_cast<const float4*>(pt + (q * 4 + t) * kTokPitch);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float& s = acc[q][i * 4 + t];
              s = fmaf(wv[i].w, b.w, fmaf(wv[i].z, b.z, fmaf(wv[i].y, b.y, fmaf(wv[i].x, b.x, s))));
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&g.empty[pos.stage]);
    pos.next(ring.stages);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q * 4 < w.n) {
      const float s = reduce_many(acc[q]);
      if ((lane & 1) == 0) red[(half * kRows + r0 + (lane >> 3)) * kRedLd + q * 4 + ((lane >> 1) & 3)] = s;
    }
  }
  return true;
}

__device__ __forceinline__ float silu_of(float z, const __nv_bfloat16*) { return silu_f32(z); }
__device__ __forceinline__ float silu_of(float z, const float*) { return z / (1.f + expf(-z)); }
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void put4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
// A hidden value into its row, and what the row leaves of it into the next.
// The first term is held to bf16's largest number, so that a value between that
// and fp32's largest keeps its rest (infinity minus infinity is none), and an
// infinite value or a NaN is the second term alone.
__device__ __forceinline__ void put_hidden(uint8_t* p, float v, const __nv_bfloat16*) {
  constexpr float kMost = 3.38953139e38f;  // (2 - 2^-7) 2^127
  const __nv_bfloat16 hi = __float2bfloat16_rn(fminf(fmaxf(v, -kMost), kMost));
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

// few_up's products.
template <typename X>
__device__ void consume_up(const FewArgs& a, Ctrl& c, Group& g, const Ring& ring, float* red2, int group, int first,
                           int step) {
  const Work<X, true> work(a, c.plan.n_act, 1);
  const int hid_chunks = (a.I * (int)sizeof(X) + kChunk - 1) / kChunk;
  const int tid = threadIdx.x - (group * kGroupWarps + 2) * 32;
  Pos pos;
  int buf = 0;
  for (Walk at(first, step, work.n_blk); at.s < c.plan.n_act; at.next()) {
    Item w;
    w.s = at.s, w.blk = at.blk, w.part = 0, w.c0 = 0, w.c1 = work.chunks;
    w.first = c.plan.base[w.s], w.n = c.plan.base[w.s + 1] - w.first;
    float* red = red2 + buf * red_floats<X>();
    buf ^= 1;
    const bool ok =
        multiply<true>(w, a, c, g, ring, tid >> 5, a.d * (int)sizeof(X), pos, red, static_cast<const X*>(nullptr));
    if (!math_sync_all(group, ok)) return;
    const int u = tid & 7, n = tid >> 3, unit = w.blk * 8 + u;
    if (n < w.n && unit < a.I) {
      const float gt = sum_parts<X>(red, u, n), up = sum_parts<X>(red, 8 + u, n);
      const int ch = unit * (int)sizeof(X) / kChunk, at = unit * (int)sizeof(X) % kChunk;
      put_hidden(static_cast<uint8_t*>(a.h) + hidden_at<X>(w.first, w.n, hid_chunks, ch, n * Traits<X>::kHid) + at,
                 silu_of(gt, static_cast<const X*>(nullptr)) * up, static_cast<const X*>(nullptr));
    }
  }
}

__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// Waits until `ready` says so, at most limit_ns; false: gave up.
template <typename F>
__device__ __forceinline__ bool poll(const FewArgs& a, Ctrl& c, F ready) {
  const uint64_t t0 = globaltimer_ns();
  while (!ready()) {
    __nanosleep(100);
    if (c.abort) return false;
    if (globaltimer_ns() - t0 > a.limit_ns) {
      c.abort = 1;
      atomicOr(a.status, MOE_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The joins of a group, by a warp of its own: the fence and the atomic's round
// trip after every item would take as long as its product. Parts that are
// finished by now are counted, up to 32 at once, and the blocks of columns
// whose last part that was are added up: part by part of the columns, over a
// token's experts in slot order.
template <typename X>
__device__ void join(const FewArgs& a, Ctrl& c, Group& g, const Work<X, false>& work) {
  const int lane = threadIdx.x & 31;
  const int R = a.T * a.k, all = c.plan.n_act * work.split;
  int done = 0;
  while (true) {
    int f = 0;
    bool ok = true;
    if (lane == 0)
      ok = poll(a, c, [&] {
        f = g.finished;
        return f < 0 || f > done;
      });
    if (!__all_sync(0xffffffffu, ok)) return;
    f = __shfl_sync(0xffffffffu, f, 0);
    // what lane 0 saw finished, the other lanes count: its read is ordered in
    // front of the warp's barrier, and their atomics behind a fence
    if (lane == 0) __threadfence_block();
    __syncwarp();
    const bool more = f >= 0;
    const int ready = more ? f : ~f;
    fence_gpu();
    while (done < ready) {
      const int n = min(32, ready - done);
      int blk = -1;
      if (lane < n) {
        blk = g.blk[(done + lane) % kJoinQueue];
        if (atomicAdd(&a.done[blk], 1) != all - 1) blk = -1;
      }
      uint32_t last = __ballot_sync(0xffffffffu, blk >= 0);
      // the parts are read by other lanes than the one whose atomic was the
      // last: it fences, and the warp's barrier hands that on
      fence_gpu();
      __syncwarp();
      while (last) {
        const int b = __shfl_sync(0xffffffffu, blk, __ffs(last) - 1);
        last &= last - 1;
        for (int u = lane; u < a.T * (kRows / 4); u += 32) {
          const int t = u / (kRows / 4), col = b * kRows + u % (kRows / 4) * 4;
          if (col >= a.d) continue;
          const float* y = a.y + (size_t)t * a.k * a.d + col;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = 0; p < work.split; ++p) {
#pragma unroll
            for (int j = 0; j < kMaxTopK; ++j) {
              if (j < a.k) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(y + ((size_t)p * R + j) * a.d));
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
              }
            }
          }
          put4(static_cast<X*>(a.out) + (size_t)t * a.d + col, s);
        }
      }
      done += n;
      if (lane == 0) g.joined = done;
    }
    if (!more) return;
  }
}

// few_down's products.
template <typename X>
__device__ void consume_down(const FewArgs& a, Ctrl& c, Group& g, const Ring& ring, float* red2, int group) {
  const int tid = threadIdx.x - (group * kGroupWarps + 2) * 32;
  const int R = a.T * a.k;
  Pos pos;
  int buf = 0;
  for (int n_item = 0;; ++n_item) {
    // the stage says which item begins
    bool ok = __all_sync(0xffffffffu, mbar_wait(&g.full[pos.stage], pos.phase, &c.abort, a.status, a.limit_ns));
    const int4 at = ok ? g.item[pos.stage] : make_int4(-1, 0, 0, 0);
    const int i = at.x;
    Item w;
    w.s = max(at.x, 0) & 0xff, w.part = max(at.x, 0) >> 8, w.blk = at.y, w.c0 = at.z, w.c1 = at.w;
    w.first = c.plan.base[w.s], w.n = c.plan.base[w.s + 1] - w.first;
    float* red = red2 + buf * red_floats<X>();
    buf ^= 1;
    if (i >= 0)
      ok = multiply<false>(w, a, c, g, ring, tid >> 5, a.I * (int)sizeof(X), pos, red, static_cast<const X*>(nullptr));
    // behind this barrier the parts of the items before this one are written
    if (!math_sync_all(group, ok)) return;
    if (tid < 32) {
      if (tid == 0) {
        __threadfence_block();
        g.finished = i >= 0 ? n_item : ~n_item;
      }
      if (i >= 0 && n_item >= kJoinQueue && !poll(a, c, [&] { return g.joined > n_item - kJoinQueue; })) ok = false;
      if (tid == 0) g.blk[n_item % kJoinQueue] = w.blk;
    }
    if (i < 0) return;
    const int r = tid & 15, n = tid >> 4, col = w.blk * kRows + r;
    if (n < w.n && col < a.d)
      a.y[((size_t)w.part * R + c.plan.tj[w.first + n]) * a.d + col] =
          c.plan.gate[w.first + n] * sum_parts<X>(red, r, n);
  }
}

template <typename X, bool kUp>
__device__ void stream(const FewMaps& maps, const FewArgs& a, Ctrl& c, uint8_t* smem_ring, float* red) {
  const int lane = threadIdx.x & 31;
  const int group = (int)(threadIdx.x >> 5) / kGroupWarps, role = (int)(threadIdx.x >> 5) % kGroupWarps;
  const Ring ring = ring_of<X, kUp>(smem_ring, c.plan, group);
  if (group >= ring.groups) return;
  Group& g = c.group[group];
  const int first = blockIdx.x * ring.groups + group, step = gridDim.x * ring.groups;
  Pos pos;
  int issued = 0;
  if (role == 0) {
    if (elect_one()) {
      bool ok;
      if constexpr (kUp)
        ok = produce_up_weights<X>(maps, a, c, g, ring, first, step, pos, issued);
      else
        ok = produce_down<X>(maps, a, c, g, ring, first, step, pos, issued);
      // few_down's first stages, while this kernel ends and that one starts
      if (kUp && ok && group == 0)
        prefetch_weights<X, false>(maps, a, c.plan.expert, c.plan.n_act, c.plan.down_split, blockIdx.x,
                                   a.down_blocks);
      if (!ok || c.abort) drain(a, g, ring, pos, issued);
    }
    __syncwarp();
  } else if (role == 1) {
    if constexpr (kUp) {
      const bool ok = produce_up_tokens<X>(a, c, g, ring, first, step, pos, issued);
      if (lane == 0 && (!ok || c.abort)) drain(a, g, ring, pos, issued);
      __syncwarp();
    } else {
      join<X>(a, c, g, Work<X, false>(a, c.plan.n_act, c.plan.down_split));
    }
  } else {
    red += group * 2 * red_floats<X>();
    if constexpr (kUp)
      consume_up<X>(a, c, g, ring, red, group, first, step);
    else
      consume_down<X>(a, c, g, ring, red, group);
  }
}

template <typename X, bool kUp>
__device__ __forceinline__ void init_ctrl(Ctrl& c) {
  if (threadIdx.x == 0) {
    for (int q = 0; q < Traits<X>::kGroups; ++q) {
      c.group[q].finished = c.group[q].joined = 0;
      for (int s = 0; s < kMaxStages; ++s) {
        mbar_init(&c.group[q].full[s], kUp ? 2 : 1);  // few_up has two producers
        mbar_init(&c.group[q].empty[s], kMathWarps);
      }
    }
    c.abort = 0;
    fence_mbarrier_init();
  }
}

template <typename X>
__device__ __forceinline__ void carve(uint8_t* smem, Ctrl** c, float** red, uint8_t** ring) {
  *c = reinterpret_cast<Ctrl*>(smem);
  *red = reinterpret_cast<float*>(smem + (sizeof(Ctrl) + 127) / 128 * 128);
  *ring = reinterpret_cast<uint8_t*>(*red + 2 * Traits<X>::kGroups * red_floats<X>());
}

template <typename X>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(threads<X>(), 1) few_up_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  Ctrl* c;
  float* red;
  uint8_t* ring;
  carve<X>(smem, &c, &red, &ring);
  init_ctrl<X, true>(*c);
  if (a.likely && threadIdx.x == 32) prefetch_weights<X, true>(maps, a, nullptr, a.E, 1, blockIdx.x, gridDim.x);
  float* part = reinterpret_cast<float*>(ring);                     // [kCluster][T][E]
  float* scratch = part + (size_t)kCluster * a.T * a.E;             // [kWarps][16][kPassLd]
  const int rank = (int)cluster_ctarank();
  __syncwarp();    // single threads of warps 0 and 1 were at work, and the barrier's instructions take whole warps
  cluster_sync();  // the peers' shared memory exists
  pdl_wait();
  pdl_trigger();
  if (a.own && threadIdx.x == 0) {
    a.head[kFewUpAt + blockIdx.x] = 0;
    if (blockIdx.x == 0) atomicExch(a.status, 0);
  }
  if (blockIdx.x == 0) {  // few_down counts on zeros
    for (int i = threadIdx.x; i < (a.d + kRows - 1) / kRows; i += blockDim.x) a.done[i] = 0;
    if (threadIdx.x == 0) *a.next = 0;
  }
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) c->bias[e] = a.br ? a.br[e] : 0.f;
  // this CTA's columns
  const int unit = 32, units = (a.d + unit - 1) / unit;
  const int c0 = min(a.d, rank * units / kCluster * unit), c1 = min(a.d, (rank + 1) * units / kCluster * unit);
  logits_part(static_cast<const X*>(a.x), static_cast<const X*>(a.wr), a.T, a.d, a.E, c0, c1, c->bias, scratch,
              part, rank);
  cluster_sync();  // all parts are here, and no peer writes here any more
  const bool first = blockIdx.x == 0;
  choose(a, part, reinterpret_cast<uint32_t*>(scratch), *c, first);
  __syncthreads();
  make_plan<X>(a, c->plan, c->idx, c->gate);
  if (first) {
    for (int i = threadIdx.x; i < kPlanWords; i += blockDim.x) a.head[kFewPlanAt + i] = reinterpret_cast<const int32_t*>(&c->plan)[i];
    if (a.counts || a.aux) statistics(a, part, *c);
  }
  fence_async();  // the ring's memory was written above, and is next by the copies
  __syncthreads();
  stream<X, true>(maps, a, *c, ring, red);
  if (a.own && c->abort) atomicOr(&a.head[kFewUpAt + blockIdx.x], MOE_DEV_TIMEOUT);  // who gave up sees its own mark
}

template <typename X>
__global__ void __launch_bounds__(threads<X>(), 1) few_down_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  Ctrl* c;
  float* red;
  uint8_t* ring;
  carve<X>(smem, &c, &red, &ring);
  init_ctrl<X, false>(*c);
  pdl_wait();
  pdl_trigger();
  static_assert(kFewUpWords <= threads<X>(), "a thread for each of few_up's words");
  if (blockIdx.x == 0 && (int)threadIdx.x < a.own)  // few_up's status bits
    if (const int bits = a.head[kFewUpAt + threadIdx.x]) atomicOr(a.status, bits);
  for (int i = threadIdx.x; i < kPlanWords; i += blockDim.x) reinterpret_cast<int32_t*>(&c->plan)[i] = a.head[kFewPlanAt + i];
  __syncthreads();
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
  cfg.blockDim = dim3(threads<X>(), 1, 1);
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
cudaError_t launch(const FewMaps& m, FewArgs a, cudaStream_t stream) {
  // the routing's scratch lies where the rings are, and a single group's has at least three stages
  constexpr int kRing = kSmemTotal - fixed_bytes<X>();
  static_assert(4 * (kCluster * kFewTokens * kMaxExperts + threads<X>() / 32 * kFewTokens * kPassLd) <= kRing, "routing scratch");
  static_assert(3 * (kWeightBytes + Traits<X>::kHid * kFewTokens * kTokPitch + 128) <= kRing, "ring");
  Device dev;
  cudaError_t err = device_info<X>(&dev);
  if (err != cudaSuccess) return err;
  a.down_blocks = dev.sms;
  // an expert is left out with probability (1 - k / E)^T if they are drawn
  // evenly: where that is rare, all experts' first weights are asked for
  // before the routing is known
  double out = 1.0;
  for (int t = 0; t < a.T; ++t) out *= 1.0 - (double)a.k / a.E;
  a.likely = out < 0.05;
  const int up_blocks = dev.clusters * kCluster;
  if (up_blocks > kFewUpWords) return cudaErrorInvalidConfiguration;
  if (a.own) a.own = up_blocks;
  err = launch_pdl(few_up_kernel<X>, dim3(up_blocks), dim3(threads<X>()), kSmemTotal, stream, m, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(few_down_kernel<X>, dim3(dev.sms), dim3(threads<X>()), kSmemTotal, stream, m, a);
}

}  // namespace

FewWorkspace few_layout(int T, int d, int k, int I, moe_dtype dtype) {
  const size_t R = (size_t)T * k, el = dtype == MOE_BF16 ? 2 : 4;
  FewWorkspace w;
  // room for finer parts where there are few rows: that is where the blocks
  // of 16 columns do not go evenly into the SMs
  w.split = R > 0 && 256 / R < kFewMaxSplit ? (int)(256 / R) : kFewMaxSplit;
  size_t o = 0;
  w.head = o; o = align256(o + 4 * (kFewUpAt + kFewUpWords));
  w.next = o; o = align256(o + 4);
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
