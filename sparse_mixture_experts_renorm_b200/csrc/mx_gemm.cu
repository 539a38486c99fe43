// mx_gemm.cu — grouped products of MXFP4 matrices on block-scaled tcgen05
// (kind::mxf4) with a pair of CTAs (cta_group::2) per 256 x 256 tile.
//
//   product:  out[r, n] = g_r * sum_k A[r, k] B[e(r), n, k]
//   gate/up:  H[r, i]   = MXFP4( SiLU(A[r] . Wg[e, i]) * (A[r] . Wu[e, i]) )
//
// for the rows r of group e (an expert's dispatched rows). The tensor cores
// multiply E2M1 codes exactly, apply the two E8M0 scales of every 32 products
// and add in fp32, so nothing is rounded before the epilogue.
//
// Rows are the UMMA M operand (128 per CTA), weight rows the N operand (128
// staged by each CTA; for gate/up CTA 0 stages the gate rows of the block's
// 128 hidden units and CTA 1 their up rows, so a TMEM lane holds one row's
// gate values in columns 0-127 and its up values in 128-255, and neither
// SwiGLU nor the quantisation of H leaves the thread). A pipeline stage is 256
// columns of K: 128 bytes of codes a row with the 128-byte swizzle, as for 64
// bf16, and 1024 bytes of scales per 128 rows, which one thread copies to TMEM
// (tcgen05.cp) in front of the stage's four UMMAs. Both CTAs need the scales
// of all 256 weight rows. 35 KB a stage, 6 stages (a load's round trip is 1.4 us
// and a stage's products take 0.28: five stages run dry). The issuing thread is the
// one that elect.sync names: the compiler then keeps the operands in uniform
// registers. With a test of the lane it moved them there in front of every
// instruction, 99 cycles for a copy and 135 for a product, and a stage took
// 1434 cycles of the 512 that its products last; now 553.
//
// TMEM: the accumulator takes 256 of 512 columns, the scales 32 columns for
// each of 4 rotating buffers, so there is no room for a second accumulator of
// 256 columns. Instead sixteen epilogue warps first bring their 64 columns into
// registers and release the accumulator, then do the arithmetic and the stores
// while the next tile's UMMAs run.
//
// Persistent: clusters walk the tiles (groups in order, weight block outer,
// row tile inner). Every wait is bounded.
//
// Measured: 8192 x 14336 x 4096 to bf16 in 161 to 169 us, 5.9 PFLOP/s (bursts;
// the tensor pipe is busy 79 % of the time). Run for seconds it draws the 1 kW that
// the card allows, the clock falls from 1.9 to 1.4 GHz and it takes 195 us;
// with zeros for codes it does not. A tile costs 0.9 us beside its products
// (the last of them, the accumulator's way out, the first stage): 28 % for the
// 8 stages of K = 2048. 32 rows through the Mixtral-shaped experts are bound by
// the weights' bytes: gate/up 90 us, 5.5 TB/s.
#include "mx.cuh"
#include "mx_internal.h"
#include "mx_umma.cuh"

namespace moe {
namespace {

constexpr int kMxStages = 6;
constexpr int kMxEpiWarps = 16;
constexpr int kMxThreads = 64 + 32 * kMxEpiWarps;
constexpr int kHalf = 128 * 128;                // 128 rows x 256 codes
constexpr int kSfBytes = 3 * kMxStageBytes;     // scales of 128 rows, and of 256 weight rows
constexpr int kMxSmem = kMxStages * (2 * kHalf + kSfBytes) + 1024 + 4096;
constexpr uint32_t kStageTx = 2u * (2 * kHalf + kSfBytes);  // both CTAs, all rows
constexpr uint32_t kSfCol = 256;                // first TMEM column of the scales
constexpr int kSfBufs = 4, kSfCols = 32;
static_assert(kMxSmem <= 227 * 1024, "shared memory");

// kN lanes, each with kN 16-byte units of its own row: lane l of them gets
// unit l of every one of their rows, so that a store of the warp writes 16 kN
// consecutive bytes of a row. Whole lines (8) cost half as many shuffles again
// and are better where a kernel's loads wait for its stores (the experts' down
// product: 58 us against 63 for the fine-grained layer), half lines (4) where
// HBM takes the results anyway (8192 x 14336 x 4096: 167 against 169).
template <int kN>
__device__ __forceinline__ void transpose_units(uint32_t (&w)[kN][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < kN; o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      if (u & o) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[u][i] : w[u + o][i], o);
        if (up)
          w[u][i] = got;
        else
          w[u + o][i] = got;
      }
    }
  }
}

// kForm: what is written (MxForm); the hidden rows: gate/up, see above. Maps: codes of A and of the weights (boxes of 128 rows x
// 128 bytes), scales of A and of the weights (boxes of 1024 bytes). For the
// product tmB1/tmSB1 repeat tmB0/tmSB0.
template <int kForm>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                   const __grid_constant__ CUtensorMap tmSA,
                   const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                   const __grid_constant__ CUtensorMap tmSB0, const __grid_constant__ CUtensorMap tmSB1,
                   const int32_t* __restrict__ offsets, int G, int M, int N, int K, int group_tiles,
                   const MxOut out, int32_t* status, uint64_t limit_ns) {
  constexpr bool kGateUp = kForm == kMxHidden;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kMxStages * kHalf;
  uint8_t* sS = smem + 2 * kMxStages * kHalf;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kMxStages * (2 * kHalf + kSfBytes));
  uint64_t* full = bars;               // leader: the stage's bytes of both CTAs
  uint64_t* empty = bars + kMxStages;  // both: stage consumed by the pair's UMMAs
  uint64_t* tfull = bars + 2 * kMxStages;
  uint64_t* tempty = tfull + 1;        // leader: the epilogue warps of both CTAs
  uint64_t* done = tempty + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 4);  // [G + 1]
  int* s_mt = s_off + kMaxExperts + 1;              // [G + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = (int)cluster_id_x();
  const int ncl = (int)num_clusters_x();
  const int n_wb = kGateUp ? (N + 127) / 128 : (N + 255) / 256;
  const int KB = mx_stages(K);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * kMxEpiWarps);
    mbar_init(done, 1);
    *s_abort = 0;
    *s_bad = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, 512);
    tmem_relinquish_pair();
  }
  // Rows that a group lacks are not loaded. The tensor cores multiply what is
  // there all the same, with most of the power if it is data: zeros.
  for (int i = threadIdx.x; i < kMxStages * kHalf / 16; i += kMxThreads)
    reinterpret_cast<uint4*>(sA)[i] = make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  // the groups' rows and the prefix of their 256-row tiles
  for (int i = threadIdx.x; i <= G; i += blockDim.x) {
    const int o = offsets ? offsets[i] : i * M;
    s_off[i] = o;
    const int next = i < G ? (offsets ? offsets[i + 1] : (i + 1) * M) : o;
    if (o < 0 || next < o || (offsets && next > M)) *s_bad = 1;
  }
  __syncthreads();
  if (*s_bad) {  // not a partition of the rows: nothing is computed
    if (threadIdx.x == 0) atomicOr(status, MOE_DEV_INTERNAL);
  }
  if (warp == 0) {
    int run = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      const int t = (g < G && !*s_bad) ? (s_off[g + 1] - s_off[g] + 255) >> 8 : 0;
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
      }
      if (g < G) s_mt[g] = run + incl - t;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_mt[G] = run;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  const int total = s_mt[G] * n_wb;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        const MxTile t = mx_tile(tile, n_wb, s_off, s_mt, G);
        const int arow = t.row0 + t.m * 256 + (int)rank * 128;
        const int asf = (2 * (s_mt[t.g] + t.m) + (int)rank) * KB;
        // gate/up: rank 0 stages the gate rows, rank 1 the up rows
        const int brow = kGateUp ? t.g * N + t.n * 128 : t.g * N + t.n * 256 + (int)rank * 128;
        const CUtensorMap* mB = kGateUp && rank ? &tmB1 : &tmB0;
        const int bsf0 = (t.g * group_tiles + (kGateUp ? t.n : 2 * t.n)) * KB;
        const int bsf1 = kGateUp ? bsf0 : bsf0 + KB;
        // this CTA's rows that exist, in boxes of 32, and the other's
        const int rows = t.cnt - t.m * 256;
        const int boxes0 = min(4, (rows + 31) >> 5), boxes1 = max(0, min(4, (rows - 128 + 31) >> 5));
        const int boxes = leader ? boxes0 : boxes1;
        const uint32_t tx = kStageTx - (uint32_t)((8 - boxes0 - boxes1) * (kHalf / 4));
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, s_abort, status, limit_ns)) {
            ok = false;
            break;
          }
          const uint32_t fbar = map_to_cta(&full[stage], 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], tx);
          uint8_t* ss = sS + stage * kSfBytes;
          if (boxes == 4) {
            tma_load_2d_pair(sA + stage * kHalf, &tmA, fbar, kb * 128, arow);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(sA + stage * kHalf + b * (kHalf / 4), &tmA32, fbar, kb * 128, arow + 32 * b);
          }
          tma_load_2d_pair(sB + stage * kHalf, mB, fbar, kb * 128, brow);
          tma_load_2d_pair(ss, &tmSA, fbar, 0, asf + kb);
          tma_load_2d_pair(ss + kMxStageBytes, &tmSB0, fbar, 0, bsf0 + kb);
          tma_load_2d_pair(ss + 2 * kMxStageBytes, &tmSB1, fbar, 0, bsf1 + kb);
          ++issued;
          if (++stage == kMxStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // loads land on the leader's barriers: it waits for the last phase of
      // each stage it armed (these cover both CTAs' bytes)
      if (leader) {
        const int n = issued < kMxStages ? issued : kMxStages;
        for (int i = 0; i < n; ++i) {
          if (stage == 0) {
            stage = kMxStages;
            phase ^= 1u;
          }
          --stage;
          mbar_wait(&full[stage], phase, nullptr, status, limit_ns);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------ MMA issuer (leader only) --
    if (leader && elect_one()) {
      // few instructions a stage: the epilogue's warps share this warp's
      // scheduler, and while they compute the products wait for this one
      const uint64_t a0 = sw128_kmajor_desc(smem_u32(sA)), b0 = sw128_kmajor_desc(smem_u32(sB));
      const uint64_t s0 = scales_desc(smem_u32(sS));
      const int whole = K / kMxStageCols;  // stages of four steps of 64 columns; the last may have fewer
      int stage = 0;
      uint32_t phase = 0;
      uint32_t acc_phase = 0;
      uint32_t sf = tmem_base + kSfCol;
      uint64_t adesc = a0, bdesc = b0, sdesc = s0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&full[stage], phase, s_abort, status, limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // columns: A's two tiles at 0 and 4, B's two at 8 and 16 (eight
          // columns: the scales of 2 x 128 weight rows). A short last stage's
          // second half is copied too and not used.
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            tc_cp_scales_pair(sf + 4 * t, sdesc + (512 >> 4) * t);
            tc_cp_scales_pair(sf + 8 + 8 * t, sdesc + (kMxStageBytes >> 4) + (512 >> 4) * t);
            tc_cp_scales_pair(sf + 12 + 8 * t, sdesc + (2 * kMxStageBytes >> 4) + (512 >> 4) * t);
          }
          if (kb == 0) {  // the accumulator; the scales did not have to wait for it
            if (!mbar_wait(tempty, acc_phase ^ 1u, s_abort, status, limit_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          if (kb < whole) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc_mma_mxf4_pair(tmem_base, adesc + 2 * s, bdesc + 2 * s, idesc_mxf4(256, 256, s & 1 ? 2u : 0u),
                               sf + 4 * (s >> 1), sf + 8 + 8 * (s >> 1), s > 0 ? 1u : (uint32_t)kb);
          } else {
            const int steps = (K - kb * kMxStageCols + 63) >> 6;
#pragma unroll 1
            for (int s = 0; s < steps; ++s)
              tc_mma_mxf4_pair(tmem_base, adesc + 2 * s, bdesc + 2 * s, idesc_mxf4(256, 256, s & 1 ? 2u : 0u),
                               sf + 4 * (s >> 1), sf + 8 + 8 * (s >> 1), (uint32_t)(kb | s));
          }
          tc_commit_pair_both(&empty[stage]);
          sf = sf == tmem_base + kSfCol + (kSfBufs - 1) * kSfCols ? tmem_base + kSfCol : sf + kSfCols;
          adesc += kHalf >> 4;
          bdesc += kHalf >> 4;
          sdesc += kSfBytes >> 4;
          if (++stage == kMxStages) {
            stage = 0;
            phase ^= 1u;
            adesc = a0, bdesc = b0, sdesc = s0;
          }
        }
        if (!ok) break;
        tc_commit_pair_both(tfull);
        acc_phase ^= 1u;
      }
      tc_commit_pair_local(done);
      mbar_wait(done, 0, nullptr, status, limit_ns);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue --
    // TMEM lane = a row of this CTA's half of the tile. The four groups of
    // four warps take 64 columns each, or 32 units of the gate and up halves.
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t tempty_leader = map_to_cta(tempty, 0);
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t acc_phase = 0;
    const int rt = q * 32 + lane;  // row of this CTA's 128
    for (int tile = cid; tile < total; tile += ncl) {
      const MxTile t = mx_tile(tile, n_wb, s_off, s_mt, G);
      const int first = t.m * 256 + (int)rank * 128 + q * 32;  // this warp's first row in its group
      float gate = 0.f;  // asked for before the wait
      if (kForm == kMxY16 && first + lane < t.cnt) gate = __ldg(out.gate + t.row0 + first + lane);
      if (!__all_sync(0xffffffffu, mbar_wait(tfull, acc_phase, s_abort, status, limit_ns))) break;
      acc_phase ^= 1u;
      tc_fence_after();
      uint32_t v[2][32];
      __syncwarp();
      tmem_ld_x32(tbase + (kGateUp ? part * 32 : part * 64), v[0]);
      tmem_ld_x32(tbase + (kGateUp ? 128 + part * 32 : part * 64 + 32), v[1]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader);
      if (first >= t.cnt) continue;  // none of them exists
      if (kGateUp) {
        const int unit0 = t.n * 128 + part * 32;
        float h[32];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          h[i] = silu_f32(__uint_as_float(v[0][i])) * __uint_as_float(v[1][i]);
          m = max(m, __float_as_uint(h[i]) & 0x7fffffffu);
        }
        const uint32_t sb = unit0 < N ? mx_scale_byte(m) : 0u;
        const float inv = mx_inv_scale(sb);
#pragma unroll
        for (int i = 0; i < 32; ++i) h[i] *= inv;
        if (first + lane < t.cnt) {
          if (unit0 < N)
            *reinterpret_cast<uint4*>(out.h + (size_t)(t.row0 + first + lane) * (N / 2) + unit0 / 2) =
                make_uint4(mx_pack8(h), mx_pack8(h + 8), mx_pack8(h + 16), mx_pack8(h + 24));
          // one of the four bytes of this row in the block's tile of scales
          out.h_scales[mx_scale_at((size_t)(2 * (s_mt[t.g] + t.m) + (int)rank), mx_stages(N), rt, t.n * 4 + part)] =
              (uint8_t)sb;
        }
      } else {
        // kN units of every row at a time
        constexpr int kN = kForm == kMxY16 ? 8 : 4;
        constexpr int el = kForm == kMxF32 ? 4 : 2, cols = 16 * kN / el;
#pragma unroll
        for (int p = 0; p < 64 / cols; ++p) {
          uint32_t w[kN][4];
          if (kForm == kMxF32) {
#pragma unroll
            for (int i = 0; i < cols; ++i) w[i >> 2][i & 3] = v[p >> 1][(p & 1) * 16 + i];
          } else if (kForm == kMxBf16) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i >> 2][i & 3] = pack_bf16x2(__uint_as_float(v[p & 1][2 * i]), __uint_as_float(v[p & 1][2 * i + 1]));
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float m = 0.f;
#pragma unroll
              for (int i = 0; i < 32; ++i) m = max_abs_nan(m, __uint_as_float(v[c][i]));
              // the largest of the gated values: rounding does not change which it is
              const uint32_t e = y16_exp(__float_as_uint(fabsf(gate) * m));
              const float inv = y16_inv(e), f = gate * inv;
              if (__all_sync(0xffffffffu, e != 0xffu && fabsf(f) <= 3.0e38f)) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  w[(4 * c + (i >> 2)) % kN][i & 3] =
                      y16_pack(__uint_as_float(v[c][2 * i]), __uint_as_float(v[c][2 * i + 1]), f);
              } else {  // gate * inv out of range, or a block that is kept as bf16
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float x = gate * __uint_as_float(v[c][2 * i]), y = gate * __uint_as_float(v[c][2 * i + 1]);
                  w[(4 * c + (i >> 2)) % kN][i & 3] = e == 0xffu ? pack_bf16x2(x, y) : y16_pack(x, y, inv);
                }
              }
              const int col = t.n * 256 + part * 64 + c * 32;
              if (first + lane < t.cnt && col < N)
                out.y_exp[y16_exp_at((size_t)M, col, (size_t)(t.row0 + first + lane))] = (uint8_t)e;
            }
          }
          transpose_units(w);
          const int col = t.n * 256 + part * 64 + p * cols + (lane & (kN - 1)) * (16 / el), r0 = lane & ~(kN - 1);
          uint8_t* dst = static_cast<uint8_t*>(out.out) + ((size_t)(t.row0 + first + r0) * N + col) * el;
          if (col < N) {
#pragma unroll
            for (int r = 0; r < kN; ++r)
              if (first + r0 + r < t.cnt)
                *reinterpret_cast<uint4*>(dst + (size_t)r * N * el) = make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its shared memory or TMEM
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int kForm>
cudaError_t launch(const MxMaps& m, const int32_t* offsets, int G, int M, int N, int K, int group_tiles,
                   const MxOut& out, int32_t* status, cudaStream_t stream) {
  static std::atomic<int> cache[64];
  constexpr bool kGateUp = kForm == kMxHidden;
  auto kern = mx_gemm_kernel<kForm>;
  const int pairs = max_pairs(reinterpret_cast<const void*>(kern), kMxThreads, kMxSmem, cache);
  if (pairs <= 0) return cudaErrorInvalidConfiguration;
  const long long n_wb = kGateUp ? (N + 127) / 128 : (N + 255) / 256;
  const long long row_tiles = offsets ? (long long)M / 256 + G : (long long)G * ((M + 255) / 256);
  const long long most = row_tiles * n_wb;
  const int clusters = (int)(most < pairs ? most : pairs);
  if (clusters <= 0) return cudaSuccess;
  return launch_pdl(kern, dim3(2 * clusters), dim3(kMxThreads), kMxSmem, stream, m.a, m.a32, m.sa, m.b0, m.b1, m.sb0, m.sb1,
                    offsets, G, M, N, K, group_tiles, out, status, kWaitLimitNs);
}

}  // namespace

cudaError_t launch_mx_product(const MxMaps& m, const int32_t* offsets, int G, int M, int N, int K, int group_tiles,
                              const MxOut& out, int32_t* status, cudaStream_t stream) {
  // By the average, as the lengths are known only on the device. us there and
  // here, in a graph, weights from memory:
  //   rows in every group       8           64          96          128         192
  //   64 x 1408 x 2048      22.5 24.4   25.2 26.0   26.7 27.4   28.0 28.3   39.8 30.1
  //   8 x 4096 x 14336      46.5 51.0   45.4 49.8   46.3 50.9   47.2 51.7   62.8 53.5
  //   8 x 14336 x 4096      49.1 55.4   49.5 57.3   50.5 58.4   52.2 59.2   74.4 61.0
  //   1 x 4096 x 4096        8.7 11.3    9.2 10.5    9.2 10.9    9.2 11.1    9.6 11.3
  // Its tiles hold 128 rows, so groups of equal length cross between 128 and 192.
  // Uneven ones do before, and half of that leaves room for them: 64 groups of 60
  // rows on average, the largest of 809, 26.7 and 26.0; one of 4000 rows among 63
  // of one, 29.9 and 28.8 (K 1408, N 2048: 32.8 and 30.6, the worst that was seen)
  if ((long long)M <= (offsets ? 64ll * G : 64ll))
    return launch_mx_product_rows(m, offsets, G, M, N, K, group_tiles, out, status, stream);
  if (out.form == kMxY16) return launch<kMxY16>(m, offsets, G, M, N, K, group_tiles, out, status, stream);
  if (out.form == kMxF32) return launch<kMxF32>(m, offsets, G, M, N, K, group_tiles, out, status, stream);
  return launch<kMxBf16>(m, offsets, G, M, N, K, group_tiles, out, status, stream);
}

cudaError_t launch_mx_gateup(const MxMaps& m, const int32_t* offsets, int G, int M, int N, int K, int group_tiles,
                             const MxOut& out, int32_t* status, cudaStream_t stream) {
  return launch<kMxHidden>(m, offsets, G, M, N, K, group_tiles, out, status, stream);
}

}  // namespace moe
