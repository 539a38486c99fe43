// mx_gemm_rows.cu — the grouped MXFP4 product of mx_gemm.cu for groups of few
// rows:
//
//   out[r, n] = g_r * sum_k A[r, k] B[e(r), n, k]
//
// The tile of mx_gemm.cu is 256 rows high: a group of 100 leaves the tensor
// cores more than half of every tile to multiply for nobody. Here weight rows
// are the UMMA M operand (256 a pair of CTAs, 128 each) and the group's rows
// the N operand, as many as there are (up to 128, in steps of 32; each CTA
// stages half of them). A TMEM lane then holds one weight row, that is one
// column of the result, and its columns are the group's rows, so that a warp
// stores 32 consecutive columns of one row at a time. The accumulator takes
// 128 columns at most, so there are two, and the epilogue runs beside the next
// tile's products. 26 KB a stage, 8 stages; otherwise as there.
//
// Taken where groups have at most 64 rows on average (mx_gemm.cu has both sides
// measured: past 128 rows a group takes twice the tiles, and stores of single
// columns). Bound by the weights' bytes: 64 rows over 8 groups of 4096 x
// 14336 in 46 us, 5.4 TB/s, with the weights in memory (40 us when the call is
// repeated and L2 still holds a part of them).
#include "mx_umma.cuh"

namespace moe {
namespace {

constexpr int kStages = 8;
constexpr int kEpiWarps = 16;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTokens = 128;                 // rows of a tile
constexpr int kWBytes = 128 * 128;           // 128 weight rows x 256 codes
constexpr int kBoxBytes = 32 * 128;          // 32 rows of A
constexpr int kABytes = 2 * kBoxBytes;
constexpr int kScaleBytes = 2 * kMxStageBytes;
constexpr int kSmem = kStages * (kWBytes + kABytes + kScaleBytes) + 1024 + 4096;
constexpr uint32_t kScaleCol = 256;          // first TMEM column of the scales
constexpr int kScaleBufs = 4, kScaleCols = 16;
static_assert(kSmem <= 227 * 1024, "shared memory");

// Rows that a tile multiplies: those that there are, in steps of 32.
__device__ __forceinline__ int tile_rows(const MxTile& t) { return min(kTokens, (t.cnt - t.m * kTokens + 31) & ~31); }

template <int kForm>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_gemm_rows_kernel(const __grid_constant__ CUtensorMap tmA32, const __grid_constant__ CUtensorMap tmSA,
                        const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmSB,
                        const int32_t* __restrict__ offsets, int G, int M, int N, int K, int group_tiles,
                        const MxOut out, int32_t* status, uint64_t limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sA = smem + kStages * kWBytes;
  uint8_t* sS = smem + kStages * (kWBytes + kABytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * (kWBytes + kABytes + kScaleBytes));
  uint64_t* full = bars;             // leader: the stage's bytes of both CTAs
  uint64_t* empty = bars + kStages;  // both: stage consumed by the pair's UMMAs
  uint64_t* tfull = bars + 2 * kStages;  // both: an accumulator is complete
  uint64_t* tempty = tfull + 2;          // leader: the epilogue warps of both CTAs have read it
  uint64_t* done = tempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_bad = reinterpret_cast<int*>(s_tmem + 2);
  int* s_off = reinterpret_cast<int*>(s_tmem + 4);  // [G + 1]
  int* s_mt = s_off + kMaxExperts + 1;              // [G + 1] tiles of kTokens rows before a group
  int* s_sc = s_mt + kMaxExperts + 1;               // [G] tile row of its first scales

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = (int)cluster_id_x();
  const int ncl = (int)num_clusters_x();
  const int n_wb = (N + 255) / 256;
  const int KB = mx_stages(K);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(done, 1);
    *s_abort = 0;
    *s_bad = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, 512);
    tmem_relinquish_pair();
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();
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
    int run = 0, scales = 0;
    for (int g0 = 0; g0 < G; g0 += 32) {
      const int g = g0 + lane;
      const int cnt = g < G && !*s_bad ? s_off[g + 1] - s_off[g] : 0;
      const int t = (cnt + kTokens - 1) / kTokens, u = 2 * ((cnt + 255) >> 8);
      int ti = t, ui = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, ti, o), b = __shfl_up_sync(0xffffffffu, ui, o);
        if (lane >= o) ti += a, ui += b;
      }
      if (g < G) {
        s_mt[g] = run + ti - t;
        s_sc[g] = scales + ui - u;
      }
      run += __shfl_sync(0xffffffffu, ti, 31);
      scales += __shfl_sync(0xffffffffu, ui, 31);
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
        const int half = tile_rows(t) / 2;  // this CTA's rows: 16, 32, 48 or 64
        const int boxes = (half + 31) >> 5;
        const int arow = t.row0 + t.m * kTokens + (int)rank * half;
        const int asf = (s_sc[t.g] + t.m) * KB;
        const int brow = t.g * N + t.n * 256 + (int)rank * 128;
        const int bsf = (t.g * group_tiles + 2 * t.n + (int)rank) * KB;
        const uint32_t tx = 2u * (kWBytes + kScaleBytes + (uint32_t)(boxes * kBoxBytes));
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, s_abort, status, limit_ns)) {
            ok = false;
            break;
          }
          const uint32_t fbar = map_to_cta(&full[stage], 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], tx);
          uint8_t* ss = sS + stage * kScaleBytes;
          tma_load_2d_pair(sW + stage * kWBytes, &tmB, fbar, kb * 128, brow);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d_pair(sA + stage * kABytes + b * kBoxBytes, &tmA32, fbar, kb * 128, arow + 32 * b);
          tma_load_2d_pair(ss, &tmSB, fbar, 0, bsf + kb);
          tma_load_2d_pair(ss + kMxStageBytes, &tmSA, fbar, 0, asf + kb);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // loads land on the leader's barriers: it waits for the last phase of
      // each stage it armed (these cover both CTAs' bytes)
      if (leader) {
        const int n = issued < kStages ? issued : kStages;
        for (int i = 0; i < n; ++i) {
          if (stage == 0) {
            stage = kStages;
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
      const uint64_t w0 = sw128_kmajor_desc(smem_u32(sW)), a0 = sw128_kmajor_desc(smem_u32(sA));
      const uint64_t s0 = scales_desc(smem_u32(sS));
      const int whole = K / kMxStageCols;
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      uint32_t sf = tmem_base + kScaleCol;
      uint64_t wdesc = w0, adesc = a0, sdesc = s0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        const MxTile t = mx_tile(tile, n_wb, s_off, s_mt, G);
        const int rows = tile_rows(t);
        const uint32_t id0 = idesc_mxf4(256, 0, 0u) | (static_cast<uint32_t>(rows >> 3) << 17);
        const uint32_t id2 = idesc_mxf4(256, 0, 2u) | (static_cast<uint32_t>(rows >> 3) << 17);
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kTokens);
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, s_abort, status, limit_ns)) break;
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&full[stage], phase, s_abort, status, limit_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // columns: the weights' two tiles of scales at 0 and 4, A's at 8 and 12
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            tc_cp_scales_pair(sf + 4 * s, sdesc + (512 >> 4) * s);
            tc_cp_scales_pair(sf + 8 + 4 * s, sdesc + (kMxStageBytes >> 4) + (512 >> 4) * s);
          }
          const int steps = kb < whole ? 4 : (K - kb * kMxStageCols + 63) >> 6;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s >= steps) break;
            tc_mma_mxf4_pair(d, wdesc + 2 * s, adesc + 2 * s, s & 1 ? id2 : id0, sf + 4 * (s >> 1),
                             sf + 8 + 4 * (s >> 1), s > 0 ? 1u : (uint32_t)kb);
          }
          tc_commit_pair_both(&empty[stage]);
          sf = sf == tmem_base + kScaleCol + (kScaleBufs - 1) * kScaleCols ? tmem_base + kScaleCol : sf + kScaleCols;
          wdesc += kWBytes >> 4;
          adesc += kABytes >> 4;
          sdesc += kScaleBytes >> 4;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
            wdesc = w0, adesc = a0, sdesc = s0;
          }
        }
        if (!ok) break;
        tc_commit_pair_both(&tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tc_commit_pair_local(done);
      mbar_wait(done, 0, nullptr, status, limit_ns);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue --
    // TMEM lane = a weight row of this CTA's 128; the four groups of four warps
    // take 32 rows of A each.
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = cid; tile < total; tile += ncl) {
      const MxTile t = mx_tile(tile, n_wb, s_off, s_mt, G);
      const int first = t.m * kTokens + part * 32;  // first row in its group
      const int n = min(32, t.cnt - first);         // <= 0: none
      float gate = 0.f;                             // lane i: row i's; asked for before the wait
      if (kForm == kMxY16 && lane < n) gate = __ldg(out.gate + t.row0 + first + lane);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, s_abort, status, limit_ns))) break;
      tc_fence_after();
      uint32_t v[32];
      __syncwarp();
      if (n > 0) {
        tmem_ld_x32(tbase + acc * kTokens + part * 32, v);
        tmem_ld_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(map_to_cta(&tempty[acc], 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
      const int col0 = t.n * 256 + (int)rank * 128 + q * 32, col = col0 + lane;
      if (n <= 0 || col0 >= N) continue;
      const bool live = col < N;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (i < n) {
          const size_t row = (size_t)(t.row0 + first + i);
          if (kForm == kMxY16) {
            const float x = __shfl_sync(0xffffffffu, gate, i) * __uint_as_float(v[i]);
            const uint32_t e = y16_exp(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7fffffffu));
            const uint32_t w = e == 0xffu ? pack_bf16x2(x, 0.f) : y16_pack(x, 0.f, y16_inv(e));
            static_cast<uint16_t*>(out.out)[row * N + col] = (uint16_t)w;
            if (lane == 0) out.y_exp[y16_exp_at((size_t)M, col, row)] = (uint8_t)e;
          } else if (live) {
            if (kForm == kMxF32)
              static_cast<uint32_t*>(out.out)[row * N + col] = v[i];
            else
              static_cast<__nv_bfloat16*>(out.out)[row * N + col] = __float2bfloat16_rn(__uint_as_float(v[i]));
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
  auto kern = mx_gemm_rows_kernel<kForm>;
  const int pairs = max_pairs(reinterpret_cast<const void*>(kern), kThreads, kSmem, cache);
  if (pairs <= 0) return cudaErrorInvalidConfiguration;
  const long long n_wb = (N + 255) / 256;
  const long long row_tiles =
      offsets ? (long long)M / kTokens + G : (long long)G * ((M + kTokens - 1) / kTokens);
  const long long most = row_tiles * n_wb;
  const int clusters = (int)(most < pairs ? most : pairs);
  if (clusters <= 0) return cudaSuccess;
  return launch_pdl(kern, dim3(2 * clusters), dim3(kThreads), kSmem, stream, m.a32, m.sa, m.b0, m.sb0, offsets, G, M, N,
                    K, group_tiles, out, status, kWaitLimitNs);
}

}  // namespace

cudaError_t launch_mx_product_rows(const MxMaps& m, const int32_t* offsets, int G, int M, int N, int K, int group_tiles,
                                   const MxOut& out, int32_t* status, cudaStream_t stream) {
  if (out.form == kMxY16) return launch<kMxY16>(m, offsets, G, M, N, K, group_tiles, out, status, stream);
  if (out.form == kMxF32) return launch<kMxF32>(m, offsets, G, M, N, K, group_tiles, out, status, stream);
  return launch<kMxBf16>(m, offsets, G, M, N, K, group_tiles, out, status, stream);
}

}  // namespace moe
