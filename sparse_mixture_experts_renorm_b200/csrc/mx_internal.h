// mx_internal.h — launchers of the MXFP4 kernels (host-side declarations).
#pragma once

#include "moe_internal.h"

namespace moe {

// Rows of 128-row scale tiles that one group of `rows` rows takes (a group
// starts at a new pair of tiles).
inline long long mx_group_tiles(long long rows) { return (rows + 255) / 256 * 2; }
// Pieces of 256 columns (one pipeline stage of the product) of a row.
inline int mx_stage_count(int cols) { return (int)(((unsigned)cols + 255) / 256); }

// Rows to MXFP4 and back. offsets == NULL: x is [n_rows / rows, rows, cols],
// every group padded to group_tiles tile rows of scales; otherwise x is
// [n_rows, cols] with G <= kMaxExperts groups at offsets[0..G]. tile_rows: tile
// rows that the scales hold (nothing is written or read past them).
cudaError_t launch_mx_quantize(moe_dtype dtype, const void* x, long long n_rows, int rows, int cols,
                               const int32_t* offsets, int G, int group_tiles, size_t tile_rows, void* data,
                               void* scales, cudaStream_t stream);
cudaError_t launch_mx_dequantize(moe_dtype dtype, const void* data, const void* scales, long long n_rows, int rows,
                                 int cols, const int32_t* offsets, int G, int group_tiles, size_t tile_rows, void* out,
                                 cudaStream_t stream);

// Tensor maps of one MXFP4 product: codes of A in boxes of 128 and of 32 rows,
// its scales, and those of one or two weights (the product repeats the first).
struct MxMaps {
  CUtensorMap a, a32, sa, b0, b1, sb0, sb1;
};

// Where an MXFP4 product writes: out [M, N] in bf16, fp32 or, each row
// multiplied by gate[row], as 16-bit numbers with their exponents in y_exp
// (mx.cuh, y16); or for gate/up the MXFP4 hidden rows.
enum MxForm { kMxBf16, kMxF32, kMxY16, kMxHidden };
struct MxOut {
  void* out;
  int form;
  const float* gate;
  uint8_t* y_exp;
  uint8_t* h;
  uint8_t* h_scales;
};

// out[r] = gate[r] * A[r] . B[g]^T for the rows r of each group g (offsets
// NULL: G groups of M rows each; otherwise M rows in all). N: weight rows per
// group, group_tiles: tile rows of scales per weight group.
cudaError_t launch_mx_product(const MxMaps& m, const int32_t* offsets, int G, int M, int N, int K, int group_tiles,
                              const MxOut& out, int32_t* status, cudaStream_t stream);
// The same for groups of few rows (mx_gemm_rows.cu); launch_mx_product takes it by itself.
cudaError_t launch_mx_product_rows(const MxMaps& m, const int32_t* offsets, int G, int M, int N, int K, int group_tiles,
                                   const MxOut& out, int32_t* status, cudaStream_t stream);
// H[r] = MXFP4(SiLU(A[r] . B0[g]^T) * (A[r] . B1[g]^T)), N hidden units.
cudaError_t launch_mx_gateup(const MxMaps& m, const int32_t* offsets, int G, int M, int N, int K, int group_tiles,
                             const MxOut& out, int32_t* status, cudaStream_t stream);

// Codes [rows, row_bytes] in boxes of box_rows x 128 bytes (128-byte swizzle),
// and scales as rows of 1024 bytes, one row a box. False on failure.
bool make_tmap_mx_codes(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes, uint32_t box_rows = 128);
bool make_tmap_mx_scales(CUtensorMap* map, const void* base, uint64_t rows);

// The dispatch of given choices: per block of kRouterTokensTc tokens the
// counts of every expert, the rank of every (token, slot) among the block's
// assignments of its expert (slots of a token in order), and zeros in
// blk_psum. A choice outside [0, E) sets MOE_DEV_INTERNAL and gets rank -1.
cudaError_t launch_mx_count(const int32_t* topk_idx, int T, int E, int k, int32_t* lrank, int32_t* blk_cnt,
                            float* blk_psum, int32_t* status, cudaStream_t stream);

// How the dispatch gets the rows of the experts: from the routing scan's
// results (blk_base, offsets and mtile), from the counts of each block of rb
// tokens, or from the choices themselves. In the last two cases it writes
// counts, offsets and mtile.
enum MxScan { kScanDone, kScanBlocks, kScanAll };
// At most this many choices are counted by every block of the dispatch (1.3 us
// for 4096), and this many counts of token blocks summed by each; more take
// kernels of their own.
constexpr int kScanAllMost = 4096, kScanBlocksMost = 8192;
struct MxDispatch {
  MxScan scan;
  int rb;
  const int32_t* topk_idx;
  const float* topk_gate;
  const int32_t* lrank;    // [T, k] rank among the token block's choices of the expert (not for kScanAll)
  const int32_t* blk;      // [nb, E] base rows (kScanDone) or counts (kScanBlocks)
  int32_t *counts, *offsets, *mtile;
};
// Each token's row of x to MXFP4 once, written at the row of each of its
// choices; also inv [T, k] (-1 for a choice out of range) and the rows' gates.
cudaError_t launch_mx_dispatch(moe_dtype dtype, const void* x, int T, int d, int E, int k, const MxDispatch& a,
                               int32_t* inv, float* rgate, void* data, void* scales, int32_t* status,
                               cudaStream_t stream);

// out[t] = sum over t's choices of the rows Y[inv[t, j]] (y16, gated already).
cudaError_t launch_mx_combine(const void* y, const uint8_t* y_exp, const int32_t* inv, int T, int d, int k, void* out,
                              int32_t* status, cudaStream_t stream);

}  // namespace moe
