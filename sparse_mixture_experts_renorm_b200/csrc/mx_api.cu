// mx_api.cu — the C ABI of the MXFP4 operators (include/moe.h): argument
// checks, the workspace of the experts and the launch sequence
//   (router or count) -> scan -> dispatch + quantise -> gate/up + SwiGLU +
//   quantise -> down -> combine
// (without a router the dispatch does the scan, and for few choices the count)
// on the caller's stream. Nothing here synchronises the host or allocates.
#include "mx_internal.h"

using namespace moe;

namespace {

constexpr long long kIntMax = (1ll << 31) - 1;
// Rows of a product's operands: the end of a tile of 256 is an int as well.
constexpr long long kProductRows = kIntMax - 255;

// Byte offsets inside the workspace of the experts.
struct MxWorkspace {
  size_t status, offsets, counts, mtile, aux, blk_cnt, blk_psum, lrank, inv, rgate, xq, xq_sc, h, h_sc, y, y_exp, total;
  long long tiles;  // tile rows of the scales of the dispatched rows
};

MxWorkspace mx_layout(int T, int d, int E, int k, int I) {
  const size_t R = (size_t)T * k;
  const size_t nb = (size_t)router_blocks(T, MOE_F32);
  MxWorkspace w;
  // every expert with rows ends in at most one partial 256-row tile
  w.tiles = 2 * ((long long)(R / 256) + (long long)(R < (size_t)E ? R : (size_t)E));
  size_t o = 0;
  w.status = o;   o = align256(o + 4);
  w.offsets = o;  o = align256(o + 4 * (size_t)(E + 1));
  w.counts = o;   o = align256(o + 4 * (size_t)E);
  w.mtile = o;    o = align256(o + 4 * (size_t)(E + 1 + kMaxShared));
  w.aux = o;      o = align256(o + 4);
  w.blk_cnt = o;  o = align256(o + 4 * nb * E);
  w.blk_psum = o; o = align256(o + 4 * nb * E);
  w.lrank = o;    o = align256(o + 4 * R);
  w.inv = o;      o = align256(o + 4 * R);
  w.rgate = o;    o = align256(o + 4 * R);
  w.xq = o;       o = align256(o + R * (size_t)(d / 2));
  w.xq_sc = o;    o = align256(o + (size_t)w.tiles * mx_stage_count(d) * 1024);
  w.h = o;        o = align256(o + R * (size_t)(I / 2));
  w.h_sc = o;     o = align256(o + (size_t)w.tiles * mx_stage_count(I) * 1024);
  w.y = o;        o = align256(o + 2 * R * (size_t)d);
  w.y_exp = o;    o = align256(o + 8 * R * (size_t)mx_stage_count(d));
  w.total = o;
  return w;
}

moe_status check_matrix(int groups, long long rows, int cols, const char* what) {
  if (groups <= 0 || rows < 0 || cols <= 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: groups and columns must be positive and rows not negative (got %d, %d, %lld)",
                what, groups, cols, rows);
  if (cols % 32 != 0) return fail(MOE_ERR_UNSUPPORTED, "%s: MXFP4 needs columns %% 32 == 0 (got %d)", what, cols);
  if (rows > kIntMax || (long long)groups * rows > kIntMax)
    return fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows", what);
  return MOE_OK;
}

// The same with offsets: `rows` are those of all groups together.
moe_status check_ragged(int groups, long long rows, int cols, const char* what) {
  return groups <= 0 ? check_matrix(groups, 1, cols, what) : check_matrix(1, rows, cols, what);
}

moe_status check_mx_shape(int T, int d, int E, int k, int I) {
  moe_status st = check_shape(T, 64, E, k, 64, MOE_BF16);  // T, E and k as for the layer
  if (st != MOE_OK) return st;
  if (d <= 0 || I <= 0) return fail(MOE_ERR_INVALID_ARG, "d and I must be positive (got d=%d I=%d)", d, I);
  if (d % 32 != 0 || I % 32 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "MXFP4 experts need d %% 32 == 0 and I %% 32 == 0 (got d=%d I=%d)", d, I);
  if ((long long)d * I > kIntMax || (long long)E * I > kProductRows || (long long)E * d > kProductRows ||
      (long long)T * k > kProductRows)
    return fail(MOE_ERR_UNSUPPORTED, "d*I must be < 2^31, and E*I, E*d and T*k at most 2^31 - 256");
  return MOE_OK;
}

bool row_maps(MxMaps* m, const void* a, uint64_t rows, uint64_t row_bytes) {
  return make_tmap_mx_codes(&m->a, a, rows, row_bytes) && make_tmap_mx_codes(&m->a32, a, rows, row_bytes, 32);
}

bool weight_maps(MxMaps* m, const void* b0, const void* s0, const void* b1, const void* s1, uint64_t E, uint64_t N,
                 uint64_t K) {
  const uint64_t rows = E * (uint64_t)mx_group_tiles((long long)N) * mx_stage_count((int)K);
  return make_tmap_mx_codes(&m->b0, b0, E * N, K / 2) && make_tmap_mx_codes(&m->b1, b1, E * N, K / 2) &&
         make_tmap_mx_scales(&m->sb0, s0, rows) && make_tmap_mx_scales(&m->sb1, s1, rows);
}

moe_status mx_layer(const void* x, const void* w_router, const float* b_router, const moe_mx_weights* w, int T, int d,
                    int E, int k, int I, int renorm, moe_dtype dtype, void* out, int32_t* topk_idx, float* topk_gate,
                    int32_t* counts, float* aux, void* workspace, size_t workspace_bytes, int32_t* status_dev,
                    void* stream_ptr, bool route) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  moe_status st = check_mx_shape(T, d, E, k, I);
  if (st == MOE_OK && route) st = check_shape(T, d, E, k, dtype == MOE_BF16 ? 64 : I, dtype);
  if (st != MOE_OK) return st;
  if (route && renorm != 0 && renorm != 1)
    return fail(MOE_ERR_INVALID_ARG, "renorm must be 0 or 1 (got %d)", renorm);
  if (!w || w->struct_bytes < sizeof(moe_mx_weights))
    return fail(MOE_ERR_INVALID_ARG, "moe_mx_weights is NULL or its struct_bytes is too small");
  if (T > 0) {
    if (!x || !out || !topk_idx || !topk_gate || (route && !w_router) || !w->gate || !w->gate_scales || !w->up ||
        !w->up_scales || !w->down || !w->down_scales)
      return fail(MOE_ERR_INVALID_ARG, "a required pointer (x, weights, scales, out, topk_idx, topk_gate) is NULL");
    const void* al[] = {x, out, w->gate, w->gate_scales, w->up, w->up_scales, w->down, w->down_scales,
                        route ? w_router : nullptr};
    for (const void* p : al)
      if (!aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "x, weights, scales and out must be 16-byte aligned");
  }
  const MxWorkspace l = mx_layout(T, d, E, k, I);
  if (!workspace || workspace_bytes < l.total)
    return fail(MOE_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu%s)", l.total, workspace_bytes,
                workspace ? "" : ", NULL");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* status = status_dev ? status_dev : reinterpret_cast<int32_t*>(ws + l.status);
  int32_t* cnt = counts ? counts : reinterpret_cast<int32_t*>(ws + l.counts);
  float* aux_p = aux ? aux : reinterpret_cast<float*>(ws + l.aux);
  cudaError_t err = cudaSuccess;
  if (!status_dev) err = cudaMemsetAsync(status, 0, sizeof(int32_t), stream);
  if (err == cudaSuccess && T == 0) {
    err = cudaMemsetAsync(cnt, 0, sizeof(int32_t) * E, stream);
    if (err == cudaSuccess) err = cudaMemsetAsync(aux_p, 0, sizeof(float), stream);
  }
  if (err != cudaSuccess) return fail_cuda(err, "clearing the status word");
  if (T == 0) return MOE_OK;

  const int R = T * k;
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + l.offsets);
  int32_t* mtile = reinterpret_cast<int32_t*>(ws + l.mtile);
  int32_t* blk_cnt = reinterpret_cast<int32_t*>(ws + l.blk_cnt);
  float* blk_psum = reinterpret_cast<float*>(ws + l.blk_psum);
  int32_t* lrank = reinterpret_cast<int32_t*>(ws + l.lrank);
  int32_t* inv = reinterpret_cast<int32_t*>(ws + l.inv);
  float* rgate = reinterpret_cast<float*>(ws + l.rgate);
  uint8_t *xq = ws + l.xq, *xq_sc = ws + l.xq_sc, *h = ws + l.h, *h_sc = ws + l.h_sc, *y = ws + l.y;

  MxMaps up, down;
  if (!row_maps(&up, xq, (uint64_t)R, (uint64_t)d / 2) ||
      !make_tmap_mx_scales(&up.sa, xq_sc, (uint64_t)l.tiles * mx_stage_count(d)) ||
      !weight_maps(&up, w->gate, w->gate_scales, w->up, w->up_scales, E, I, d) ||
      !row_maps(&down, h, (uint64_t)R, (uint64_t)I / 2) ||
      !make_tmap_mx_scales(&down.sa, h_sc, (uint64_t)l.tiles * mx_stage_count(I)) ||
      !weight_maps(&down, w->down, w->down_scales, w->down, w->down_scales, E, d, I))
    return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (driver entry point unavailable or bad pointer)");

  MxDispatch md = {};
  md.scan = kScanDone;
  md.rb = kRouterTokensTc;
  const int nb = (T + kRouterTokensTc - 1) / kRouterTokensTc;
  bool scan = false;  // by its kernel
  if (route) {
    md.rb = router_block_tokens(dtype);
    RouterNorm rn = {};
    RouterScan rs;
    rs.counts = cnt;
    rs.offsets = offsets;
    rs.mtile = mtile;
    rs.aux = aux_p;
    scan = !router_does_scan(T, E, dtype);
    err = launch_router(dtype, x, w_router, b_router, T, d, E, k, renorm, rn, topk_idx, topk_gate, lrank, blk_cnt,
                        blk_psum, nullptr, rs, status, stream);
    if (err != cudaSuccess) return fail_cuda(err, "router kernel");
  } else if (R <= kScanAllMost) {
    md.scan = kScanAll;
  } else {
    if ((long long)nb * E <= kScanBlocksMost)
      md.scan = kScanBlocks;
    else
      scan = true;
    err = launch_mx_count(topk_idx, T, E, k, lrank, blk_cnt, blk_psum, status, stream);
    if (err != cudaSuccess) return fail_cuda(err, "count kernel");
  }
  if (scan) {
    err = launch_route_scan((T + md.rb - 1) / md.rb, T, E, k, -1, 0, blk_cnt, blk_psum, nullptr, cnt, offsets, mtile, aux_p,
                            nullptr, nullptr, nullptr, 0, stream);
    if (err != cudaSuccess) return fail_cuda(err, "routing scan kernel");
  }
  md.topk_idx = topk_idx;
  md.topk_gate = topk_gate;
  md.lrank = lrank;
  md.blk = blk_cnt;
  md.counts = cnt;
  md.offsets = offsets;
  md.mtile = mtile;
  err = launch_mx_dispatch(dtype, x, T, d, E, k, md, inv, rgate, xq, xq_sc, status, stream);
  if (err != cudaSuccess) return fail_cuda(err, "dispatch kernel");
  MxOut hid = {};
  hid.form = kMxHidden;
  hid.h = h;
  hid.h_scales = h_sc;
  err = launch_mx_gateup(up, offsets, E, R, I, d, (int)mx_group_tiles(I), hid, status, stream);
  if (err != cudaSuccess) return fail_cuda(err, "gate/up product (MXFP4)");
  MxOut yo = {};
  yo.out = y;
  yo.form = kMxY16;
  yo.y_exp = ws + l.y_exp;
  yo.gate = rgate;
  err = launch_mx_product(down, offsets, E, R, d, I, (int)mx_group_tiles(d), yo, status, stream);
  if (err != cudaSuccess) return fail_cuda(err, "down product (MXFP4)");
  err = launch_mx_combine(y, ws + l.y_exp, inv, T, d, k, out, status, stream);
  if (err != cudaSuccess) return fail_cuda(err, "combine kernel");
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_mx_scale_bytes(int groups, int rows, int cols, int ragged) {
  if ((ragged ? check_ragged : check_matrix)(groups, rows, cols, "moe_mx_scale_bytes") != MOE_OK) return 0;
  const long long tiles = ragged ? 2 * ((long long)rows / 256 + (rows < groups ? rows : groups))
                                 : groups * mx_group_tiles(rows);
  return (size_t)(tiles > 2 ? tiles : 2) * mx_stage_count(cols) * 1024;
}

static moe_status convert_args(const void* a, const void* data, const void* scales, size_t scale_bytes,
                               const int32_t* offsets, int groups, int rows, int cols, moe_dtype dtype,
                               size_t* tile_rows, const char* what) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  const moe_status st = (offsets ? check_ragged : check_matrix)(groups, rows, cols, what);
  if (st != MOE_OK) return st;
  if (offsets && groups > kMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "%s: at most %d groups of rows with offsets (got %d)", what, kMaxExperts, groups);
  const size_t need = moe_mx_scale_bytes(groups, rows, cols, offsets != nullptr);  // not 0: the sizes are valid
  if (need == 0) return MOE_ERR_INVALID_ARG;
  if (scale_bytes < need)
    return fail(MOE_ERR_INVALID_ARG, "%s: the scales need %zu bytes (got %zu)", what, need, scale_bytes);
  if (rows > 0) {
    if (!a || !data || !scales) return fail(MOE_ERR_INVALID_ARG, "%s: a required pointer is NULL", what);
    if (!aligned16(a) || !aligned16(data) || !aligned16(scales))
      return fail(MOE_ERR_INVALID_ARG, "%s: values, codes and scales must be 16-byte aligned", what);
    if ((offsets ? 1ll : (long long)groups) * rows * (cols / 8) / 1024 >= kIntMax)
      return fail(MOE_ERR_UNSUPPORTED, "%s: the matrix is too large for one call", what);
  }
  *tile_rows = scale_bytes / ((size_t)mx_stage_count(cols) * 1024);
  return MOE_OK;
}

moe_status moe_mx_quantize(const void* x, const int32_t* offsets, int groups, int rows, int cols, moe_dtype dtype,
                           void* data, void* scales, size_t scale_bytes, void* stream) {
  size_t tile_rows = 0;
  const moe_status st =
      convert_args(x, data, scales, scale_bytes, offsets, groups, rows, cols, dtype, &tile_rows, "moe_mx_quantize");
  if (st != MOE_OK || rows == 0) return st;
  const cudaError_t err =
      launch_mx_quantize(dtype, x, offsets ? rows : (long long)groups * rows, rows, cols, offsets, groups,
                         (int)mx_group_tiles(rows), tile_rows, data, scales, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? MOE_OK : fail_cuda(err, "MXFP4 quantisation kernel");
}

moe_status moe_mx_dequantize(const void* data, const void* scales, size_t scale_bytes, const int32_t* offsets,
                             int groups, int rows, int cols, moe_dtype dtype, void* out, void* stream) {
  size_t tile_rows = 0;
  const moe_status st = convert_args(out, data, scales, scale_bytes, offsets, groups, rows, cols, dtype, &tile_rows,
                                     "moe_mx_dequantize");
  if (st != MOE_OK || rows == 0) return st;
  const cudaError_t err =
      launch_mx_dequantize(dtype, data, scales, offsets ? rows : (long long)groups * rows, rows, cols, offsets, groups,
                           (int)mx_group_tiles(rows), tile_rows, out, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? MOE_OK : fail_cuda(err, "MXFP4 dequantisation kernel");
}

moe_status moe_mx_matmul(const void* a, const void* a_scales, const void* b, const void* b_scales,
                         const int32_t* offsets, int groups, int M, int N, int K, moe_dtype out_dtype, void* out,
                         int32_t* status_dev, void* stream) {
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARG, "unknown output dtype %d", (int)out_dtype);
  moe_status st = (offsets ? check_ragged : check_matrix)(groups, M, K, "moe_mx_matmul (A)");
  if (st == MOE_OK) st = check_matrix(groups, N, K, "moe_mx_matmul (B)");
  if (st != MOE_OK) return st;
  if (N <= 0) return fail(MOE_ERR_INVALID_ARG, "N must be positive (got %d)", N);
  if (N % 8 != 0) return fail(MOE_ERR_UNSUPPORTED, "the product needs N %% 8 == 0 (got %d)", N);
  if (groups > kMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "at most %d groups (got %d)", kMaxExperts, groups);
  const long long a_tiles =
      offsets ? 2 * ((long long)M / 256 + (M < groups ? M : groups)) : groups * mx_group_tiles(M);
  const long long b_tiles = groups * mx_group_tiles(N);
  const int stages = mx_stage_count(K);
  if ((offsets ? 1ll : (long long)groups) * M > kProductRows || (long long)groups * N > kProductRows ||
      a_tiles * stages > kIntMax || b_tiles * stages > kIntMax || (a_tiles / 2) * ((N + 255) / 256) > kIntMax)
    return fail(MOE_ERR_UNSUPPORTED, "the product is too large for one call");
  if (M == 0) return MOE_OK;
  if (!a || !a_scales || !b || !b_scales || !out || !status_dev)
    return fail(MOE_ERR_INVALID_ARG, "a required pointer (codes, scales, out, status_dev) is NULL");
  if (!aligned16(a) || !aligned16(a_scales) || !aligned16(b) || !aligned16(b_scales) || !aligned16(out))
    return fail(MOE_ERR_INVALID_ARG, "codes, scales and out must be 16-byte aligned");
  MxMaps m;
  if (!row_maps(&m, a, (offsets ? 1ull : (uint64_t)groups) * M, (uint64_t)K / 2) ||
      !make_tmap_mx_scales(&m.sa, a_scales, (uint64_t)a_tiles * stages) ||
      !weight_maps(&m, b, b_scales, b, b_scales, groups, N, K))
    return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (driver entry point unavailable or bad pointer)");
  MxOut o = {};
  o.out = out;
  o.form = out_dtype == MOE_F32 ? kMxF32 : kMxBf16;
  const cudaError_t err = launch_mx_product(m, offsets, groups, M, N, K, (int)mx_group_tiles(N), o, status_dev,
                                            static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? MOE_OK : fail_cuda(err, "MXFP4 product kernel");
}

size_t moe_mx_workspace_size(int T, int d, int E, int k, int I) {
  if (check_mx_shape(T, d, E, k, I) != MOE_OK) return 0;
  return mx_layout(T, d, E, k, I).total;
}

moe_status moe_mx_experts(const void* x, const int32_t* topk_idx, const float* topk_gate, const moe_mx_weights* w,
                          int T, int d, int E, int k, int I, moe_dtype dtype, void* out, int32_t* counts,
                          void* workspace, size_t workspace_bytes, int32_t* status_dev, void* stream) {
  return mx_layer(x, nullptr, nullptr, w, T, d, E, k, I, 0, dtype, out, const_cast<int32_t*>(topk_idx),
                  const_cast<float*>(topk_gate), counts, nullptr, workspace, workspace_bytes, status_dev, stream,
                  false);
}

moe_status moe_mx_forward(const void* x, const void* w_router, const float* b_router, const moe_mx_weights* w, int T,
                          int d, int E, int k, int I, int renorm, moe_dtype dtype, void* out, int32_t* topk_idx,
                          float* topk_gate, int32_t* counts, float* aux, void* workspace, size_t workspace_bytes,
                          int32_t* status_dev, void* stream) {
  return mx_layer(x, w_router, b_router, w, T, d, E, k, I, renorm, dtype, out, topk_idx, topk_gate, counts, aux,
                  workspace, workspace_bytes, status_dev, stream, true);
}

}  // extern "C"
