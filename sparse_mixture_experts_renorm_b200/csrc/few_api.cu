// few_api.cu — the C ABI of the layer for a few tokens (include/moe.h):
// argument checks and the workspace of few.cu's two kernels.
#include "few_internal.h"

using namespace moe;

namespace {

moe_status check_few(int T, int d, int E, int k, int I, moe_dtype dtype) {
  moe_status st = check_shape(T, 64, E, k, 64, dtype);  // T, E, k and the type as for the layer
  if (st != MOE_OK) return st;
  if (d <= 0 || I <= 0) return fail(MOE_ERR_INVALID_ARG, "d and I must be positive (got d=%d I=%d)", d, I);
  if (T > kFewTokens)
    return fail(MOE_ERR_UNSUPPORTED, "moe_forward_few takes at most %d tokens (got %d)", kFewTokens, T);
  const int unit = dtype == MOE_BF16 ? 8 : 4;
  if (d % unit != 0 || I % unit != 0)
    return fail(MOE_ERR_UNSUPPORTED, "d and I must be multiples of %d (got d=%d I=%d)", unit, d, I);
  // row lengths in bytes, rows of all experts and the items of a product are 32-bit numbers
  constexpr long long most = (1ll << 31) - 1;
  if ((long long)d * 4 > most || (long long)I * 4 > most || (long long)E * I > most || (long long)E * d > most)
    return fail(MOE_ERR_UNSUPPORTED, "4 d, 4 I, E*I and E*d must be < 2^31 (got d=%d I=%d E=%d)", d, I, E);
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_few_workspace_size(int T, int d, int E, int k, int I, moe_dtype dtype) {
  if (check_few(T, d, E, k, I, dtype) != MOE_OK) return 0;
  return few_layout(T, d, k, I, dtype).total;
}

moe_status moe_forward_few(const void* x, const void* w_router, const float* b_router, const void* w_gate,
                           const void* w_up, const void* w_down, int T, int d, int E, int k, int I, int renorm,
                           moe_dtype dtype, void* out, int32_t* topk_idx, float* topk_gate, int32_t* counts,
                           float* aux, void* workspace, size_t workspace_bytes, int32_t* status_dev,
                           void* stream_ptr) {
  const moe_status st = check_few(T, d, E, k, I, dtype);
  if (st != MOE_OK) return st;
  if (renorm != 0 && renorm != 1) return fail(MOE_ERR_INVALID_ARG, "renorm must be 0 or 1 (got %d)", renorm);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (T == 0) {
    if (status_dev && status_dev == workspace && workspace_bytes < sizeof(int32_t))
      return fail(MOE_ERR_WORKSPACE, "the workspace has no room for the call's status word (%zu bytes)", workspace_bytes);
    cudaError_t err = counts ? cudaMemsetAsync(counts, 0, sizeof(int32_t) * E, stream) : cudaSuccess;
    if (err == cudaSuccess && aux) err = cudaMemsetAsync(aux, 0, sizeof(float), stream);
    if (err == cudaSuccess && status_dev && status_dev == workspace)
      err = cudaMemsetAsync(status_dev, 0, sizeof(int32_t), stream);
    return err == cudaSuccess ? MOE_OK : fail_cuda(err, "zeroing counts, the statistic and the status word for T=0");
  }
  if (!x || !w_router || !w_gate || !w_up || !w_down || !out || !topk_idx || !topk_gate || !status_dev)
    return fail(MOE_ERR_INVALID_ARG,
                "a required pointer (x, weights, out, topk_idx, topk_gate, status_dev) is NULL");
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) ||
      !aligned16(out))
    return fail(MOE_ERR_INVALID_ARG, "x, weights and out must be 16-byte aligned");
  const FewWorkspace l = few_layout(T, d, k, I, dtype);
  if (!workspace || workspace_bytes < l.total)
    return fail(MOE_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu%s)", l.total, workspace_bytes,
                workspace ? "" : ", NULL");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  FewArgs a = {};
  a.x = x, a.wr = w_router, a.wg = w_gate, a.wu = w_up, a.wd = w_down, a.br = b_router;
  a.T = T, a.d = d, a.E = E, a.k = k, a.I = I, a.renorm = renorm;
  a.out = out, a.idx = topk_idx, a.gate = topk_gate, a.counts = counts, a.aux = aux;
  a.head = reinterpret_cast<int32_t*>(ws + l.head);
  a.next = reinterpret_cast<int32_t*>(ws + l.next);
  a.done = reinterpret_cast<int32_t*>(ws + l.done);
  a.h = ws + l.h;
  a.y = reinterpret_cast<float*>(ws + l.y);
  a.split = l.split;
  a.status = status_dev;
  a.own = status_dev == workspace;
  a.limit_ns = kWaitLimitNs;
  FewMaps m;
  if (!make_tmap_few(&m.wg, w_gate, dtype, (uint64_t)E * I, (uint64_t)d, 8) ||
      !make_tmap_few(&m.wu, w_up, dtype, (uint64_t)E * I, (uint64_t)d, 8) ||
      !make_tmap_few(&m.wd, w_down, dtype, (uint64_t)E * d, (uint64_t)I, 16))
    return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (driver entry point unavailable or bad pointer)");
  const cudaError_t err = launch_few(dtype, m, a, stream);
  return err == cudaSuccess ? MOE_OK : fail_cuda(err, "few-token kernels");
}

}  // extern "C"
