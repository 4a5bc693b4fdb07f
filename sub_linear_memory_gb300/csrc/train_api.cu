// train_api.cu -- the slim_group_norm* and slim_adamw entry points of
// include/slim_attn.h: argument checks and dispatch.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "common.cuh"
#include "train.h"

namespace slim {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxCols = 16384, kMaxRows = 1 << 30;

struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

#define SLIM_TRY(expr)                    \
  do {                                    \
    const slim_status try_st = (expr);    \
    if (try_st != SLIM_OK) return try_st; \
  } while (0)

slim_status finish(cudaError_t err, cudaStream_t st) {
  if (err != cudaSuccess) return SLIM_ERR_CUDA;
#ifdef SLIM_DEBUG
  return slim_attn_sync_status((slim_stream_t)st);
#else
  (void)st;
  return SLIM_OK;
#endif
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

slim_status check_sizes(int rows, int cols, int groups, float eps) {
  if (rows < 0 || cols < 1 || groups < 1 || cols % groups || !(eps >= 0.f)) return SLIM_ERR_INVALID_ARG;
  return cols > kMaxCols || rows > kMaxRows ? SLIM_ERR_UNSUPPORTED : SLIM_OK;
}

slim_status check_ptr(const void *p, size_t size) {
  if (!p) return SLIM_ERR_INVALID_ARG;
  return aligned(p, size) ? SLIM_OK : SLIM_ERR_UNSUPPORTED;
}

template <typename T>
slim_status run_norm(const void *x, const float *gamma, const float *beta, const void *gate, long long gate_row,
                     float eps, void *y, int rows, int cols, int groups, cudaStream_t st) {
  NvtxRange range("slim_group_norm");
  SLIM_TRY(check_sizes(rows, cols, groups, eps));
  if (rows == 0) return SLIM_OK;
  SLIM_TRY(check_ptr(x, sizeof(T)));
  SLIM_TRY(check_ptr(gamma, 4));
  SLIM_TRY(check_ptr(beta, 4));
  SLIM_TRY(check_ptr(y, sizeof(T)));
  if (y == x || y == gate) return SLIM_ERR_INVALID_ARG;
  if (gate && rows > 1 && gate_row < cols) return SLIM_ERR_INVALID_ARG;
  if (!aligned(gate, sizeof(T))) return SLIM_ERR_UNSUPPORTED;
  return finish(group_norm<T>(x, gamma, beta, gate, gate ? gate_row : 0, eps, y, rows, cols, groups, st), st);
}

template <typename T>
slim_status run_norm_bwd(const void *dy, const void *x, const float *gamma, const float *beta, const void *gate,
                         long long gate_row, float eps, void *dx, void *dgate, long long dgate_row, float *dgamma,
                         float *dbeta, void *workspace, size_t workspace_bytes, int rows, int cols, int groups, cudaStream_t st) {
  NvtxRange range("slim_group_norm_bwd");
  SLIM_TRY(check_sizes(rows, cols, groups, eps));
  if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return SLIM_ERR_UNSUPPORTED;
  if (rows == 0) {
    for (float *sum : {dgamma, dbeta})
      if (sum && cudaMemsetAsync(sum, 0, sizeof(float) * cols, st) != cudaSuccess) return SLIM_ERR_CUDA;
    return SLIM_OK;
  }
  SLIM_TRY(check_ptr(dy, sizeof(T)));
  SLIM_TRY(check_ptr(x, sizeof(T)));
  SLIM_TRY(check_ptr(gamma, 4));
  SLIM_TRY(check_ptr(beta, 4));
  SLIM_TRY(check_ptr(dx, sizeof(T)));
  if (!gate != !dgate || (gate && rows > 1 && (gate_row < cols || dgate_row < cols))) return SLIM_ERR_INVALID_ARG;
  if (!aligned(gate, sizeof(T)) || !aligned(dgate, sizeof(T))) return SLIM_ERR_UNSUPPORTED;
  for (const void *out : {dx, dgate})
    if (out && (out == dy || out == x || out == gate)) return SLIM_ERR_INVALID_ARG;
  if (dx == dgate) return SLIM_ERR_INVALID_ARG;
  if (dgamma || dbeta) {
    if (!workspace || workspace_bytes < group_norm_bwd_workspace(rows, cols, groups)) return SLIM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SLIM_ERR_UNSUPPORTED;
  }
  return finish(group_norm_bwd<T>(dy, x, gamma, beta, gate, gate ? gate_row : 0, eps, dx, dgate, gate ? dgate_row : 0, dgamma, dbeta, workspace, rows, cols,
                                  groups, st),
                st);
}

bool fraction(double b) { return b >= 0.0 && b < 1.0; }

slim_status run_adamw(const slim_adamw_tensor *tensors, int n, const slim_adamw_options *options, int *count,
                      bool g_f32, cudaStream_t st) {
  NvtxRange range("slim_adamw");
  if (!options || n < 0 || (n && !tensors) || !count) return SLIM_ERR_INVALID_ARG;
  const slim_adamw_options &o = *options;
  if (!fraction(o.beta1) || !fraction(o.beta2) || !(o.eps >= 0.f) || (o.bits != 8 && o.bits != 32))
    return SLIM_ERR_INVALID_ARG;
  if (!aligned(count, 4) || !aligned(o.lr_device, 4)) return SLIM_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i) {
    const slim_adamw_tensor &t = tensors[i];
    if (t.n < 0) return SLIM_ERR_INVALID_ARG;
    if (t.n > (1ll << 40)) return SLIM_ERR_UNSUPPORTED;
    if (t.n == 0 || !t.grad) continue;
    if (!t.param || !t.m || !t.v || (o.bits == 8 && (!t.m_scales || !t.v_scales))) return SLIM_ERR_INVALID_ARG;
    if (!aligned(t.param, 4) || !aligned(t.grad, g_f32 ? 4 : 2) || !aligned(t.m, o.bits == 8 ? 16 : 4) ||
        !aligned(t.v, o.bits == 8 ? 16 : 4))
      return SLIM_ERR_UNSUPPORTED;
  }
  return finish(adamw(tensors, n, o, g_f32, count, st), st);
}

}  // namespace
}  // namespace slim

using namespace slim;

extern "C" {

slim_status slim_group_norm(const void *x, const float *gamma, const float *beta, const void *gate, long long gate_row, float eps, void *y,
                            int rows, int cols, int groups, slim_stream_t stream) {
  return run_norm<bf16>(x, gamma, beta, gate, gate_row, eps, y, rows, cols, groups, (cudaStream_t)stream);
}

slim_status slim_group_norm_f32(const float *x, const float *gamma, const float *beta, const float *gate, long long gate_row, float eps,
                                float *y, int rows, int cols, int groups, slim_stream_t stream) {
  return run_norm<float>(x, gamma, beta, gate, gate_row, eps, y, rows, cols, groups, (cudaStream_t)stream);
}

slim_status slim_group_norm_bwd(const void *dy, const void *x, const float *gamma, const float *beta, const void *gate,
                                long long gate_row, float eps, void *dx, void *dgate, long long dgate_row, float *dgamma, float *dbeta, void *workspace,
                                size_t workspace_bytes, int rows, int cols, int groups, slim_stream_t stream) {
  return run_norm_bwd<bf16>(dy, x, gamma, beta, gate, gate_row, eps, dx, dgate, dgate_row, dgamma, dbeta, workspace, workspace_bytes, rows,
                            cols, groups, (cudaStream_t)stream);
}

slim_status slim_group_norm_bwd_f32(const float *dy, const float *x, const float *gamma, const float *beta,
                                    const float *gate, long long gate_row, float eps, float *dx, float *dgate,
                                    long long dgate_row, float *dgamma, float *dbeta,
                                    void *workspace, size_t workspace_bytes, int rows, int cols, int groups,
                                    slim_stream_t stream) {
  return run_norm_bwd<float>(dy, x, gamma, beta, gate, gate_row, eps, dx, dgate, dgate_row, dgamma, dbeta, workspace, workspace_bytes, rows,
                             cols, groups, (cudaStream_t)stream);
}

size_t slim_group_norm_bwd_workspace_bytes(int rows, int cols, int groups) {
  if (check_sizes(rows, cols, groups, 0.f) != SLIM_OK || rows == 0) return 0;
  return group_norm_bwd_workspace(rows, cols, groups);
}

slim_status slim_adamw(const slim_adamw_tensor *tensors, int n, const slim_adamw_options *options, int *count,
                       slim_stream_t stream) {
  return run_adamw(tensors, n, options, count, false, (cudaStream_t)stream);
}

slim_status slim_adamw_f32(const slim_adamw_tensor *tensors, int n, const slim_adamw_options *options, int *count,
                           slim_stream_t stream) {
  return run_adamw(tensors, n, options, count, true, (cudaStream_t)stream);
}

}  // extern "C"
