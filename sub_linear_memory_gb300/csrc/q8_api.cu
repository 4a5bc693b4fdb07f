// q8_api.cu -- the slim_q8_* entry points of include/slim_attn.h: argument
// checks and dispatch of the 8-bit layer operators.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "kernels.h"
#include "q8.h"
#include "q8_common.cuh"

namespace slim {
namespace q8 {
namespace {

constexpr int kMaxNormCols = 16384;  // a row in the registers of 16 warps
constexpr int kMaxK = 131072;        // scale words of a product's k in tensor memory
constexpr int kMaxRowTiles = 65535;  // 128-row tiles along a grid axis

struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Negative sizes, or more blocks than the kernels' 32-bit block index counts.
slim_status check_size(int rows, int cols) {
  if (rows < 0 || cols < 0) return SLIM_ERR_INVALID_ARG;
  if ((long long)rows * blocks_of(cols) >= (1ll << 31)) return SLIM_ERR_UNSUPPORTED;
  return SLIM_OK;
}

// Both buffers of an 8-bit matrix; optional: both NULL, or neither.
slim_status check_mat(const void *codes, const void *scales, bool optional) {
  if (!codes != !scales || (!codes && !optional)) return SLIM_ERR_INVALID_ARG;
  return aligned(codes, 16) && aligned(scales, 4) ? SLIM_OK : SLIM_ERR_UNSUPPORTED;
}

template <typename T>
slim_status check_rows(const void *p) {
  if (!p) return SLIM_ERR_INVALID_ARG;
  return aligned(p, sizeof(T)) ? SLIM_OK : SLIM_ERR_UNSUPPORTED;
}

slim_status finish(cudaError_t err, cudaStream_t st) {
  if (err != cudaSuccess) return SLIM_ERR_CUDA;
#ifdef SLIM_DEBUG
  return slim_attn_sync_status((slim_stream_t)st);
#else
  (void)st;
  return SLIM_OK;
#endif
}

#define SLIM_TRY(expr)                       \
  do {                                       \
    const slim_status try_st = (expr);       \
    if (try_st != SLIM_OK) return try_st;    \
  } while (0)

template <typename T>
slim_status run_quantize(const void *x, void *codes, void *scales, void *z_codes, void *z_scales, bool act, int rows,
                         int cols, cudaStream_t st) {
  NvtxRange range(act ? "slim_q8_gelu" : "slim_q8_quantize");
  SLIM_TRY(check_size(rows, cols));
  if (rows == 0 || cols == 0) return SLIM_OK;
  SLIM_TRY(check_rows<T>(x));
  SLIM_TRY(check_mat(codes, scales, false));
  SLIM_TRY(check_mat(z_codes, z_scales, true));
  return finish(quantize<T>(x, codes, scales, z_codes, z_scales, act, rows, cols, st), st);
}

template <typename T>
slim_status run_dequantize(const void *codes, const void *scales, void *x, int rows, int cols, int block_rows,
                           cudaStream_t st) {
  NvtxRange range("slim_q8_dequantize");
  SLIM_TRY(check_size(rows, cols));
  if (block_rows != 1 && block_rows != kBlock) return SLIM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return SLIM_OK;
  SLIM_TRY(check_rows<T>(x));
  SLIM_TRY(check_mat(codes, scales, false));
  return finish(dequantize<T>(codes, scales, x, rows, cols, block_rows, st), st);
}

template <typename T>
slim_status run_pack_weight(const void *w, void *codes, void *scales, void *codes_t, void *scales_t, int n, int k,
                            cudaStream_t st) {
  NvtxRange range("slim_q8_pack_weight");
  SLIM_TRY(check_size(n, k));
  SLIM_TRY(check_size(k, n));
  if (blocks_of(n) > kMaxRowTiles) return SLIM_ERR_UNSUPPORTED;
  if (n == 0 || k == 0) return SLIM_OK;
  SLIM_TRY(check_rows<T>(w));
  SLIM_TRY(check_mat(codes, scales, false));
  SLIM_TRY(check_mat(codes_t, scales_t, true));
  return finish(pack_weight<T>(w, codes, scales, codes_t, scales_t, n, k, st), st);
}

template <typename T>
slim_status run_rms_norm(const void *x, const void *res, const float *gamma, float eps, void *h, float *rstd,
                         void *y_codes, void *y_scales, void *h_codes, void *h_scales, int rows, int cols,
                         cudaStream_t st) {
  NvtxRange range("slim_q8_rms_norm");
  SLIM_TRY(check_size(rows, cols));
  if (cols < 1 || !(eps >= 0.f)) return SLIM_ERR_INVALID_ARG;
  if (cols > kMaxNormCols) return SLIM_ERR_UNSUPPORTED;
  if (rows == 0) return SLIM_OK;
  SLIM_TRY(check_rows<T>(x));
  SLIM_TRY(check_rows<float>(gamma));
  if (!aligned(res, sizeof(T)) || !aligned(h, sizeof(T)) || !aligned(rstd, 4)) return SLIM_ERR_UNSUPPORTED;
  SLIM_TRY(check_mat(y_codes, y_scales, false));
  SLIM_TRY(check_mat(h_codes, h_scales, true));
  return finish(rms_norm<T>(x, res, gamma, eps, h, rstd, y_codes, y_scales, h_codes, h_scales, rows, cols, st), st);
}

template <typename T>
slim_status run_rms_norm_bwd(const void *dy, const void *h, const void *h_codes, const void *h_scales,
                             const float *rstd, const float *gamma, const void *dres, void *dh, float *dgamma,
                             void *workspace, size_t workspace_bytes, int rows, int cols, cudaStream_t st) {
  NvtxRange range("slim_q8_rms_norm_bwd");
  SLIM_TRY(check_size(rows, cols));
  if (cols < 1) return SLIM_ERR_INVALID_ARG;
  if (cols > kMaxNormCols) return SLIM_ERR_UNSUPPORTED;
  if (!aligned(dgamma, 4)) return SLIM_ERR_UNSUPPORTED;
  if (rows == 0) {
    if (dgamma && cudaMemsetAsync(dgamma, 0, sizeof(float) * cols, st) != cudaSuccess) return SLIM_ERR_CUDA;
    return SLIM_OK;
  }
  if (!h == !h_codes) return SLIM_ERR_INVALID_ARG;
  SLIM_TRY(check_rows<T>(dy));
  SLIM_TRY(check_rows<T>(dh));
  SLIM_TRY(check_rows<float>(rstd));
  SLIM_TRY(check_rows<float>(gamma));
  if (!aligned(h, sizeof(T)) || !aligned(dres, sizeof(T))) return SLIM_ERR_UNSUPPORTED;
  SLIM_TRY(check_mat(h_codes, h_scales, true));
  if (dgamma) {
    if (!workspace || workspace_bytes < rms_norm_bwd_workspace(rows, cols)) return SLIM_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SLIM_ERR_UNSUPPORTED;
  }
  return finish(
      rms_norm_bwd<T>(dy, h, h_codes, h_scales, rstd, gamma, dres, dh, dgamma, workspace, rows, cols, st), st);
}

template <typename T>
slim_status run_gelu_bwd(const void *da, const void *z_codes, const void *z_scales, void *dz, void *dz_codes,
                         void *dz_scales, int rows, int cols, cudaStream_t st) {
  NvtxRange range("slim_q8_gelu_bwd");
  SLIM_TRY(check_size(rows, cols));
  if (rows == 0 || cols == 0) return SLIM_OK;
  SLIM_TRY(check_rows<T>(da));
  SLIM_TRY(check_rows<T>(dz));
  SLIM_TRY(check_mat(z_codes, z_scales, false));
  SLIM_TRY(check_mat(dz_codes, dz_scales, true));
  return finish(gelu_bwd<T>(da, z_codes, z_scales, dz, dz_codes, dz_scales, rows, cols, st), st);
}

slim_status run_matmul(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales,
                       void *out, bool f32, int rows, int n, int k, cudaStream_t st) {
  NvtxRange range("slim_q8_matmul");
  SLIM_TRY(check_size(rows, k));
  SLIM_TRY(check_size(n, k));
  if (k > kMaxK || blocks_of(rows) > kMaxRowTiles || blocks_of(n) > kMaxRowTiles) return SLIM_ERR_UNSUPPORTED;
  if (rows == 0 || n == 0) return SLIM_OK;
  SLIM_TRY(f32 ? check_rows<float>(out) : check_rows<__nv_bfloat16>(out));
  if (k == 0) {
    const size_t bytes = (size_t)rows * n * (f32 ? 4 : 2);
    return finish(cudaMemsetAsync(out, 0, bytes, st), st);
  }
  SLIM_TRY(check_mat(a_codes, a_scales, false));
  SLIM_TRY(check_mat(b_codes, b_scales, false));
  int *status = device_status_ptr();
  if (!status) return SLIM_ERR_CUDA;
  return finish(matmul(a_codes, a_scales, b_codes, b_scales, out, f32, rows, n, k, status, st), st);
}

}  // namespace
}  // namespace q8
}  // namespace slim

using namespace slim::q8;
using bf16 = __nv_bfloat16;

extern "C" {

size_t slim_q8_codes_bytes(int rows, int cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return (size_t)rows * blocks_of(cols) * kBlock;
}

size_t slim_q8_scales_bytes(int rows, int cols, int block_rows) {
  if (rows <= 0 || cols <= 0 || (block_rows != 1 && block_rows != kBlock)) return 0;
  return (size_t)(block_rows == 1 ? rows : blocks_of(rows)) * scale_pitch(cols);
}

slim_status slim_q8_quantize(const void *x, void *codes, void *scales, int rows, int cols, slim_stream_t stream) {
  return run_quantize<bf16>(x, codes, scales, nullptr, nullptr, false, rows, cols, (cudaStream_t)stream);
}

slim_status slim_q8_quantize_f32(const float *x, void *codes, void *scales, int rows, int cols,
                                 slim_stream_t stream) {
  return run_quantize<float>(x, codes, scales, nullptr, nullptr, false, rows, cols, (cudaStream_t)stream);
}

slim_status slim_q8_dequantize(const void *codes, const void *scales, void *x, int rows, int cols, int block_rows,
                               slim_stream_t stream) {
  return run_dequantize<bf16>(codes, scales, x, rows, cols, block_rows, (cudaStream_t)stream);
}

slim_status slim_q8_dequantize_f32(const void *codes, const void *scales, float *x, int rows, int cols,
                                   int block_rows, slim_stream_t stream) {
  return run_dequantize<float>(codes, scales, x, rows, cols, block_rows, (cudaStream_t)stream);
}

slim_status slim_q8_pack_weight(const void *w, void *codes, void *scales, void *codes_t, void *scales_t, int n,
                                int k, slim_stream_t stream) {
  return run_pack_weight<bf16>(w, codes, scales, codes_t, scales_t, n, k, (cudaStream_t)stream);
}

slim_status slim_q8_pack_weight_f32(const float *w, void *codes, void *scales, void *codes_t, void *scales_t, int n,
                                    int k, slim_stream_t stream) {
  return run_pack_weight<float>(w, codes, scales, codes_t, scales_t, n, k, (cudaStream_t)stream);
}

slim_status slim_q8_rms_norm(const void *x, const void *res, const float *gamma, float eps, void *h, float *rstd,
                             void *y_codes, void *y_scales, void *h_codes, void *h_scales, int rows, int cols,
                             slim_stream_t stream) {
  return run_rms_norm<bf16>(x, res, gamma, eps, h, rstd, y_codes, y_scales, h_codes, h_scales, rows, cols,
                            (cudaStream_t)stream);
}

slim_status slim_q8_rms_norm_f32(const float *x, const float *res, const float *gamma, float eps, float *h,
                                 float *rstd, void *y_codes, void *y_scales, void *h_codes, void *h_scales, int rows,
                                 int cols, slim_stream_t stream) {
  return run_rms_norm<float>(x, res, gamma, eps, h, rstd, y_codes, y_scales, h_codes, h_scales, rows, cols,
                             (cudaStream_t)stream);
}

slim_status slim_q8_rms_norm_bwd(const void *dy, const void *h, const void *h_codes, const void *h_scales,
                                 const float *rstd, const float *gamma, const void *dres, void *dh, float *dgamma,
                                 void *workspace, size_t workspace_bytes, int rows, int cols, slim_stream_t stream) {
  return run_rms_norm_bwd<bf16>(dy, h, h_codes, h_scales, rstd, gamma, dres, dh, dgamma, workspace, workspace_bytes,
                                rows, cols, (cudaStream_t)stream);
}

slim_status slim_q8_rms_norm_bwd_f32(const float *dy, const float *h, const void *h_codes, const void *h_scales,
                                     const float *rstd, const float *gamma, const float *dres, float *dh,
                                     float *dgamma, void *workspace, size_t workspace_bytes, int rows, int cols,
                                     slim_stream_t stream) {
  return run_rms_norm_bwd<float>(dy, h, h_codes, h_scales, rstd, gamma, dres, dh, dgamma, workspace, workspace_bytes,
                                 rows, cols, (cudaStream_t)stream);
}

size_t slim_q8_rms_norm_bwd_workspace_bytes(int rows, int cols) {
  if (rows <= 0 || cols < 1 || cols > kMaxNormCols) return 0;
  return rms_norm_bwd_workspace(rows, cols);
}

slim_status slim_q8_gelu(const void *z, void *a_codes, void *a_scales, void *z_codes, void *z_scales, int rows,
                         int cols, slim_stream_t stream) {
  return run_quantize<bf16>(z, a_codes, a_scales, z_codes, z_scales, true, rows, cols, (cudaStream_t)stream);
}

slim_status slim_q8_gelu_f32(const float *z, void *a_codes, void *a_scales, void *z_codes, void *z_scales, int rows,
                             int cols, slim_stream_t stream) {
  return run_quantize<float>(z, a_codes, a_scales, z_codes, z_scales, true, rows, cols, (cudaStream_t)stream);
}

slim_status slim_q8_gelu_bwd(const void *da, const void *z_codes, const void *z_scales, void *dz, void *dz_codes,
                             void *dz_scales, int rows, int cols, slim_stream_t stream) {
  return run_gelu_bwd<bf16>(da, z_codes, z_scales, dz, dz_codes, dz_scales, rows, cols, (cudaStream_t)stream);
}

slim_status slim_q8_gelu_bwd_f32(const float *da, const void *z_codes, const void *z_scales, float *dz,
                                 void *dz_codes, void *dz_scales, int rows, int cols, slim_stream_t stream) {
  return run_gelu_bwd<float>(da, z_codes, z_scales, dz, dz_codes, dz_scales, rows, cols, (cudaStream_t)stream);
}

slim_status slim_q8_matmul(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales,
                           void *out, int rows, int n, int k, slim_stream_t stream) {
  return run_matmul(a_codes, a_scales, b_codes, b_scales, out, false, rows, n, k, (cudaStream_t)stream);
}

slim_status slim_q8_matmul_f32(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales,
                               float *out, int rows, int n, int k, slim_stream_t stream) {
  return run_matmul(a_codes, a_scales, b_codes, b_scales, out, true, rows, n, k, (cudaStream_t)stream);
}

slim_status slim_q8_wgrad(const void *dy, const void *x_codes, const void *x_scales, float *dw, int accumulate,
                          void *workspace, size_t workspace_bytes, int rows, int n, int k, slim_stream_t stream) {
  NvtxRange range("slim_q8_wgrad");
  cudaStream_t st = (cudaStream_t)stream;
  SLIM_TRY(check_size(rows, k));
  SLIM_TRY(check_size(rows, n));
  SLIM_TRY(check_size(n, k));
  if (n == 0 || k == 0) return SLIM_OK;
  SLIM_TRY(check_rows<float>(dw));
  if (rows == 0) {
    if (!accumulate && cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)n * k, st) != cudaSuccess) return SLIM_ERR_CUDA;
    return SLIM_OK;
  }
  SLIM_TRY(check_rows<bf16>(dy));
  SLIM_TRY(check_mat(x_codes, x_scales, false));
  const size_t need = wgrad_workspace(rows, n, k);
  if (need && (!workspace || workspace_bytes < need)) return SLIM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return SLIM_ERR_UNSUPPORTED;
  int *status = slim::device_status_ptr();
  if (!status) return SLIM_ERR_CUDA;
  return finish(wgrad(dy, x_codes, x_scales, dw, accumulate != 0, workspace, rows, n, k, status, st), st);
}

size_t slim_q8_wgrad_workspace_bytes(int rows, int n, int k) {
  if (rows <= 0 || n <= 0 || k <= 0) return 0;
  return wgrad_workspace(rows, n, k);
}

}  // extern "C"
