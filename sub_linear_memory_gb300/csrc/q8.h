// q8.h -- host-side entry points of the 8-bit layer operators (shapes already
// checked; every call only enqueues work on `st`).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace slim {
namespace q8 {

// q8_rows.cu.  z_codes, h_codes, dz_codes, codes_t: NULL where not wanted.
template <typename T>
cudaError_t quantize(const void *x, void *codes, void *scales, void *z_codes, void *z_scales, bool gelu, int rows,
                     int cols, cudaStream_t st);
template <typename T>
cudaError_t dequantize(const void *codes, const void *scales, void *x, int rows, int cols, int block_rows,
                       cudaStream_t st);
template <typename T>
cudaError_t gelu_bwd(const void *da, const void *z_codes, const void *z_scales, void *dz, void *dz_codes,
                     void *dz_scales, int rows, int cols, cudaStream_t st);
template <typename T>
cudaError_t pack_weight(const void *w, void *codes, void *scales, void *codes_t, void *scales_t, int n, int k,
                        cudaStream_t st);

// q8_norm.cu
template <typename T>
cudaError_t rms_norm(const void *x, const void *res, const float *gamma, float eps, void *h, float *rstd,
                     void *y_codes, void *y_scales, void *h_codes, void *h_scales, int rows, int cols,
                     cudaStream_t st);
size_t rms_norm_bwd_workspace(int rows, int cols);
template <typename T>
cudaError_t rms_norm_bwd(const void *dy, const void *h, const void *h_codes, const void *h_scales, const float *rstd,
                         const float *gamma, const void *dres, void *dh, float *dgamma, void *workspace, int rows,
                         int cols, cudaStream_t st);

// q8_matmul.cu: out (bf16 or fp32) = a . b^T.
cudaError_t matmul(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales, void *out,
                   bool f32, int rows, int n, int k, int *status, cudaStream_t st);

// q8_wgrad.cu: dw (+)= dy^T . x.
size_t wgrad_workspace(int rows, int n, int k);
cudaError_t wgrad(const void *dy, const void *x_codes, const void *x_scales, float *dw, bool accumulate,
                  void *workspace, int rows, int n, int k, int *status, cudaStream_t st);

}  // namespace q8
}  // namespace slim
