// train.h -- host-side entry points of the group norm and of AdamW (arguments
// already checked; every call only enqueues work on `st`).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "../../include/slim_attn.h"

namespace slim {

// group_norm.cu.  gate: NULL, or z, rows gate_row elements apart.
template <typename T>
cudaError_t group_norm(const void *x, const float *gamma, const float *beta, const void *gate, long long gate_row,
                       float eps, void *y, int rows, int cols, int groups, cudaStream_t st);
size_t group_norm_bwd_workspace(int rows, int cols, int groups);
template <typename T>
cudaError_t group_norm_bwd(const void *dy, const void *x, const float *gamma, const float *beta, const void *gate,
                           long long gate_row, float eps, void *dx, void *dgate, long long dgate_row, float *dgamma, float *dbeta, void *workspace, int rows,
                           int cols, int groups, cudaStream_t st);

// adamw.cu
cudaError_t adamw(const slim_adamw_tensor *tensors, int n, const slim_adamw_options &o, bool g_f32, int *count,
                  cudaStream_t st);

}  // namespace slim
