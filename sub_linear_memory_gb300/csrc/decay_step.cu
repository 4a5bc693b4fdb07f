// decay_step.cu -- linear attention with a decay, one token of each sequence:
//   S = lambda S + k v^T,  o = scale q^T S
// for the state of the sequence's place and every query head of a key-value
// head.  The state is read and written once (8 dk dv bytes a head), which is
// all that counts.
#include "decay_common.cuh"
#include "kernels.h"

namespace slim {
namespace decay {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 8;

// The row that has this slot: the first of those that name it.
__device__ __forceinline__ bool taken_before(const int *slots, int row, int slot) {
  int found = 0;
  for (int i = threadIdx.x; i < row; i += kThreads) found |= slots[i] == slot;
  return __syncthreads_or(found) != 0;
}

// A block has one key-value head of one row; VEC columns and every
// (threads / (dv / VEC))-th row of the state are one thread's, kBatch rows at a
// time with their loads ahead of the stores: a row at a time, each load behind
// the last row's store, 128 rows of 16 heads of 64 took 22 us a call, this way
// 17.5, and 129 of 12 / 4 heads of 128 30 and 17 (their states' bytes: 10).
template <typename T, int VEC, int MOST>
__global__ void __launch_bounds__(kThreads) step_kernel(Step s) {
  extern __shared__ float sm[];
  const int head = blockIdx.x % s.heads, row = blockIdx.x / s.heads, t = threadIdx.x;
  float *k = sm, *q = k + s.dk, *part = q + s.groups * s.dk;  // part [thread rows][groups][dv]
  const int cols = (s.dv + VEC - 1) / VEC, lanes = min(cols, kThreads), rows = kThreads / lanes;
  long long at = row;
  if (s.slots) {
    at = s.slots[row];
    if (at < 0 || at >= s.places || taken_before(s.slots, row, (int)at)) at = -1;
  }
  const T *kp = static_cast<const T *>(s.k) + row * s.k_row + (long long)head * s.dk;
  const T *qp = static_cast<const T *>(s.q) + row * s.q_row + (long long)head * s.groups * s.dk;
  const T *vp = static_cast<const T *>(s.v) + row * s.v_row + (long long)head * s.dv;
  T *op = static_cast<T *>(s.o) + row * s.o_row + (long long)head * s.groups * s.dv;
  if (at < 0) {  // a row without a place
    for (int i = t; i < s.groups * s.dv; i += kThreads) op[i] = from_f32<T>(0.f);
    return;
  }
  for (int i = t; i < s.dk; i += kThreads) k[i] = to_f32(kp[i]);
  for (int i = t; i < s.groups * s.dk; i += kThreads) q[i] = to_f32(qp[i]) * s.scale;
  __syncthreads();
  const float lambda = exp2f(log2_decay(s.log_decay, head));
  float *state = s.state + ((size_t)at * s.heads + head) * s.dk * s.dv;
  const int r0 = t / lanes, c0 = t % lanes;
  for (int col = c0; col < cols; col += lanes) {
    if (r0 >= rows) continue;
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = col * VEC + i < s.dv ? to_f32(vp[col * VEC + i]) : 0.f;
    for (int g0 = 0; g0 < s.groups; g0 += MOST) {
      float acc[MOST][VEC] = {};
      for (int rb = r0; rb < s.dk; rb += rows * kBatch) {
        float x[kBatch][VEC];
        float *p = state + (size_t)rb * s.dv + col * VEC;
        const size_t next = (size_t)rows * s.dv;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (rb + b * rows >= s.dk) continue;
          if constexpr (VEC == 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + b * next);
            x[b][0] = f.x, x[b][1] = f.y, x[b][2] = f.z, x[b][3] = f.w;
          } else {
            x[b][0] = p[b * next];
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int r = rb + b * rows;
          if (r >= s.dk) continue;
          if (g0 == 0) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[b][i] = fmaf(x[b][i], lambda, k[r] * v[i]);
            if constexpr (VEC == 4)
              *reinterpret_cast<float4 *>(p + b * next) = make_float4(x[b][0], x[b][1], x[b][2], x[b][3]);
            else
              p[b * next] = x[b][0];
          }
#pragma unroll
          for (int g = 0; g < MOST; ++g)
            if (g0 + g < s.groups) {
              const float qv = q[(g0 + g) * s.dk + r];
#pragma unroll
              for (int i = 0; i < VEC; ++i) acc[g][i] = fmaf(qv, x[b][i], acc[g][i]);
            }
        }
      }
#pragma unroll
      for (int g = 0; g < MOST; ++g)
        if (g0 + g < s.groups)
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (col * VEC + i < s.dv) part[(r0 * s.groups + g0 + g) * s.dv + col * VEC + i] = acc[g][i];
    }
  }
  __syncthreads();
  for (int i = t; i < s.groups * s.dv; i += kThreads) {
    float sum = 0.f;
    for (int r = 0; r < rows; ++r) sum += part[r * s.groups * s.dv + i];
    op[i] = from_f32<T>(sum);
  }
}

}  // namespace

template <typename T> cudaError_t step(const Step &s, cudaStream_t st) {
  ProfScope ps("decay_step", st);
  const bool vec = s.dv % 4 == 0 && (reinterpret_cast<uintptr_t>(s.state) & 15) == 0;
  const int cols = vec ? s.dv / 4 : s.dv, rows = kThreads / min(cols, kThreads);
  const size_t bytes = sizeof(float) * ((size_t)s.dk * (1 + s.groups) + (size_t)rows * s.groups * s.dv);
  // query heads of one pass over the state: one, or up to four
  const bool one = s.groups == 1;
  auto kernel = vec ? (one ? step_kernel<T, 4, 1> : step_kernel<T, 4, 4>) : (one ? step_kernel<T, 1, 1> : step_kernel<T, 1, 4>);
  if (bytes > 48 * 1024) {
    static SharedMemory allowed[4];
    cudaError_t e = allowed[2 * vec + one].allow(kernel, 200 * 1024);  // 64 query heads take 193 KB at most
    if (e != cudaSuccess) return e;
  }
  kernel<<<s.heads * s.rows, kThreads, bytes, st>>>(s);
  return cudaGetLastError();
}

template cudaError_t step<float>(const Step &, cudaStream_t);
template cudaError_t step<__nv_bfloat16>(const Step &, cudaStream_t);

}  // namespace decay
}  // namespace slim
