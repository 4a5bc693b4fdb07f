// group_norm.cu -- group norm of each row's groups of columns (channels last),
// times the SiLU of a gate:
//   n = (x - mean) rstd,  rstd = (var + eps)^(-1/2)  over the group's columns,
//   y = (n gamma + beta) silu(z),  silu(z) = z s,  s = 1 / (1 + e^-z),
// and the gradients: with d = dy silu(z) and h = d gamma,
//   dx = rstd (h - mean(h) - n mean(h n)),  dz = dy (n gamma + beta) s (1 + z (1 - s)),
//   dgamma = sum over rows of d n,  dbeta = sum over rows of d.
//
// Memory-bound: x, z in and y out; dy, x, z in and dx, dz out.  A group lies in
// the registers of LANES lanes, N pieces of VEC columns each, so that every
// array is read once and the variance is taken from the centred values.  A
// warp stays on its columns and goes down the rows with the next row's loads
// under way, which also leaves gamma, beta and the two column sums in
// registers.
#include "kernels.h"
#include "q8_common.cuh"
#include "train.h"

namespace slim {
namespace {

using q8::load_raw8;
using q8::Raw8;
using q8::store8;
using q8::unpack8;

constexpr int kWarps = 8;

template <typename T, int VEC> struct Piece;  // VEC columns as they lie in memory
template <typename T> struct Piece<T, 8> {
  Raw8<T> raw;
  __device__ void load(const T *p, bool live) { raw = load_raw8<T, true>(p, live ? 8 : 0); }
  __device__ void get(float *v) const { unpack8(raw, v); }
};
template <typename T> struct Piece<T, 1> {
  T raw;
  __device__ void load(const T *p, bool live) { raw = live ? *p : from_f32<T>(0.f); }
  __device__ void get(float *v) const { v[0] = to_f32(raw); }
};
template <typename T, int VEC> __device__ __forceinline__ void put(T *p, bool live, const float *v) {
  if constexpr (VEC == 8) {
    store8<T, true>(p, live ? 8 : 0, v);
  } else if (live) {
    *p = from_f32<T>(v[0]);
  }
}

template <int LANES> __device__ __forceinline__ float group_sum(float s) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

struct Shape {
  int rows, cols, groups, width;
  float eps, inverse;  // 1 / width
  long long gate_row, dgate_row;  // elements from row to row of the gate and its gradient
};

// The columns of a lane: its group, and piece i at column group * width + (lane % LANES + i LANES) VEC.
template <int VEC, int LANES> struct Lane {
  int first, lane;
  bool live;
  __device__ Lane(const Shape &s) {
    const int group = blockIdx.x * (32 / LANES) + (threadIdx.x & 31) / LANES;
    lane = threadIdx.x % LANES;
    live = group < s.groups;
    first = (live ? group : 0) * s.width;
  }
  __device__ int at(int i) const { return (lane + i * LANES) * VEC; }
  __device__ bool has(const Shape &s, int i) const { return live && at(i) < s.width; }
};

// mean and rstd; v becomes the centred values
template <int VEC, int LANES, int N>
__device__ __forceinline__ float centre(const Shape &s, const Lane<VEC, LANES> &l, float v[N][VEC]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum += v[i][j];
  const float mean = group_sum<LANES>(sum) * s.inverse;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      v[i][j] = l.has(s, i) ? v[i][j] - mean : 0.f;
      sq = fmaf(v[i][j], v[i][j], sq);
    }
  return rsqrtf(fmaf(group_sum<LANES>(sq), s.inverse, s.eps));
}

template <typename T, int VEC, int LANES, int N>
__global__ void __launch_bounds__(kWarps * 32)
    forward_kernel(const T *__restrict__ x, const float *__restrict__ gamma, const float *__restrict__ beta,
                   const T *__restrict__ gate, T *__restrict__ y, Shape s) {
  const Lane<VEC, LANES> l(s);
  float ga[N][VEC], be[N][VEC];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      ga[i][j] = l.has(s, i) ? gamma[l.first + l.at(i) + j] : 0.f;
      be[i][j] = l.has(s, i) ? beta[l.first + l.at(i) + j] : 0.f;
    }
  const int step = gridDim.y * kWarps;
  int row = blockIdx.y * kWarps + (threadIdx.x >> 5);
  Piece<T, VEC> px[N], pz[N];
  auto load = [&](int r) {
    const long long at = (long long)r * s.cols + l.first;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      px[i].load(x + at + l.at(i), r < s.rows && l.has(s, i));
      if (gate) pz[i].load(gate + (long long)r * s.gate_row + l.first + l.at(i), r < s.rows && l.has(s, i));
    }
  };
  load(row);
  for (; row < s.rows; row += step) {
    float v[N][VEC], z[N][VEC];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      px[i].get(v[i]);
      if (gate) pz[i].get(z[i]);
    }
    load(row + step < s.rows ? row + step : s.rows);
    const float rstd = centre<VEC, LANES, N>(s, l, v);
    const long long at = (long long)row * s.cols + l.first;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] = fmaf(v[i][j] * rstd, ga[i][j], be[i][j]);
        if (gate) v[i][j] *= z[i][j] * sigmoid(z[i][j]);
      }
      put<T, VEC>(y + at + l.at(i), l.has(s, i), v[i]);
    }
  }
}

template <typename T, int VEC, int LANES, int N>
__global__ void __launch_bounds__(kWarps * 32)
    backward_kernel(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ gamma,
                    const float *__restrict__ beta, const T *__restrict__ gate, T *__restrict__ dx,
                    T *__restrict__ dgate, float *__restrict__ parts, Shape s) {
  __shared__ float sums[kWarps][2][32 * VEC];
  const Lane<VEC, LANES> l(s);
  float ga[N][VEC], be[N][VEC], dga[N][VEC] = {}, dbe[N][VEC] = {};
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      ga[i][j] = l.has(s, i) ? gamma[l.first + l.at(i) + j] : 0.f;
      be[i][j] = l.has(s, i) ? beta[l.first + l.at(i) + j] : 0.f;
    }
  const int step = gridDim.y * kWarps, warp = threadIdx.x >> 5;
  int row = blockIdx.y * kWarps + warp;
  Piece<T, VEC> px[N], pz[N], pd[N];
  auto load = [&](int r) {
    const long long at = (long long)r * s.cols + l.first;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool live = r < s.rows && l.has(s, i);
      px[i].load(x + at + l.at(i), live);
      pd[i].load(dy + at + l.at(i), live);
      if (gate) pz[i].load(gate + (long long)r * s.gate_row + l.first + l.at(i), live);
    }
  };
  load(row);
  for (; row < s.rows; row += step) {
    float v[N][VEC], d[N][VEC], z[N][VEC];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      px[i].get(v[i]);
      pd[i].get(d[i]);
      if (gate) pz[i].get(z[i]);
    }
    load(row + step < s.rows ? row + step : s.rows);
    const float rstd = centre<VEC, LANES, N>(s, l, v);
    const long long at = (long long)row * s.cols + l.first;
    float h0 = 0.f, h1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float n = v[i][j] * rstd;
        v[i][j] = n;
        if (gate) {
          const float zv = z[i][j], sg = sigmoid(zv);
          z[i][j] = d[i][j] * fmaf(n, ga[i][j], be[i][j]) * sg * fmaf(zv, 1.f - sg, 1.f);
          d[i][j] *= zv * sg;
        }
        dga[i][j] = fmaf(d[i][j], n, dga[i][j]);
        dbe[i][j] += d[i][j];
        d[i][j] *= ga[i][j];
        h0 += d[i][j];
        h1 = fmaf(d[i][j], n, h1);
      }
      if (gate) put<T, VEC>(dgate + (long long)row * s.dgate_row + l.first + l.at(i), l.has(s, i), z[i]);
    }
    h0 = group_sum<LANES>(h0) * s.inverse;
    h1 = group_sum<LANES>(h1) * s.inverse;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[i][j] = rstd * (d[i][j] - fmaf(v[i][j], h1, h0));
      put<T, VEC>(dx + at + l.at(i), l.has(s, i), d[i]);
    }
  }
  if (!parts) return;
  // the warps' sums of a column, in the order of the warps
  for (int i = 0; i < N; ++i) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      sums[warp][0][(threadIdx.x & 31) * VEC + j] = dga[i][j];
      sums[warp][1][(threadIdx.x & 31) * VEC + j] = dbe[i][j];
    }
    __syncthreads();
    if (warp < 2)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float t = 0.f;
        for (int k = 0; k < kWarps; ++k) t += sums[k][warp][(threadIdx.x & 31) * VEC + j];
        if (l.has(s, i)) parts[((size_t)blockIdx.y * 2 + warp) * s.cols + l.first + l.at(i) + j] = t;
      }
  }
}

// Groups wider than a warp's registers hold (over 1024 columns, or over 512
// where they are read one by one): a warp reads its group again from the
// caches for each of the sums.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    wide_forward_kernel(const T *__restrict__ x, const float *__restrict__ gamma, const float *__restrict__ beta,
                        const T *__restrict__ gate, T *__restrict__ y, Shape s) {
  const int lane = threadIdx.x & 31, first = blockIdx.x * s.width;
  for (int row = blockIdx.y * kWarps + (threadIdx.x >> 5); row < s.rows; row += gridDim.y * kWarps) {
    const long long at = (long long)row * s.cols + first, gat = (long long)row * s.gate_row + first;
    float sum = 0.f, sq = 0.f;
    for (int c = lane; c < s.width; c += 32) sum += to_f32(x[at + c]);
    const float mean = group_sum<32>(sum) * s.inverse;
    for (int c = lane; c < s.width; c += 32) {
      const float v = to_f32(x[at + c]) - mean;
      sq = fmaf(v, v, sq);
    }
    const float rstd = rsqrtf(fmaf(group_sum<32>(sq), s.inverse, s.eps));
    for (int c = lane; c < s.width; c += 32) {
      float v = fmaf((to_f32(x[at + c]) - mean) * rstd, gamma[first + c], beta[first + c]);
      if (gate) {
        const float z = to_f32(gate[gat + c]);
        v *= z * sigmoid(z);
      }
      y[at + c] = from_f32<T>(v);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    wide_backward_kernel(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ gamma,
                         const float *__restrict__ beta, const T *__restrict__ gate, T *__restrict__ dx,
                         T *__restrict__ dgate, float *__restrict__ parts, Shape s) {
  extern __shared__ float stats[];  // mean, rstd, mean(h), mean(h n) of kWarps rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.x * s.width;
  const int batches = (s.rows + gridDim.y * kWarps - 1) / (gridDim.y * kWarps);
  float *own = parts ? parts + (size_t)blockIdx.y * 2 * s.cols + first : nullptr;
  for (int b = 0; b < batches; ++b) {
    const int row0 = (b * gridDim.y + blockIdx.y) * kWarps, row = row0 + warp;
    const long long at = (long long)row * s.cols + first, gat = (long long)row * s.gate_row + first;
    if (row < s.rows) {
      float sum = 0.f, sq = 0.f, h0 = 0.f, h1 = 0.f;
      for (int c = lane; c < s.width; c += 32) sum += to_f32(x[at + c]);
      const float mean = group_sum<32>(sum) * s.inverse;
      for (int c = lane; c < s.width; c += 32) {
        const float v = to_f32(x[at + c]) - mean;
        sq = fmaf(v, v, sq);
      }
      const float rstd = rsqrtf(fmaf(group_sum<32>(sq), s.inverse, s.eps));
      for (int c = lane; c < s.width; c += 32) {
        const float n = (to_f32(x[at + c]) - mean) * rstd;
        float d = to_f32(dy[at + c]);
        if (gate) {
          const float z = to_f32(gate[gat + c]), sg = sigmoid(z);
          dgate[(long long)row * s.dgate_row + first + c] = from_f32<T>(d * fmaf(n, gamma[first + c], beta[first + c]) * sg * fmaf(z, 1.f - sg, 1.f));
          d *= z * sg;
        }
        d *= gamma[first + c];
        h0 += d;
        h1 = fmaf(d, n, h1);
      }
      h0 = group_sum<32>(h0) * s.inverse;
      h1 = group_sum<32>(h1) * s.inverse;
      for (int c = lane; c < s.width; c += 32) {
        const float n = (to_f32(x[at + c]) - mean) * rstd;
        float d = to_f32(dy[at + c]) * gamma[first + c];
        if (gate) {
          const float z = to_f32(gate[gat + c]);
          d *= z * sigmoid(z);
        }
        dx[at + c] = from_f32<T>(rstd * (d - fmaf(n, h1, h0)));
      }
      if (lane == 0) {
        stats[2 * warp] = mean;
        stats[2 * warp + 1] = rstd;
      }
    }
    if (!parts) continue;
    __syncthreads();
    // the batch's rows of each column, added to this block's sums
    for (int c = threadIdx.x; c < s.width; c += kWarps * 32) {
      float a = b ? own[c] : 0.f, e = b ? own[s.cols + c] : 0.f;
      for (int k = 0; k < kWarps && row0 + k < s.rows; ++k) {
        const long long i = (long long)(row0 + k) * s.cols + first + c;
        float d = to_f32(dy[i]);
        if (gate) {
          const float z = to_f32(gate[(long long)(row0 + k) * s.gate_row + first + c]);
          d *= z * sigmoid(z);
        }
        a = fmaf(d, (to_f32(x[i]) - stats[2 * k]) * stats[2 * k + 1], a);
        e += d;
      }
      own[c] = a;
      own[s.cols + c] = e;
    }
    __syncthreads();
  }
}

// dgamma and dbeta: the blocks' sums of each column in the order of the blocks.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float *__restrict__ parts, int n, int cols,
                                                        float *__restrict__ dgamma, float *__restrict__ dbeta) {
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), which = blockIdx.y, k0 = threadIdx.x >> 5;
  __shared__ double sums[8][32];
  double t = 0.0;
  if (c < cols)
    for (int k = k0; k < n; k += 8) t += parts[((size_t)k * 2 + which) * cols + c];
  sums[k0][threadIdx.x & 31] = t;
  __syncthreads();
  if (k0 == 0 && c < cols) {
    for (int k = 1; k < 8; ++k) t += sums[k][threadIdx.x];
    float *out = which ? dbeta : dgamma;
    if (out) out[c] = (float)t;
  }
}

// Blocks along the rows: at most as many as run at a time, `each` of eight
// warps an SM, and no more than the rows need.  At 65536 x 1024 the forward
// takes 67 us with four and 89 with two, the backward, whose registers leave
// room for two, 131 with two and 136 with four.
constexpr int kForwardBlocks = 4, kBackwardBlocks = 2;
int row_blocks(int rows, int slabs, int each) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int most = (each * sms + slabs - 1) / slabs, need = (rows + kWarps - 1) / kWarps;
  return max(1, min(min(most, need), 65535));
}

// Columns of a warp: groups of up to 256 columns with lanes a power of two
// share a warp, others have one each.
struct Cut {
  int vec, lanes, n;  // n = 0: wide
  int slabs(int groups) const { return (groups + 32 / lanes - 1) / (32 / lanes); }
};

Cut cut_for(int cols, int groups, bool vec) {
  const int width = cols / groups;
  if (vec && width % 8 == 0) {
    for (int lanes = 1; lanes <= 32; lanes *= 2)
      if (width <= lanes * 8) return Cut{8, lanes, 1};
    if (width <= 512) return Cut{8, 32, 2};
    if (width <= 1024) return Cut{8, 32, 4};
  } else {
    for (int lanes = 8; lanes <= 32; lanes *= 2)
      if (width <= lanes) return Cut{1, lanes, 1};
    if (width <= 128) return Cut{1, 32, 4};
    if (width <= 512) return Cut{1, 32, 16};
  }
  return Cut{1, 32, 0};
}

#define SLIM_GN_CUTS(M)                                                                                   \
  M(8, 1, 1) M(8, 2, 1) M(8, 4, 1) M(8, 8, 1) M(8, 16, 1) M(8, 32, 1) M(8, 32, 2) M(8, 32, 4) M(1, 8, 1)  \
  M(1, 16, 1) M(1, 32, 1) M(1, 32, 4) M(1, 32, 16)

Shape shape_of(int rows, int cols, int groups, float eps, long long gate_row, long long dgate_row) {
  return Shape{rows, cols, groups, cols / groups, eps, 1.f / (float)(cols / groups), gate_row, dgate_row};
}

}  // namespace

template <typename T>
cudaError_t group_norm(const void *x, const float *gamma, const float *beta, const void *gate, long long gate_row,
                       float eps, void *y, int rows, int cols, int groups, cudaStream_t st) {
  ProfScope ps("group_norm", st);
  const Shape s = shape_of(rows, cols, groups, eps, gate_row, 0);
  const Cut c = cut_for(cols, groups, gate_row % 8 == 0 && q8::vector_rows(cols, {x, gate, y}));
  const dim3 grid(c.slabs(groups), row_blocks(rows, c.slabs(groups), kForwardBlocks));
  const T *xp = static_cast<const T *>(x), *zp = static_cast<const T *>(gate);
  T *yp = static_cast<T *>(y);
  if (c.n == 0) {
    wide_forward_kernel<T><<<grid, kWarps * 32, 0, st>>>(xp, gamma, beta, zp, yp, s);
    return cudaGetLastError();
  }
#define SLIM_GN_RUN(V, L, N)                                                                    \
  if (c.vec == V && c.lanes == L && c.n == N) {                                                 \
    forward_kernel<T, V, L, N><<<grid, kWarps * 32, 0, st>>>(xp, gamma, beta, zp, yp, s);       \
    return cudaGetLastError();                                                                  \
  }
  SLIM_GN_CUTS(SLIM_GN_RUN)
#undef SLIM_GN_RUN
  return cudaErrorInvalidValue;
}

// Blocks' column sums, for the cut with the most blocks along the rows.
size_t group_norm_bwd_workspace(int rows, int cols, int groups) {
  int most = 1;
  for (bool vec : {false, true}) most = max(most, row_blocks(rows, cut_for(cols, groups, vec).slabs(groups), kBackwardBlocks));
  return sizeof(float) * 2 * (size_t)most * cols;
}

template <typename T>
cudaError_t group_norm_bwd(const void *dy, const void *x, const float *gamma, const float *beta, const void *gate,
                           long long gate_row, float eps, void *dx, void *dgate, long long dgate_row, float *dgamma, float *dbeta, void *workspace, int rows,
                           int cols, int groups, cudaStream_t st) {
  ProfScope ps("group_norm_bwd", st);
  const Shape s = shape_of(rows, cols, groups, eps, gate_row, dgate_row);
  const Cut c = cut_for(cols, groups,
                        gate_row % 8 == 0 && dgate_row % 8 == 0 && q8::vector_rows(cols, {dy, x, gate, dx, dgate}));
  const dim3 grid(c.slabs(groups), row_blocks(rows, c.slabs(groups), kBackwardBlocks));
  const T *dp = static_cast<const T *>(dy), *xp = static_cast<const T *>(x), *zp = static_cast<const T *>(gate);
  T *dxp = static_cast<T *>(dx), *dzp = static_cast<T *>(dgate);
  float *parts = dgamma || dbeta ? static_cast<float *>(workspace) : nullptr;
  bool done = false;
  if (c.n == 0) {
    wide_backward_kernel<T><<<grid, kWarps * 32, sizeof(float) * 2 * kWarps, st>>>(dp, xp, gamma, beta, zp, dxp, dzp,
                                                                                   parts, s);
    done = true;
  }
#define SLIM_GN_RUN(V, L, N)                                                                                    \
  if (!done && c.vec == V && c.lanes == L && c.n == N) {                                                        \
    backward_kernel<T, V, L, N><<<grid, kWarps * 32, 0, st>>>(dp, xp, gamma, beta, zp, dxp, dzp, parts, s);     \
    done = true;                                                                                                \
  }
  SLIM_GN_CUTS(SLIM_GN_RUN)
#undef SLIM_GN_RUN
  cudaError_t e = done ? cudaGetLastError() : cudaErrorInvalidValue;
  if (e != cudaSuccess || !parts) return e;
  sum_parts_kernel<<<dim3((cols + 31) / 32, 2), 256, 0, st>>>(parts, grid.y, cols, dgamma, dbeta);
  return cudaGetLastError();
}

#define SLIM_GN_FOR(T)                                                                                             \
  template cudaError_t group_norm<T>(const void *, const float *, const float *, const void *, long long, float,   \
                                     void *, int, int, int, cudaStream_t);                                         \
  template cudaError_t group_norm_bwd<T>(const void *, const void *, const float *, const float *, const void *,   \
                                         long long, float, void *, void *, long long, float *, float *, void *,    \
                                         int, int, int,                                                            \
                                         cudaStream_t);
SLIM_GN_FOR(float)
SLIM_GN_FOR(__nv_bfloat16)

}  // namespace slim
