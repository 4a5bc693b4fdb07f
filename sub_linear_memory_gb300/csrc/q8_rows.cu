// q8_rows.cu -- row-wise operators with 8-bit rows: quantize, dequantize, the
// packed weight, GeLU and its backward, root-mean-square norm with the
// residual's addition and its backward.
//
// All of them are bound by memory: each element is read and written once, in
// 16-byte accesses, and 16 neighbouring threads hold one block of 128 columns
// in registers while they agree on its scale (four shuffles).
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "q8.h"
#include "q8_common.cuh"

namespace slim {
namespace q8 {
namespace {

// ---- GeLU -------------------------------------------------------------------

// The normal distribution function and density at z.
__device__ __forceinline__ void normal_parts(float z, float &cdf, float &pdf) {
  cdf = normcdff(z);
  pdf = 0.3989422804014327f * expf(-0.5f * z * z);
}

// ---- elementwise over blocks of 128 columns -----------------------------------

constexpr int kEltThreads = 256, kEltUnroll = 4;

// GELU: a = 8 bits of GeLU(x), z (where wanted) = 8 bits of x; otherwise
// a = 8 bits of x.
template <typename T, bool GELU, bool VEC>
__global__ void __launch_bounds__(kEltThreads) quantize_kernel(const T *x, Mat8 a, Mat8 z, Shape8 s,
                                                               unsigned blocks) {
  const int lane16 = threadIdx.x & (kVecs - 1);
  const unsigned first = blockIdx.x * (unsigned)(kEltThreads / kVecs * kEltUnroll) + threadIdx.x / kVecs;
  float v[kEltUnroll][kVec];
  unsigned row[kEltUnroll];
  int blk[kEltUnroll];
#pragma unroll
  for (int u = 0; u < kEltUnroll; ++u) {
    const unsigned b = first + u * (kEltThreads / kVecs);
    row[u] = b / (unsigned)s.nb;
    blk[u] = (int)(b - row[u] * (unsigned)s.nb);
    const int col = blk[u] * kBlock + lane16 * kVec;
    load8<T, VEC>(x + (size_t)row[u] * s.cols + col, b < blocks ? s.cols - col : 0, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kEltUnroll; ++u) {
    const bool live = first + u * (kEltThreads / kVecs) < blocks;
    if (GELU) {
      if (z.codes) put_block8(v[u], z, s, row[u], blk[u], lane16, live);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        float cdf, pdf;
        normal_parts(v[u][i], cdf, pdf);
        v[u][i] *= cdf;
      }
    }
    put_block8(v[u], a, s, row[u], blk[u], lane16, live);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kEltThreads) dequantize_kernel(const uint8_t *codes, const uint8_t *scales, T *x,
                                                                 Shape8 s, int row_shift, unsigned blocks) {
  const int lane16 = threadIdx.x & (kVecs - 1);
  const unsigned first = blockIdx.x * (unsigned)(kEltThreads / kVecs * kEltUnroll) + threadIdx.x / kVecs;
  uint2 c[kEltUnroll];
  int byte[kEltUnroll];
#pragma unroll
  for (int u = 0; u < kEltUnroll; ++u) {
    const unsigned b = first + u * (kEltThreads / kVecs);
    c[u] = make_uint2(0, 0);
    byte[u] = 127;
    if (b < blocks) {
      const unsigned row = b / (unsigned)s.nb;
      c[u] = __ldg(reinterpret_cast<const uint2 *>(codes + (size_t)b * kBlock + lane16 * kVec));
      byte[u] = __ldg(scales + (size_t)(row >> row_shift) * s.pitch + (b - row * (unsigned)s.nb));
    }
  }
#pragma unroll
  for (int u = 0; u < kEltUnroll; ++u) {
    const unsigned b = first + u * (kEltThreads / kVecs);
    if (b >= blocks) break;
    const unsigned row = b / (unsigned)s.nb;
    const int col = (int)(b - row * (unsigned)s.nb) * kBlock + lane16 * kVec;
    float v[kVec];
    decode8(c[u], scale_value(byte[u]), v);
    store8<T, VEC>(x + (size_t)row * s.cols + col, s.cols - col, v);
  }
}

// dz = da (Phi(z) + z phi(z)) at the checkpointed z, and the 8 bits of dz.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kEltThreads) gelu_bwd_kernel(const T *da, const uint8_t *codes,
                                                               const uint8_t *scales, T *dz, Mat8 q, Shape8 s,
                                                               unsigned blocks) {
  const int lane16 = threadIdx.x & (kVecs - 1);
  const unsigned first = blockIdx.x * (unsigned)(kEltThreads / kVecs * kEltUnroll) + threadIdx.x / kVecs;
  float v[kEltUnroll][kVec];
  uint2 c[kEltUnroll];
  int byte[kEltUnroll];
#pragma unroll
  for (int u = 0; u < kEltUnroll; ++u) {
    const unsigned b = first + u * (kEltThreads / kVecs), row = b / (unsigned)s.nb;
    const int blk = (int)(b - row * (unsigned)s.nb), col = blk * kBlock + lane16 * kVec;
    c[u] = make_uint2(0, 0);
    byte[u] = 127;
    if (b < blocks) {
      c[u] = __ldg(reinterpret_cast<const uint2 *>(codes + (size_t)b * kBlock + lane16 * kVec));
      byte[u] = __ldg(scales + (size_t)row * s.pitch + blk);
    }
    load8<T, VEC>(da + (size_t)row * s.cols + col, b < blocks ? s.cols - col : 0, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kEltUnroll; ++u) {
    const unsigned b = first + u * (kEltThreads / kVecs), row = b / (unsigned)s.nb;
    const int blk = (int)(b - row * (unsigned)s.nb), col = blk * kBlock + lane16 * kVec;
    float z[kVec];
    decode8(c[u], scale_value(byte[u]), z);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      float cdf, pdf;
      normal_parts(z[i], cdf, pdf);
      // the 8 bits are those of dz as it is stored
      v[u][i] = rounded<T>(v[u][i] * (cdf + z[i] * pdf));
    }
    if (!VEC) {  // columns past the row: a NaN block has NaN codes there too
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (i >= s.cols - col) v[u][i] = 0.f;
    } else if (col >= s.cols) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[u][i] = 0.f;
    }
    if (b < blocks) store8<T, VEC>(dz + (size_t)row * s.cols + col, s.cols - col, v[u]);
    if (q.codes) put_block8(v[u], q, s, row, blk, lane16, b < blocks);
  }
}

// ---- packed weight --------------------------------------------------------------

// One CTA for each 128 x 128 block: its 2048 chunks of 8 columns are in the
// registers of 256 threads, so the weight is read once; the transposed codes
// go through shared memory.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) pack_weight_kernel(const T *w, Mat8 q, Mat8 qt, int n, int k) {
  __shared__ uint32_t top[8];
  __shared__ uint8_t tile[kBlock][kBlock + 4];
  const Shape8 s = shape8(n, k), st = shape8(k, n);
  const int n0 = blockIdx.y * kBlock, bk = blockIdx.x, k0 = bk * kBlock;
  const int lane16 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  float v[8][kVec];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = n0 + r0 + 16 * i, col = k0 + lane16 * kVec;
    load8<T, VEC>(w + (size_t)row * k + col, row < n ? k - col : 0, v[i]);
    m = max(m, amax8(v[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
  m = top[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, top[i]);
  const int byte = scale_byte(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    const uint2 c = encode8(v[i], byte, n0 + r < n ? k - k0 - lane16 * kVec : 0);
    if (n0 + r < n) *reinterpret_cast<uint2 *>(q.codes + ((size_t)(n0 + r) * s.nb + bk) * kBlock + lane16 * kVec) = c;
    uint32_t *t = reinterpret_cast<uint32_t *>(&tile[r][lane16 * kVec]);
    t[0] = c.x;
    t[1] = c.y;
  }
  if (threadIdx.x == 0) {
    uint8_t *sc = q.scales + (size_t)blockIdx.y * s.pitch;
    sc[bk] = (uint8_t)byte;
    if (bk == s.nb - 1)
      for (int i = s.nb; i < s.pitch; ++i) sc[i] = 127;
    if (qt.codes) {
      uint8_t *tc = qt.scales + (size_t)bk * st.pitch;
      tc[blockIdx.y] = (uint8_t)byte;
      if ((int)blockIdx.y == st.nb - 1)
        for (int i = st.nb; i < st.pitch; ++i) tc[i] = 127;
    }
  }
  if (!qt.codes) return;
  __syncthreads();
  // column c of the tile is row k0 + c of the transpose
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = r0 + 16 * i;
    if (k0 + c >= k) continue;
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo |= (uint32_t)tile[lane16 * kVec + j][c] << (8 * j);
      hi |= (uint32_t)tile[lane16 * kVec + 4 + j][c] << (8 * j);
    }
    *reinterpret_cast<uint2 *>(qt.codes + ((size_t)(k0 + c) * st.nb + blockIdx.y) * kBlock + lane16 * kVec) =
        make_uint2(lo, hi);
  }
}

// ---- root-mean-square norm --------------------------------------------------------

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the W warps of a row's group; every thread of the CTA calls.
// `part` has a slot for each warp of the CTA, and is used by one call in two
// (the caller alternates two of them), so one barrier is enough.
template <int W>
__device__ __forceinline__ float group_sum(float x, float *part) {
  x = warp_sum(x);
  if (W == 1) return x;
  const int warp = threadIdx.x >> 5, first = warp / W * W;
  if ((threadIdx.x & 31) == 0) part[warp] = x;
  __syncthreads();
  x = part[first];
#pragma unroll
  for (int i = 1; i < W; ++i) x += part[first + i];
  return x;
}

template <int W> struct NormCfg {
  static constexpr int kThreads = W > 8 ? 32 * W : 256;
  static constexpr int kRows = kThreads / (32 * W);  // rows in flight in a CTA
};

// W warps hold a row, each thread NC chunks of 8 of its columns, in registers
// between the sum of squares and the quantization: h and y are formed from one
// read of x and res.
template <typename T, int W, int NC, bool VEC>
__global__ void __launch_bounds__(NormCfg<W>::kThreads) rms_norm_kernel(const T *x, const T *res, const float *gamma,
                                                                        float eps, T *h, float *rstd, Mat8 y, Mat8 hq,
                                                                        Shape8 s) {
  __shared__ float part[NormCfg<W>::kThreads / 32];
  const int l = threadIdx.x % (32 * W), lane16 = l & (kVecs - 1);
  const long long row = (long long)blockIdx.x * NormCfg<W>::kRows + threadIdx.x / (32 * W);
  const bool live = row < s.rows;
  const size_t at = (size_t)row * s.cols;
  float v[NC][kVec];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * 32 * W + l) * kVec;
    load8<T, VEC>(x + at + col, live ? s.cols - col : 0, v[c]);
  }
  if (res) {
    float r[NC][kVec];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * 32 * W + l) * kVec;
      load8<T, VEC>(res + at + col, live ? s.cols - col : 0, r[c]);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[c][i] = rounded<T>(v[c][i] + r[c][i]);
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * 32 * W + l) * kVec;
    if (h && live) store8<T, VEC>(h + at + col, s.cols - col, v[c]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss = fmaf(v[c][i], v[c][i], ss);
  }
  ss = group_sum<W>(ss, part);
  const float root = 1.f / sqrtf(ss / (float)s.cols + eps);
  if (rstd && live && l == 0) rstd[row] = root;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int chunk = c * 32 * W + l, blk = chunk / kVecs, col = chunk * kVec;
    const bool on = live && blk < s.nb;
    if (hq.codes) put_block8(v[c], hq, s, row, blk, lane16, on);
    float g[kVec];
    load8<float, VEC>(gamma + col, s.cols - col, g);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[c][i] = col + i < s.cols ? v[c][i] * root * g[i] : 0.f;
    put_block8(v[c], y, s, row, blk, lane16, on);
  }
}

// The gradients.  CTAs walk the rows; a thread's columns stay the same, so its
// share of dgamma is summed in registers, then over the CTA's groups through
// shared memory, and a CTA writes one partial row.
constexpr int kBwdCtas = 304;  // two for each of 152 SMs: fixed, so that the order of the sums is

template <typename T, int W, int NC, bool VEC>
__global__ void __launch_bounds__(NormCfg<W>::kThreads)
    rms_norm_bwd_kernel(const T *dy, const T *h, const uint8_t *hc, const uint8_t *hs, const float *rstd,
                        const float *gamma, const T *dres, T *dh, float *partial, Shape8 s) {
  extern __shared__ float columns[];
  __shared__ float part[2][NormCfg<W>::kThreads / 32];
  constexpr int kRows = NormCfg<W>::kRows;
  const int group = threadIdx.x / (32 * W), l = threadIdx.x % (32 * W);
  float acc[NC][kVec];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[c][i] = 0.f;
  int turn = 0;
  for (long long base = (long long)blockIdx.x * kRows; base < s.rows; base += (long long)gridDim.x * kRows) {
    const long long row = base + group;
    const bool live = row < s.rows;
    const size_t at = (size_t)row * s.cols;
    const float root = live ? rstd[row] : 0.f;
    float g[NC][kVec], n[NC][kVec], r[NC][kVec];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int chunk = c * 32 * W + l, col = chunk * kVec, left = live ? s.cols - col : 0;
      load8<T, VEC>(dy + at + col, left, g[c]);
      if (hc) {
        uint2 code = make_uint2(0, 0);
        int byte = 127;
        if (left > 0) {
          const int blk = chunk / kVecs;
          code = __ldg(reinterpret_cast<const uint2 *>(hc + ((size_t)row * s.nb + blk) * kBlock + (l & 15) * kVec));
          byte = __ldg(hs + (size_t)row * s.pitch + blk);
        }
        decode8(code, scale_value(byte), n[c]);
        if (!VEC) {  // columns past the row: a NaN block's scale reaches them
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (i >= left) n[c][i] = 0.f;
        }
      } else {
        load8<T, VEC>(h + at + col, left, n[c]);
      }
      if (dres) load8<T, VEC>(dres + at + col, left, r[c]);
    }
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * 32 * W + l) * kVec;
      float gm[kVec];
      load8<float, VEC>(gamma + col, s.cols - col, gm);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        n[c][i] *= root;
        acc[c][i] = fmaf(g[c][i], n[c][i], acc[c][i]);
        g[c][i] *= gm[i];
        dot = fmaf(g[c][i], n[c][i], dot);
      }
    }
    const float mean = group_sum<W>(dot, part[turn]) / (float)s.cols;
    turn ^= 1;
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int col = (c * 32 * W + l) * kVec;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float d = root * (g[c][i] - n[c][i] * mean);
          g[c][i] = dres ? d + r[c][i] : d;
        }
        store8<T, VEC>(dh + at + col, s.cols - col, g[c]);
      }
    }
  }
  if (!partial) return;
  float *out = partial + (size_t)blockIdx.x * s.nb * kBlock;
  for (int turn_of = 0; turn_of < kRows; ++turn_of) {
    if (kRows > 1) __syncthreads();
    if (group == turn_of) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int col = (c * 32 * W + l) * kVec;
        if (col < s.nb * kBlock) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            const float x = turn_of == 0 ? acc[c][i] : columns[col + i] + acc[c][i];
            if (turn_of == kRows - 1) out[col + i] = x;
            else columns[col + i] = x;
          }
        }
      }
    }
  }
}

// dgamma: the sum of the CTAs' partial rows, 8 threads a column in a fixed order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float *partial, float *out, int parts, int pitch,
                                                         int cols) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (col < cols)
    for (int i = w; i < parts; i += 8) x += partial[(size_t)i * pitch + col];
  sum[w][lane] = x;
  __syncthreads();
  if (w == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) x += sum[i][lane];
    out[col] = x;
  }
}

// ---- launches ----------------------------------------------------------------------

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// 16-byte accesses of 8 columns: every row starts on 16 bytes.
bool vector_rows(int cols, std::initializer_list<const void *> ptrs) {
  if (cols % kVec) return false;
  for (const void *p : ptrs)
    if (!aligned(p, 16)) return false;
  return true;
}

unsigned elt_blocks(const Shape8 &s) { return (unsigned)((long long)s.rows * s.nb); }
unsigned elt_grid(unsigned blocks) {
  constexpr unsigned per = kEltThreads / kVecs * kEltUnroll;
  return blocks / per + (blocks % per != 0);
}

// Calls f(integral_constant W, integral_constant NC) for the row width: a warp
// holds up to 1024 columns (four chunks a thread); wider rows take 2 to 16 warps.
template <typename F>
void with_width(int cols, F &&f) {
  const int chunks = (blocks_of(cols) * kVecs + 31) / 32;  // chunks of 8 columns for each lane of one warp
  using std::integral_constant;
#define SLIM_W(W, NC) f(integral_constant<int, W>(), integral_constant<int, NC>())
  if (chunks <= 1) SLIM_W(1, 1);
  else if (chunks == 2) SLIM_W(1, 2);
  else if (chunks == 3) SLIM_W(1, 3);
  else if (chunks == 4) SLIM_W(1, 4);
  else if (chunks <= 6) SLIM_W(2, 3);
  else if (chunks <= 8) SLIM_W(2, 4);
  else if (chunks <= 12) SLIM_W(4, 3);
  else if (chunks <= 16) SLIM_W(4, 4);
  else if (chunks <= 24) SLIM_W(8, 3);
  else if (chunks <= 32) SLIM_W(8, 4);
  else if (chunks <= 48) SLIM_W(16, 3);
  else SLIM_W(16, 4);
#undef SLIM_W
}

}  // namespace

template <typename T>
cudaError_t quantize(const void *x, void *codes, void *scales, void *z_codes, void *z_scales, bool gelu, int rows,
                     int cols, cudaStream_t st) {
  const Shape8 s = shape8(rows, cols);
  const Mat8 a{static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales)};
  const Mat8 z{static_cast<uint8_t *>(z_codes), static_cast<uint8_t *>(z_scales)};
  const T *p = static_cast<const T *>(x);
  const unsigned blocks = elt_blocks(s), grid = elt_grid(blocks);
  const bool vec = vector_rows(cols, {x});
  ProfScope ps(gelu ? "q8_gelu" : "q8_quantize", st);
  if (gelu) {
    if (vec) quantize_kernel<T, true, true><<<grid, kEltThreads, 0, st>>>(p, a, z, s, blocks);
    else quantize_kernel<T, true, false><<<grid, kEltThreads, 0, st>>>(p, a, z, s, blocks);
  } else {
    if (vec) quantize_kernel<T, false, true><<<grid, kEltThreads, 0, st>>>(p, a, z, s, blocks);
    else quantize_kernel<T, false, false><<<grid, kEltThreads, 0, st>>>(p, a, z, s, blocks);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize(const void *codes, const void *scales, void *x, int rows, int cols, int block_rows,
                       cudaStream_t st) {
  const Shape8 s = shape8(rows, cols);
  const uint8_t *c = static_cast<const uint8_t *>(codes), *sc = static_cast<const uint8_t *>(scales);
  T *p = static_cast<T *>(x);
  const unsigned blocks = elt_blocks(s), grid = elt_grid(blocks);
  const int shift = block_rows == 1 ? 0 : 7;
  ProfScope ps("q8_dequantize", st);
  if (vector_rows(cols, {x})) dequantize_kernel<T, true><<<grid, kEltThreads, 0, st>>>(c, sc, p, s, shift, blocks);
  else dequantize_kernel<T, false><<<grid, kEltThreads, 0, st>>>(c, sc, p, s, shift, blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t gelu_bwd(const void *da, const void *z_codes, const void *z_scales, void *dz, void *dz_codes,
                     void *dz_scales, int rows, int cols, cudaStream_t st) {
  const Shape8 s = shape8(rows, cols);
  const uint8_t *c = static_cast<const uint8_t *>(z_codes), *sc = static_cast<const uint8_t *>(z_scales);
  const Mat8 q{static_cast<uint8_t *>(dz_codes), static_cast<uint8_t *>(dz_scales)};
  const T *in = static_cast<const T *>(da);
  T *out = static_cast<T *>(dz);
  const unsigned blocks = elt_blocks(s), grid = elt_grid(blocks);
  ProfScope ps("q8_gelu_bwd", st);
  if (vector_rows(cols, {da, dz})) gelu_bwd_kernel<T, true><<<grid, kEltThreads, 0, st>>>(in, c, sc, out, q, s, blocks);
  else gelu_bwd_kernel<T, false><<<grid, kEltThreads, 0, st>>>(in, c, sc, out, q, s, blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pack_weight(const void *w, void *codes, void *scales, void *codes_t, void *scales_t, int n, int k,
                        cudaStream_t st) {
  const Mat8 q{static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales)};
  const Mat8 qt{static_cast<uint8_t *>(codes_t), static_cast<uint8_t *>(scales_t)};
  const dim3 grid(blocks_of(k), blocks_of(n));
  const T *p = static_cast<const T *>(w);
  ProfScope ps("q8_pack_weight", st);
  if (vector_rows(k, {w})) pack_weight_kernel<T, true><<<grid, 256, 0, st>>>(p, q, qt, n, k);
  else pack_weight_kernel<T, false><<<grid, 256, 0, st>>>(p, q, qt, n, k);
  return cudaGetLastError();
}

template <typename T>
cudaError_t rms_norm(const void *x, const void *res, const float *gamma, float eps, void *h, float *rstd,
                     void *y_codes, void *y_scales, void *h_codes, void *h_scales, int rows, int cols,
                     cudaStream_t st) {
  const Shape8 s = shape8(rows, cols);
  const Mat8 y{static_cast<uint8_t *>(y_codes), static_cast<uint8_t *>(y_scales)};
  const Mat8 hq{static_cast<uint8_t *>(h_codes), static_cast<uint8_t *>(h_scales)};
  const T *xp = static_cast<const T *>(x), *rp = static_cast<const T *>(res);
  T *hp = static_cast<T *>(h);
  const bool vec = vector_rows(cols, {x, res, h, gamma});
  ProfScope ps("q8_rms_norm", st);
  with_width(cols, [&](auto w, auto nc) {
    constexpr int W = decltype(w)::value, NC = decltype(nc)::value;
    const unsigned grid = (unsigned)(((long long)rows + NormCfg<W>::kRows - 1) / NormCfg<W>::kRows);
    if (vec)
      rms_norm_kernel<T, W, NC, true><<<grid, NormCfg<W>::kThreads, 0, st>>>(xp, rp, gamma, eps, hp, rstd, y, hq, s);
    else
      rms_norm_kernel<T, W, NC, false><<<grid, NormCfg<W>::kThreads, 0, st>>>(xp, rp, gamma, eps, hp, rstd, y, hq, s);
  });
  return cudaGetLastError();
}

static int bwd_ctas(int rows, int cols) {
  int per = 1;
  with_width(cols, [&](auto w, auto) { per = NormCfg<decltype(w)::value>::kRows; });
  return (int)std::min<long long>(kBwdCtas, ((long long)rows + per - 1) / per);
}

size_t rms_norm_bwd_workspace(int rows, int cols) {
  return (size_t)bwd_ctas(rows, cols) * blocks_of(cols) * kBlock * sizeof(float);
}

template <typename T>
cudaError_t rms_norm_bwd(const void *dy, const void *h, const void *h_codes, const void *h_scales, const float *rstd,
                         const float *gamma, const void *dres, void *dh, float *dgamma, void *workspace, int rows,
                         int cols, cudaStream_t st) {
  const Shape8 s = shape8(rows, cols);
  const T *yp = static_cast<const T *>(dy), *hp = static_cast<const T *>(h), *rp = static_cast<const T *>(dres);
  const uint8_t *hc = static_cast<const uint8_t *>(h_codes), *hs = static_cast<const uint8_t *>(h_scales);
  T *out = static_cast<T *>(dh);
  float *partial = dgamma ? static_cast<float *>(workspace) : nullptr;
  const bool vec = vector_rows(cols, {dy, h, dres, dh, gamma});
  const int ctas = bwd_ctas(rows, cols);
  if (ctas > 0) {
    ProfScope ps("q8_rms_norm_bwd", st);
    with_width(cols, [&](auto w, auto nc) {
      constexpr int W = decltype(w)::value, NC = decltype(nc)::value;
      const size_t smem = NormCfg<W>::kRows > 1 ? (size_t)s.nb * kBlock * sizeof(float) : 0;
      if (vec)
        rms_norm_bwd_kernel<T, W, NC, true>
            <<<ctas, NormCfg<W>::kThreads, smem, st>>>(yp, hp, hc, hs, rstd, gamma, rp, out, partial, s);
      else
        rms_norm_bwd_kernel<T, W, NC, false>
            <<<ctas, NormCfg<W>::kThreads, smem, st>>>(yp, hp, hc, hs, rstd, gamma, rp, out, partial, s);
    });
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (dgamma) {
    ProfScope ps("q8_dgamma", st);
    column_sum_kernel<<<(cols + 31) / 32, 256, 0, st>>>(partial, dgamma, ctas, s.nb * kBlock, cols);
  }
  return cudaGetLastError();
}

#define SLIM_Q8_INSTANCES(T)                                                                                         \
  template cudaError_t quantize<T>(const void *, void *, void *, void *, void *, bool, int, int, cudaStream_t);      \
  template cudaError_t dequantize<T>(const void *, const void *, void *, int, int, int, cudaStream_t);               \
  template cudaError_t gelu_bwd<T>(const void *, const void *, const void *, void *, void *, void *, int, int,       \
                                   cudaStream_t);                                                                    \
  template cudaError_t pack_weight<T>(const void *, void *, void *, void *, void *, int, int, cudaStream_t);         \
  template cudaError_t rms_norm<T>(const void *, const void *, const float *, float, void *, float *, void *,        \
                                   void *, void *, void *, int, int, cudaStream_t);                                  \
  template cudaError_t rms_norm_bwd<T>(const void *, const void *, const void *, const void *, const float *,        \
                                       const float *, const void *, void *, float *, void *, int, int, cudaStream_t);
SLIM_Q8_INSTANCES(__nv_bfloat16)
SLIM_Q8_INSTANCES(float)
#undef SLIM_Q8_INSTANCES

}  // namespace q8
}  // namespace slim
