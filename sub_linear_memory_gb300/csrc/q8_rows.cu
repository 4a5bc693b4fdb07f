// q8_rows.cu -- elementwise operators with 8-bit rows: quantize, dequantize, the
// packed weight, GeLU and its backward.
//
// Each element is read and written once, in 16-byte accesses, and 16
// neighbouring threads hold one block of 128 columns in registers while they
// agree on its scale (four shuffles for two blocks).  Quantize and dequantize
// are bound by memory (32768 x 4096 bf16: 72 us, 5.6 TB/s, and 63 us, 6.4 TB/s);
// GeLU and its backward by their arithmetic (65536 x 1024 bf16: 76 and 70 us;
// without it 60 and 57; fp32 88 us, and the backward 93, 6.5 TB/s).  A backward
// that also writes the 8 bits of dz takes 86 us (4.7 TB/s), fp32 107 (6.3).  Rows
// off 8 columns or 16 bytes go element by element (65536 x 1001 bf16: quantize
// 49 us, dequantize 174, GeLU 88, backward 146).
#include "kernels.h"
#include "q8.h"
#include "q8_common.cuh"
#include "tc_common.cuh"

namespace slim {
namespace q8 {
namespace {

using tc::ex2_ftz;

// ---- GeLU -------------------------------------------------------------------

__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The normal distribution function and density at two points.  The tail
// beyond |z| is exp(-z^2 / 2) times a polynomial in u = 1 / (1 + 0.35 |z|) (the
// form of Hastings, Approximations for Digital Computers, 1955), of degree 9
// without a constant term, fitted for the smallest relative error over
// 0 <= |z| <= 14 (3e-8), so that the left tail keeps its digits.  With its
// roundings the function is within 6e-7 of its value for |z| <= 2 (most of it
// the reciprocal's unit, 2.3 times over near 0); beyond, the exponent's
// roundings take up to z^2 units 2^-24 (8e-6 at 13).  One exponential and one
// reciprocal serve both functions; the polynomial runs on two values at a time.
// normcdff and expf in its place made GeLU 3.5 times as long as its memory
// traffic.
//
// NEAR: for |z| <= 1 the function is 1/2 + z P(z^2) instead, P of degree 4
// (fitted to 3e-8 of the smaller of the two tails), which is within 1.25 *
// 2^-24.  fp32 rows take it.  bf16 rows do not: their gradient is rounded to
// 2^-8, and 65536 x 1024 would take 88 us and 82 back for 77 and 70.
template <bool NEAR>
__device__ __forceinline__ void normal_parts(float2 z, float2 &cdf, float2 &pdf) {
  const float2 t = make_float2(fabsf(z.x), fabsf(z.y));
  const float2 d = __ffma2_rn(t, make_float2(0.35f, 0.35f), make_float2(1.f, 1.f));
  const float2 u = make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
  float2 p = make_float2(-0.029146051f, -0.029146051f);
  auto step = [](float2 &y, float2 x, float c) { y = __ffma2_rn(y, x, make_float2(c, c)); };
  step(p, u, 0.14397228f);
  step(p, u, -0.25571546f);
  step(p, u, 0.1591755f);
  step(p, u, -0.023110742f);
  step(p, u, 0.10550838f);
  step(p, u, 0.11983278f);
  step(p, u, 0.13986188f);
  step(p, u, 0.13962141f);
  p = __fmul2_rn(p, u);
  const float2 sq = __fmul2_rn(t, t), a = __fmul2_rn(sq, make_float2(-0.72134752f, -0.72134752f));
  const float2 e = make_float2(ex2_ftz(a.x), ex2_ftz(a.y));
  const float2 q = __fmul2_rn(p, e);
  cdf = make_float2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
  if constexpr (NEAR) {
    float2 n = make_float2(9.15123965e-05f, 9.15123965e-05f);
    step(n, sq, -0.00116311491f);
    step(n, sq, 0.0099623967f);
    step(n, sq, -0.0664881989f);
    step(n, sq, 0.398942143f);
    n = __ffma2_rn(n, z, make_float2(0.5f, 0.5f));
    cdf = make_float2(t.x <= 1.f ? n.x : cdf.x, t.y <= 1.f ? n.y : cdf.y);
  }
  pdf = __fmul2_rn(e, make_float2(0.39894228f, 0.39894228f));
}

// ---- elementwise over blocks of 128 columns -----------------------------------

constexpr int kEltThreads = 256, kEltUnroll = 4, kEltCtas = 4;

// GELU: a = 8 bits of GeLU(x), z (where wanted) = 8 bits of x; otherwise
// a = 8 bits of x.
template <typename T, bool GELU, bool VEC>
__global__ void __launch_bounds__(kEltThreads, kEltCtas) quantize_kernel(const T *x, Mat8 a, Mat8 z, Shape8 s,
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
  auto live = [&](int u) { return first + u * (kEltThreads / kVecs) < blocks; };
  if constexpr (GELU) {
#pragma unroll
    for (int u = 0; u < kEltUnroll; ++u) {
      float act[kVec];
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        float2 cdf, pdf;
        normal_parts<sizeof(T) == 4>(make_float2(v[u][i], v[u][i + 1]), cdf, pdf);
        act[i] = v[u][i] * cdf.x;
        act[i + 1] = v[u][i + 1] * cdf.y;
      }
      int byte_a, byte_z;
      block_bytes(amax8(act), amax8(v[u]), byte_a, byte_z);
      put8(act, byte_a, a, s, row[u], blk[u], lane16, live(u));
      if (z.codes) put8(v[u], byte_z, z, s, row[u], blk[u], lane16, live(u));
    }
  } else {
#pragma unroll
    for (int u = 0; u < kEltUnroll; u += 2) {
      int byte[2];
      block_bytes(amax8(v[u]), amax8(v[u + 1]), byte[0], byte[1]);
      put8(v[u], byte[0], a, s, row[u], blk[u], lane16, live(u));
      put8(v[u + 1], byte[1], a, s, row[u + 1], blk[u + 1], lane16, live(u + 1));
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kEltThreads, kEltCtas) dequantize_kernel(const uint8_t *codes, const uint8_t *scales, T *x,
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
__global__ void __launch_bounds__(kEltThreads, kEltCtas) gelu_bwd_kernel(const T *da, const uint8_t *codes,
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
    for (int i = 0; i < kVec; i += 2) {
      float2 cdf, pdf;
      normal_parts<sizeof(T) == 4>(make_float2(z[i], z[i + 1]), cdf, pdf);
      // the 8 bits are those of dz as it is stored
      v[u][i] = rounded<T>(v[u][i] * fmaf(z[i], pdf.x, cdf.x));
      v[u][i + 1] = rounded<T>(v[u][i + 1] * fmaf(z[i + 1], pdf.y, cdf.y));
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
    if (q.codes) {
      int bits, unused;
      block_bytes(amax8(v[u]), 0, bits, unused);
      put8(v[u], bits, q, s, row, blk, lane16, b < blocks);
    }
  }
}

// ---- packed weight --------------------------------------------------------------

// One CTA for each 128 x 128 block: its 2048 chunks of 8 columns are in the
// registers of 256 threads, so the weight is read once; the transposed codes
// go through shared memory.  4096 x 1024 bf16 10 us, 4096 x 4096 19 (3.5 TB/s),
// 16384 x 8192 118 (4.6 TB/s); fp32 10, 24 and 148 (5.5 TB/s).
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

// ---- launches ----------------------------------------------------------------------

unsigned elt_blocks(const Shape8 &s) { return (unsigned)((long long)s.rows * s.nb); }
unsigned elt_grid(unsigned blocks) {
  constexpr unsigned per = kEltThreads / kVecs * kEltUnroll;
  return blocks / per + (blocks % per != 0);
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

#define SLIM_Q8_INSTANCES(T)                                                                                         \
  template cudaError_t quantize<T>(const void *, void *, void *, void *, void *, bool, int, int, cudaStream_t);      \
  template cudaError_t dequantize<T>(const void *, const void *, void *, int, int, int, cudaStream_t);               \
  template cudaError_t gelu_bwd<T>(const void *, const void *, const void *, void *, void *, void *, int, int,       \
                                   cudaStream_t);                                                                    \
  template cudaError_t pack_weight<T>(const void *, void *, void *, void *, void *, int, int, cudaStream_t);
SLIM_Q8_INSTANCES(__nv_bfloat16)
SLIM_Q8_INSTANCES(float)
#undef SLIM_Q8_INSTANCES

}  // namespace q8
}  // namespace slim
