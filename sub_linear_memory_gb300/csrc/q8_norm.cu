// q8_norm.cu -- root-mean-square norm with the residual's addition and an 8-bit
// output, and its backward from the full rows or their 8-bit checkpoint.
//
// Both are bound by memory.  A row is held by 1 to 16 warps, each thread with
// one to four chunks of 8 columns, so that everything is formed from one read
// of the inputs; what limits them is how many loads are in flight.  65536 x 1024
// bf16 with a checkpoint: forward 102 us (5.3 TB/s of 6.7; 86 us without the care
// for codes on a border, of which 1 to 9 in 67 million are off, against 25 to 50
// where y is formed in plain fp32; issue slots 76% used), backward 104 us (4.5
// TB/s, at 128 registers with spills in the row loop; 101 us, 5.3 TB/s, from the
// full rows).  fp32: forward 142 us (6.6 TB/s), backward 165 (5.3) and 190 (5.6).
// Rows whose width is no multiple of 8 columns, or that do not start on 16
// bytes, go element by element: 65536 x 1001 bf16 236 us, backward 271 and 309.
#include <cfloat>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "q8.h"
#include "q8_common.cuh"

namespace slim {
namespace q8 {
namespace {

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

// A sum kept as hi + lo: each addition's rounding goes into lo.  Where the sum
// is past fp32's range its rounding is inf - inf; fmaxf takes the number
// instead of that NaN, so hi is the infinity of a plain sum (and a NaN only
// where an operand's hi is one).
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 operator+(const Sum2 &a, const Sum2 &b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float lo = fmaxf((a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo), -FLT_MAX), hi = s + lo;
  return Sum2{hi, lo - (hi - s)};
}

// group_sum of such sums; `part` is used once.
template <int W>
__device__ __forceinline__ Sum2 group_sum2(Sum2 x, Sum2 *part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = x + Sum2{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
  if (W == 1) return x;
  const int warp = threadIdx.x >> 5, first = warp / W * W;
  if ((threadIdx.x & 31) == 0) part[warp] = x;
  __syncthreads();
  x = part[first];
#pragma unroll
  for (int i = 1; i < W; ++i) x = x + part[first + i];
  return x;
}

template <int W> struct NormCfg {
  static constexpr int kThreads = W > 8 ? 32 * W : 256;
  static constexpr int kRows = kThreads / (32 * W);  // rows in flight in a CTA
};

// How many CTAs share an SM: their rows' loads are what hides the memory's
// latency.  Forward, 65536 x 1024 bf16: 132 us with two, 110 with three, 102 with
// four; fp32 154, 142, 154.  Backward from the checkpoint: bf16 145 us with one,
// 104 with two; fp32 165 with one, 214 with two.
template <typename T, int W> constexpr int fwd_ctas() { return W > 8 ? 2 : sizeof(T) == 2 ? 4 : 3; }
template <typename T, int W> constexpr int bwd_ctas() { return W > 8 || sizeof(T) == 4 ? 1 : 2; }

// Moves those of 8 results y = v (root + rest) g by one unit of fp32 towards the
// exact product that lie just halfway between two e4m3 codes of their scale
// (three fraction bits and a one after them: the last 20 bits are 0x80000).
// Two kinds of border are left as y in fp32 has them: those between codes under
// 2^-6 of the scale, whose steps do not shrink with them, and the scale's own,
// 448 * 2^e, which is settled before this.
__device__ __forceinline__ void settle8(float *y, int byte, const float *v, const float *g, float root, float rest) {
  if (byte == kScaleNan) return;
  const float inv = scale_inverse(byte);
  uint32_t off[kVec], nearest = ~0u;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    off[i] = (__float_as_uint(y[i] * inv) & 0xFFFFFu) ^ 0x80000u;
    nearest = min(nearest, off[i]);
  }
  if (nearest != 0) return;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const float n = v[i] * root;
    const float left = fmaf(n, g[i], -y[i]) + fmaf(v[i], rest, fmaf(v[i], root, -n)) * g[i];
    if (off[i] == 0 && left != 0.f)
      y[i] = __uint_as_float(__float_as_uint(y[i]) + ((left > 0.f) == (y[i] > 0.f) ? 1u : ~0u));
  }
}

// W warps hold a row, each thread NC chunks of 8 of its columns, in registers
// between the sum of squares and the quantization: h and y are formed from one
// read of x and res.
template <typename T, int W, int NC, bool VEC>
__global__ void __launch_bounds__(NormCfg<W>::kThreads, fwd_ctas<T, W>())
    rms_norm_kernel(const T *x, const T *res, const float *gamma, float eps, T *h, float *rstd, Mat8 y, Mat8 hq,
                    Shape8 s) {
  __shared__ Sum2 part[NormCfg<W>::kThreads / 32];
  const int l = threadIdx.x % (32 * W), lane16 = l & (kVecs - 1);
  const long long row = (long long)blockIdx.x * NormCfg<W>::kRows + threadIdx.x / (32 * W);
  const bool live = row < s.rows;
  const size_t at = (size_t)row * s.cols;
  float v[NC][kVec];
  {
    Raw8<T> xr[NC], rr[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * 32 * W + l) * kVec, left = live ? s.cols - col : 0;
      xr[c] = load_raw8<T, VEC>(x + at + col, left);
      if (res) rr[c] = load_raw8<T, VEC>(res + at + col, left);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      unpack8(xr[c], v[c]);
      if (res) {
        float r[kVec];
        unpack8(rr[c], r);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[c][i] = rounded<T>(v[c][i] + r[i]);
      }
    }
  }
  // The sum of squares: 8 columns at a time in plain fp32, whose roundings are
  // many and small, and those sums without loss: the last few additions'
  // roundings would be the whole row's.
  Sum2 ss{0.f, 0.f};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = (c * 32 * W + l) * kVec;
    if (h && live) store8<T, VEC>(h + at + col, s.cols - col, v[c]);
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fmaf(v[c][2 * i], v[c][2 * i], v[c][2 * i + 1] * v[c][2 * i + 1]);
    ss = ss + Sum2{(q[0] + q[1]) + (q[2] + q[3]), 0.f};
  }
  ss = group_sum2<W>(ss, part);
  const float cols = (float)s.cols, mean = ss.hi / cols;
  const Sum2 m = Sum2{mean, (fmaf(-mean, cols, ss.hi) + ss.lo) / cols} + Sum2{eps, 0.f};
  const float root = 1.f / sqrtf(m.hi);  // 0 where the sum is past fp32's range
  if (rstd && live && l == 0) rstd[row] = root;
  // What the rounding of root left out, by one Newton step.  y is formed with
  // it and with the rounding of its first product; where y then lies on a
  // border between two codes, what is left of it decides (settle8).  So a normal
  // e4m3 code is that of the exact y, under the scale of the block's largest y in
  // fp32, unless it is within about 2^-27 of a border.
  // (Where a product overflows the remainder is NaN, and so is the block.)
  // No step where root is 0, or so large that its square is past fp32's range.
  float rest = 0.f;
  const float sq = root * root;
  if (m.hi < INFINITY && sq < INFINITY) {
    const float sq_lo = fmaf(root, root, -sq);
    rest = 0.5f * root * (fmaf(-m.hi, sq, 1.f) - fmaf(m.hi, sq_lo, m.lo * sq));
  }
  const float2 root2 = make_float2(root, root), rest2 = make_float2(rest, rest);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int chunk = c * 32 * W + l, blk = chunk / kVecs, col = chunk * kVec;
    const bool on = live && blk < s.nb;
    float g[kVec], out[kVec];
    load8<float, VEC>(gamma + col, s.cols - col, g);
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      const float2 x = make_float2(v[c][i], v[c][i + 1]), gg = make_float2(g[i], g[i + 1]);
      const float2 n = __fmul2_rn(x, root2);
      const float2 lost = __ffma2_rn(x, rest2, __ffma2_rn(x, root2, make_float2(-n.x, -n.y)));
      const float2 full = __ffma2_rn(n, gg, __fmul2_rn(lost, gg));
      // columns past the row are 0 whatever root is
      out[i] = (VEC ? col : col + i) < s.cols ? full.x : 0.f;
      out[i + 1] = (VEC ? col : col + i + 1) < s.cols ? full.y : 0.f;
    }
    int byte_y, byte_h;
    block_bytes(amax8(out), amax8(v[c]), byte_y, byte_h);
    settle8(out, byte_y, v[c], g, root, rest);
    put8(out, byte_y, y, s, row, blk, lane16, on);
    if (hq.codes) put8(v[c], byte_h, hq, s, row, blk, lane16, on);
  }
}

// The gradients.  CTAs walk the rows; a thread's columns stay the same, so its
// share of dgamma is summed in registers, then over the CTA's groups through
// shared memory, and a CTA writes one partial row.  The rows are kept as they
// were read between the sum over a row and dh, and unpacked twice.
constexpr int kBwdCtas = 304;  // two for each of 152 SMs: fixed, so that the order of the sums is

template <typename T, int W, int NC, bool VEC, bool KEPT8>
__global__ void __launch_bounds__(NormCfg<W>::kThreads, bwd_ctas<T, W>())
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
    Raw8<T> yr[NC], rr[NC], kr[KEPT8 ? 1 : NC];
    uint2 code[KEPT8 ? NC : 1];
    int byte[KEPT8 ? NC : 1];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int chunk = c * 32 * W + l, col = chunk * kVec, left = live ? s.cols - col : 0;
      yr[c] = load_raw8<T, VEC>(dy + at + col, left);
      if constexpr (KEPT8) {
        code[c] = make_uint2(0, 0);
        byte[c] = 127;
        if (left > 0) {
          const int blk = chunk / kVecs;
          code[c] = __ldg(reinterpret_cast<const uint2 *>(hc + ((size_t)row * s.nb + blk) * kBlock + (l & 15) * kVec));
          byte[c] = __ldg(hs + (size_t)row * s.pitch + blk);
        }
      } else {
        kr[c] = load_raw8<T, VEC>(h + at + col, left);
      }
      if (dres) rr[c] = load_raw8<T, VEC>(dres + at + col, left);
    }
    // dy and n = h * rstd of a chunk
    auto chunk_of = [&](int c, float *y, float *n) {
      unpack8(yr[c], y);
      if constexpr (KEPT8) {
        decode8(code[c], scale_value(byte[c]), n);
        if (!VEC) {  // columns past the row: a NaN block's scale reaches them
          const int left = live ? s.cols - (c * 32 * W + l) * kVec : 0;
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (i >= left) n[i] = 0.f;
        }
      } else {
        unpack8(kr[c], n);
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) n[i] *= root;
    };
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * 32 * W + l) * kVec;
      float y[kVec], n[kVec], gm[kVec];
      chunk_of(c, y, n);
      load8<float, VEC>(gamma + col, s.cols - col, gm);
      float d[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        acc[c][i] = fmaf(y[i], n[i], acc[c][i]);
        d[i & 1] = fmaf(y[i] * gm[i], n[i], d[i & 1]);
      }
      dot += d[0] + d[1];
    }
    const float mean = group_sum<W>(dot, part[turn]) / (float)s.cols;
    turn ^= 1;
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int col = (c * 32 * W + l) * kVec;
        float y[kVec], n[kVec], gm[kVec], r[kVec];
        chunk_of(c, y, n);
        load8<float, VEC>(gamma + col, s.cols - col, gm);
        if (dres) unpack8(rr[c], r);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float d = root * (y[i] * gm[i] - n[i] * mean);
          y[i] = dres ? d + r[i] : d;
        }
        store8<T, VEC>(dh + at + col, s.cols - col, y);
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

static int bwd_grid(int rows, int cols) {
  int per = 1;
  with_width(cols, [&](auto w, auto) { per = NormCfg<decltype(w)::value>::kRows; });
  return (int)std::min<long long>(kBwdCtas, ((long long)rows + per - 1) / per);
}

size_t rms_norm_bwd_workspace(int rows, int cols) {
  return (size_t)bwd_grid(rows, cols) * blocks_of(cols) * kBlock * sizeof(float);
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
  const int ctas = bwd_grid(rows, cols);
  if (ctas > 0) {
    ProfScope ps("q8_rms_norm_bwd", st);
    with_width(cols, [&](auto w, auto nc) {
      constexpr int W = decltype(w)::value, NC = decltype(nc)::value;
      const size_t smem = NormCfg<W>::kRows > 1 ? (size_t)s.nb * kBlock * sizeof(float) : 0;
      auto kern = vec ? (hc ? rms_norm_bwd_kernel<T, W, NC, true, true> : rms_norm_bwd_kernel<T, W, NC, true, false>)
                      : (hc ? rms_norm_bwd_kernel<T, W, NC, false, true> : rms_norm_bwd_kernel<T, W, NC, false, false>);
      kern<<<ctas, NormCfg<W>::kThreads, smem, st>>>(yp, hp, hc, hs, rstd, gamma, rp, out, partial, s);
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
  template cudaError_t rms_norm<T>(const void *, const void *, const float *, float, void *, float *, void *,        \
                                   void *, void *, void *, int, int, cudaStream_t);                                  \
  template cudaError_t rms_norm_bwd<T>(const void *, const void *, const void *, const void *, const float *,        \
                                       const float *, const void *, void *, float *, void *, int, int, cudaStream_t);
SLIM_Q8_INSTANCES(__nv_bfloat16)
SLIM_Q8_INSTANCES(float)
#undef SLIM_Q8_INSTANCES

}  // namespace q8
}  // namespace slim
