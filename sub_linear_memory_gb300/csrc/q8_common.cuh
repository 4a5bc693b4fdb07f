// q8_common.cuh -- the 8-bit form of rows and weights (e4m3 codes, one
// power-of-two scale for each block of 128 columns) and row access.
#pragma once

#include <cuda_fp8.h>

#include <initializer_list>

#include "common.cuh"

namespace slim {
namespace q8 {

constexpr int kBlock = 128;   // columns (and weight rows) under one scale
constexpr int kVec = 8;       // columns one thread handles at a time
constexpr int kVecs = kBlock / kVec;  // 16 threads share a block

__host__ __device__ inline int blocks_of(int cols) { return cols / kBlock + (cols % kBlock != 0); }
__host__ __device__ inline int scale_pitch(int cols) { return (blocks_of(cols) + 3) / 4 * 4; }

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr int kScaleNan = 255, kScaleMax = 247;

// Scale byte of a block from the bits of its largest magnitude (as unsigned
// integers the magnitudes of floats are ordered, and infinities and NaNs lie
// above every number).  448 = 1.75 * 2^8, so with amax = f * 2^E the smallest
// e with amax <= 448 * 2^e is E - 8, plus one where the fraction f is over
// 1.75: a carry out of the fraction when 2^23 - 1 - 0x600000 is added.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  if (amax_bits >= kInfBits) return kScaleNan;
  const int e = (int)((amax_bits + 0x1FFFFFu) >> 23) - 135;
  return min(max(e, -117), 120) + 127;
}

// 2^-e of a number's scale byte: exact.
__device__ __forceinline__ float scale_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// 2^e of a scale byte.
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte == kScaleNan ? 0x7fffffffu : byte == 0 ? 0x00400000u : (uint32_t)byte << 23);
}

// Largest magnitude (its bits) of 8 values, two to an instruction.  max.NaN
// returns a NaN where there is one.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ uint32_t amax8(const float *v) {
  float m = max3_nan(fabsf(v[0]), fabsf(v[1]), fabsf(v[2]));
  m = max3_nan(m, fabsf(v[3]), fabsf(v[4]));
  m = max3_nan(m, fabsf(v[5]), fabsf(v[6]));
  return __float_as_uint(max3_nan(m, fabsf(v[7]), 0.f));
}

// The scale bytes of two blocks from this thread's share of each; the blocks'
// 16 threads agree.  A scale byte never falls as the magnitude grows (a NaN
// block's is the largest), so the bytes can be compared in place of the
// magnitudes, and two of them travel in one shuffle.
__device__ __forceinline__ void block_bytes(uint32_t amax0, uint32_t amax1, int &byte0, int &byte1) {
  uint32_t m = (uint32_t)scale_byte(amax0) | (uint32_t)scale_byte(amax1) << 16;
#pragma unroll
  for (int o = 1; o < kVecs; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  byte0 = (int)(m & 0xffffu);
  byte1 = (int)(m >> 16);
}

// The codes of a NaN block: NaN in the `left` columns inside the row.
__device__ __forceinline__ uint2 nan_codes8(int left) {
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = min(max(left - 4 * i, 0), 4);
    c[i] = m == 4 ? 0x7f7f7f7fu : 0x7f7f7f7fu & ((1u << (8 * m)) - 1);
  }
  return make_uint2(c[0], c[1]);
}

// The codes of 8 values (`left` of them inside the row) of a block with this
// scale byte: value times 2^-e, rounded to e4m3.  The product with a power of
// two is exact (or far below the smallest code), so this is the only rounding.
// Under the largest scale, 2^120, the codes stop at 240, since 256 * 2^120 is
// past fp32: a finite value stays finite.
__device__ __forceinline__ uint2 encode8(const float *v, int byte, int left) {
  if (byte == kScaleNan) return nan_codes8(left);
  const float inv = scale_inverse(byte);
  float2 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(inv, inv));
  if (byte == kScaleMax) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = make_float2(fminf(fmaxf(x[i].x, -240.f), 240.f), fminf(fmaxf(x[i].y, -240.f), 240.f));
  }
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __nv_cvt_float2_to_fp8x2(x[i], __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// 8 codes times 2^e (every e4m3 number is an fp16 number).
__device__ __forceinline__ void decode8(uint2 c, float s, float *v) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

// 8 consecutive columns of a row as they lie in memory, `left` of them inside it
// (the rest are 0).  VEC: the row is aligned and left is 8 or <= 0.  Plain
// loads, not the read-only path: outputs may be the inputs' own buffers.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 w; };
template <> struct Raw8<float> { float4 a, b; };

template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load_raw8(const T *p, int left) {
  if constexpr (!VEC) {
    T v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = i < left ? p[i] : from_f32<T>(0.f);
    Raw8<T> r;
    memcpy(&r, v, sizeof(r));
    return r;
  } else if constexpr (sizeof(T) == 2) {
    return Raw8<T>{left > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0)};
  } else {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    return left > 0 ? Raw8<T>{reinterpret_cast<const float4 *>(p)[0], reinterpret_cast<const float4 *>(p)[1]}
                    : Raw8<T>{z, z};
  }
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float *v) {
  const uint32_t u[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float *v) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *p, int left, float *v) {
  unpack8(load_raw8<T, VEC>(p, left), v);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, int left, const float *v);

template <>
__device__ __forceinline__ void store8<__nv_bfloat16, true>(__nv_bfloat16 *p, int left, const float *v) {
  if (left <= 0) return;
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
template <>
__device__ __forceinline__ void store8<float, true>(float *p, int left, const float *v) {
  if (left <= 0) return;
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16, false>(__nv_bfloat16 *p, int left, const float *v) {
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < left) p[i] = __float2bfloat16_rn(v[i]);
}
template <>
__device__ __forceinline__ void store8<float, false>(float *p, int left, const float *v) {
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < left) p[i] = v[i];
}

// 16-byte accesses of 8 columns: every row starts on 16 bytes.
inline bool vector_rows(int cols, std::initializer_list<const void *> ptrs) {
  if (cols % kVec) return false;
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

// What a value becomes when it is stored as T.
template <typename T> __device__ __forceinline__ float rounded(float x) { return to_f32(from_f32<T>(x)); }

// An 8-bit matrix and its pitches.
struct Mat8 {
  uint8_t *codes, *scales;
};
struct Shape8 {
  int rows, cols, nb, pitch;  // nb blocks of 128 columns, `pitch` scale bytes a row
};
__host__ __device__ inline Shape8 shape8(int rows, int cols) { return Shape8{rows, cols, blocks_of(cols), scale_pitch(cols)}; }

// Store the codes of this thread's 8 values of block `blk` of a row under its
// scale byte and, once, that byte; the last block's thread also writes the
// bytes that pad the row's scales.  live: the block exists.
__device__ __forceinline__ void put8(const float *v, int byte, const Mat8 &m, const Shape8 &s, long long row, int blk,
                                     int lane16, bool live) {
  const int col = blk * kBlock + lane16 * kVec;
  const uint2 c = encode8(v, byte, s.cols - col);
  if (!live) return;
  *reinterpret_cast<uint2 *>(m.codes + row * s.nb * kBlock + col) = c;
  if (lane16 == 0) {
    uint8_t *sc = m.scales + row * s.pitch;
    sc[blk] = (uint8_t)byte;
    if (blk == s.nb - 1)
      for (int i = s.nb; i < s.pitch; ++i) sc[i] = 127;
  }
}

}  // namespace q8
}  // namespace slim
