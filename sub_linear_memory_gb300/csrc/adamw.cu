// adamw.cu -- one AdamW step (decoupled weight decay) over many tensors:
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = (1 - lr wd) p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps),
// t = the count of steps, this one included.
//
// Memory-bound: with fp32 states 28 bytes a parameter (fp32 gradients), with
// 8-bit states 16 and two scale bytes in and out for 128.  One launch goes
// over every tensor: their pointers travel as the kernel's argument and a
// block finds its tensor by its number among them.  A thread has four
// consecutive elements of each of four blocks of 128, all loads ahead of the
// arithmetic.
//
// 8-bit states are a one-row 8-bit matrix each (e4m3 codes, a power-of-two
// scale for 128 elements), m, and in place of v its root r: the codes' range
// of 2^17.8 within a block is then one of 2^35.6 in v.  Each value is rounded
// up or down at random with the probability of its place between two codes,
// because what a step changes, (1 - b2) / 2 of r or less, is far below half a
// code's step of 1/16: to nearest it would never be seen.  r > 0 is not
// rounded to 0, so that m / sqrt(v) stays bounded.  The random numbers are
// Philox4x32-10's of (seed, t, tensor, element / 4): a step gives the same
// result however it is launched.  p takes the step from the moments before
// they are rounded.
#include <cmath>

#include "kernels.h"
#include "philox.cuh"
#include "q8_common.cuh"
#include "train.h"

namespace slim {
namespace {

constexpr int kThreads = 256, kEach = 4, kPasses = 4, kChunk = kThreads * kEach * kPasses;

struct Entry {
  float *p;
  const void *g;
  void *m, *v;                // fp32, or codes
  uint8_t *m_scales, *v_scales;
  long long n;
  int index, first;           // the tensor's number, and the launch's first block of it
};
template <int MOST> struct Entries {
  int n;
  Entry at[MOST];
};
struct Numbers {
  const float *lr_now;
  float lr, b1, b2, a1, a2, eps, wd, log_b1, log_b2;  // a = 1 - b
  uint32_t seed0, seed1;
  int *count;  // steps done, blocks done
  int last;    // the step's last launch: it moves the count on
};

// 4 consecutive elements, `left` of them inside the tensor; vec: aligned
template <typename T> __device__ __forceinline__ void load4(const T *p, int left, bool vec, float *v) {
  if (vec && left >= 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = *reinterpret_cast<const float4 *>(p);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
      v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? to_f32(p[i]) : 0.f;
  }
}
__device__ __forceinline__ void store4(float *p, int left, bool vec, const float *v) {
  if (vec && left >= 4) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = v[i];
  }
}

__device__ __forceinline__ void decode4(uint32_t c, float s, float *v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

// |x| 2^-e <= 448 to one of the two codes around it: 20 random bits are added
// below the three that stay.  Codes below 2^-6 lie as far apart as those from
// there to 2^-5, so 2^-6 more puts them there.
__device__ __forceinline__ float round_at_random(float w, uint32_t bits20) {
  const float up = w < 0.015625f ? 0.015625f : 0.f;
  return __uint_as_float((__float_as_uint(w + up) + bits20) & 0xFFF00000u) - up;
}

// The codes of 4 values of a block of 128 (one warp's), and its scale byte.
// `shift`: where the values' random bits lie in the words.
__device__ __forceinline__ uint32_t encode4(const float *x, const uint32_t *words, int shift, bool never_zero, int &byte) {
  float top = q8::max3_nan(fabsf(x[0]), fabsf(x[1]), fabsf(x[2]));
  top = q8::max3_nan(top, fabsf(x[3]), 0.f);
  byte = (int)__reduce_max_sync(0xffffffffu, (unsigned)q8::scale_byte(__float_as_uint(top)));
  if (byte == q8::kScaleNan) return 0x7f7f7f7fu;
  const float inv = q8::scale_inverse(byte), most = byte == q8::kScaleMax ? 240.f : 448.f;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fabsf(x[i]);
    float w = fminf(round_at_random(a * inv, shift ? words[i] >> 12 & 0xFFFF0u : words[i] << 4 & 0xFFFF0u), most);
    if (never_zero && a > 0.f) w = fmaxf(w, 0.001953125f);
    y[i] = copysignf(w, x[i]);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// The hardware's root and inverse, within two units: the step's own rounding into p is far larger (a root that is held
// in 8 bits is rounded to nearest).  Roots of numbers below fp32's normal range are 0.
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Elements [chunk, chunk + count) of a tensor.  WHOLE: kChunk of them, aligned.  `now` is written by thread 0 and
// read behind the barrier.
template <typename G, bool EIGHT, bool WHOLE>
__device__ __forceinline__ void chunk_step(const Entry &e, long long chunk, int count, const Numbers &o, const float *now) {
  const int t = threadIdx.x;
  float *pp = e.p + chunk;
  const G *gp = static_cast<const G *>(e.g) + chunk;
  uint8_t *mq = nullptr, *vq = nullptr, *msq = nullptr, *vsq = nullptr;
  float *mp = nullptr, *vp = nullptr;
  if constexpr (EIGHT) {
    mq = static_cast<uint8_t *>(e.m) + chunk, vq = static_cast<uint8_t *>(e.v) + chunk;
    msq = e.m_scales + chunk / q8::kBlock, vsq = e.v_scales + chunk / q8::kBlock;
  } else {
    mp = static_cast<float *>(e.m) + chunk, vp = static_cast<float *>(e.v) + chunk;
  }
  const bool vec_p = WHOLE || (reinterpret_cast<uintptr_t>(e.p) & 15) == 0,
             vec_g = WHOLE || (reinterpret_cast<uintptr_t>(e.g) & (4 * sizeof(G) - 1)) == 0;
  bool vec_s = true;
  if constexpr (!EIGHT && !WHOLE)
    vec_s = ((reinterpret_cast<uintptr_t>(e.m) | reinterpret_cast<uintptr_t>(e.v)) & 15) == 0;
  float p[kPasses][4], g[kPasses][4], m[kPasses][4], v[kPasses][4];
  uint32_t mc[kPasses], vc[kPasses];
  int ms[kPasses], vs[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int at = (i * kThreads + t) * kEach, left = WHOLE ? 4 : count - at;
    load4(pp + at, left, vec_p, p[i]);
    load4(gp + at, left, vec_g, g[i]);
    if constexpr (EIGHT) {
      // codes lie in whole blocks of 128
      const bool live = WHOLE || at / q8::kBlock * q8::kBlock < count;
      mc[i] = live ? *reinterpret_cast<const uint32_t *>(mq + at) : 0u;
      vc[i] = live ? *reinterpret_cast<const uint32_t *>(vq + at) : 0u;
      ms[i] = live ? msq[at / q8::kBlock] : 127;
      vs[i] = live ? vsq[at / q8::kBlock] : 127;
    } else {
      load4(mp + at, left, vec_s, m[i]);
      load4(vp + at, left, vec_s, v[i]);
    }
  }
  __syncthreads();
  const float rate = -now[0], root_c2 = now[1], keep = now[2];
  const uint32_t steps = __float_as_uint(now[3]);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int at = (i * kThreads + t) * kEach, left = WHOLE ? 4 : count - at;
    if constexpr (EIGHT) {
      decode4(mc[i], q8::scale_value(ms[i]), m[i]);
      decode4(vc[i], q8::scale_value(vs[i]), v[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] *= v[i][j];
    }
    float r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float gv = g[i][j];
      // each product and sum rounded by itself, and the root to nearest: whoever forms the moments by elementary
      // operations gets the same codes
      m[i][j] = __fadd_rn(__fmul_rn(m[i][j], o.b1), __fmul_rn(gv, o.a1));
      v[i][j] = __fadd_rn(__fmul_rn(v[i][j], o.b2), __fmul_rn(__fmul_rn(gv, gv), o.a2));
      r[j] = EIGHT ? __fsqrt_rn(v[i][j]) : root(v[i][j]);
      p[i][j] = fmaf(p[i][j], keep, rate * m[i][j] * inverse(fmaf(r[j], root_c2, o.eps)));
    }
    store4(pp + at, left, vec_p, p[i]);
    if constexpr (EIGHT) {
      const unsigned long long element = (unsigned long long)(chunk + at);
      uint32_t w[4] = {(uint32_t)(element >> 2), (uint32_t)e.index, (uint32_t)(element >> 34), steps};
      philox4x32_10(w, o.seed0, o.seed1);
      if (left < 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m[i][j] = j < left ? m[i][j] : 0.f;
          r[j] = j < left ? r[j] : 0.f;
        }
      }
      int mb, vb;
      const uint32_t m4 = encode4(m[i], w, 0, false, mb), v4 = encode4(r, w, 16, true, vb);
      if (WHOLE || at / q8::kBlock * q8::kBlock < count) {
        // past the tensor's end codes stay 0, in a NaN block too
        const uint32_t inside = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        *reinterpret_cast<uint32_t *>(mq + at) = m4 & inside;
        *reinterpret_cast<uint32_t *>(vq + at) = v4 & inside;
        if ((t & 31) == 0) {
          msq[at / q8::kBlock] = (uint8_t)mb;
          vsq[at / q8::kBlock] = (uint8_t)vb;
        }
      }
    } else {
      store4(mp + at, left, vec_s, m[i]);
      store4(vp + at, left, vec_s, v[i]);
    }
  }
}

template <typename G, bool EIGHT, int MOST>
// Four blocks an SM (two, at the 104 registers it would take: 220 us).
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Entries<MOST> entries, Numbers o) {
  __shared__ float now[4];
  const int t = threadIdx.x;
  if (t == 0) {
    const float steps = (float)(o.count[0] + 1), lr = o.lr_now ? *o.lr_now : o.lr;
    // 1 - b^t without the difference's loss
    now[0] = lr / -expm1f(steps * o.log_b1);
    now[1] = rsqrtf(-expm1f(steps * o.log_b2));
    now[2] = 1.f - lr * o.wd;
    now[3] = __int_as_float(o.count[0] + 1);
  }
  int lo = 0, hi = entries.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (entries.at[mid].first <= (int)blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const Entry e = entries.at[lo];
  const long long chunk = (long long)((int)blockIdx.x - e.first) * kChunk;
  bool vec = (reinterpret_cast<uintptr_t>(e.p) & 15) == 0 && (reinterpret_cast<uintptr_t>(e.g) & (4 * sizeof(G) - 1)) == 0;
  if constexpr (!EIGHT) vec = vec && ((reinterpret_cast<uintptr_t>(e.m) | reinterpret_cast<uintptr_t>(e.v)) & 15) == 0;
  // Whole chunks of aligned tensors take no look at the end (8-bit states of 54 M weights: 198 -> 170 us;
  // 190 with roots to nearest).
  if (vec && e.n - chunk >= kChunk)
    chunk_step<G, EIGHT, true>(e, chunk, kChunk, o, now);
  else
    chunk_step<G, EIGHT, false>(e, chunk, (int)(e.n - chunk < kChunk ? e.n - chunk : kChunk), o, now);
  if (o.last && t == 0) {
    // every block has read the count when the last one comes here
    __threadfence();
    if (atomicAdd(o.count + 1, 1) == (int)gridDim.x - 1) {
      o.count[1] = 0;
      o.count[0] += 1;
    }
  }
}

template <typename G, bool EIGHT, int MOST>
cudaError_t launch(const Entry *entries, int n, int blocks, const Numbers &o, cudaStream_t st) {
  static_assert(sizeof(Entries<MOST>) + sizeof(Numbers) <= 32764, "kernel arguments");
  Entries<MOST> e;
  e.n = n;
  for (int i = 0; i < n; ++i) e.at[i] = entries[i];
  adamw_kernel<G, EIGHT, MOST><<<blocks, kThreads, 0, st>>>(e, o);
  return cudaGetLastError();
}

constexpr int kFew = 48, kMany = 496;  // tensors of one launch: 3.5 or 32 KB of arguments

}  // namespace

cudaError_t adamw(const slim_adamw_tensor *tensors, int n, const slim_adamw_options &o, bool g_f32, int *count,
                  cudaStream_t st) {
  ProfScope ps("adamw", st);
  Numbers numbers{o.lr_device, o.lr, (float)o.beta1, (float)o.beta2, (float)(1.0 - o.beta1), (float)(1.0 - o.beta2), o.eps,
                  o.weight_decay, (float)std::log(o.beta1), (float)std::log(o.beta2), (uint32_t)o.seed, (uint32_t)(o.seed >> 32), count, 0};
  int at = 0;
  do {
    Entry entries[kMany];
    int used = 0;
    long long blocks = 0;
    for (; at < n && used < kMany; ++at) {
      const slim_adamw_tensor &t = tensors[at];
      if (t.n == 0 || !t.grad) continue;
      const long long more = (t.n + kChunk - 1) / kChunk;
      if (blocks + more > 0x7fffffffll) break;
      entries[used++] = Entry{t.param, t.grad, t.m, t.v, static_cast<uint8_t *>(t.m_scales),
                              static_cast<uint8_t *>(t.v_scales), t.n, at, (int)blocks};
      blocks += more;
    }
    bool rest = false;
    for (int i = at; i < n && !rest; ++i) rest = tensors[i].n > 0 && tensors[i].grad;
    numbers.last = !rest;
    if (used == 0) {  // a step without a gradient counts too
      entries[used++] = Entry{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, 0, 0};
      blocks = 1;
    }
    const bool eight = o.bits == 8;
    cudaError_t e;
#define SLIM_ADAMW(G, E)                                                                          \
  (used <= kFew ? launch<G, E, kFew>(entries, used, (int)blocks, numbers, st)                     \
                : launch<G, E, kMany>(entries, used, (int)blocks, numbers, st))
    if (g_f32)
      e = eight ? SLIM_ADAMW(float, true) : SLIM_ADAMW(float, false);
    else
      e = eight ? SLIM_ADAMW(__nv_bfloat16, true) : SLIM_ADAMW(__nv_bfloat16, false);
#undef SLIM_ADAMW
    if (e != cudaSuccess) return e;
    if (!rest) break;
  } while (true);
  return cudaSuccess;
}

}  // namespace slim
