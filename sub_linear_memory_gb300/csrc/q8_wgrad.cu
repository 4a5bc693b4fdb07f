// q8_wgrad.cu -- weight gradient from the 8-bit checkpoint of a product's
// input: dw [n][k] (+)= sum over rows of dy[row][n] x[row][k].
//
// The sum runs over rows, across which the scales of x differ, so the tensor
// cores cannot apply them; but code * 2^e is exactly a bf16 number, and dy is
// bf16.  Eight warps turn each tile of codes into bf16 in shared memory (a
// shift, two masks and one packed multiply for two codes) while the tensor
// cores (kind::f16, both operands MN-major) work on the tile before.
//
// Split: an output tile is 128 (n) x 256 (k), and the rows are cut into steps
// of 64.  All steps of all tiles form one line that is cut evenly over the
// CTAs, so every SM has the same share whatever the shape; a CTA that does not
// hold all steps of a tile leaves a partial tile in the workspace, and a
// second kernel adds the partials in the order of the line.
#include <algorithm>

#include "kernels.h"
#include "q8.h"
#include "q8_tc.cuh"
#include "tma_host.h"

namespace slim {
namespace q8 {
namespace {

constexpr int kCtas = 152;      // one per SM
constexpr int kTn = 128, kTk = 256, kStep = 64;
constexpr int kMinSteps = 4;    // per CTA: a partial tile costs about this much
constexpr int kThreads = 384;   // producer, MMA, two idle, eight converting warps
constexpr int kStages = 4;
constexpr uint32_t kABytes = kStep * kTn * 2, kCBytes = kStep * kTk, kBBytes = kStep * kTk * 2;
constexpr uint32_t kStageBytes = kABytes + kCBytes;
enum {
  S_FULL = 0, S_EMPTY = S_FULL + kStages, S_BFULL = S_EMPTY + kStages, S_BEMPTY = S_BFULL + 2, S_ACC = S_BEMPTY + 2,
  S_ACCFREE, S_COUNT
};
constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + 2 * kBBytes + 256;

struct Cut {
  int steps;        // per tile
  int tiles_k;      // output tiles along k
  long long units;  // tiles * steps
  int ctas;
  __host__ __device__ long long begin(int c) const { return units * c / ctas; }
};

Cut cut_of(int rows, int n, int k) {
  Cut c;
  c.steps = rows / kStep + (rows % kStep != 0);
  c.tiles_k = k / kTk + (k % kTk != 0);
  c.units = (long long)c.steps * c.tiles_k * (n / kTn + (n % kTn != 0));
  c.ctas = (int)std::max<long long>(1, std::min<long long>(kCtas, c.units / kMinSteps));
  return c;
}

// Two e4m3 codes in bytes 0 and 1 (or 2 and 3) of w as bf16 bits: sign and the
// seven bits moved to the top of exponent and fraction, i.e. the value times
// 2^-120 (the exponent biases are 7 and 127; subnormal codes become subnormal
// bf16 numbers).
__device__ __forceinline__ uint32_t widen(uint32_t w, uint32_t sel) {
  const uint32_t t = __byte_perm(w, 0, sel);  // a code in the high byte of each half
  return ((t >> 4) & 0x07f007f0u) | (t & 0x80008000u);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 2^(120 + e) as a pair of equal bf16 numbers for a scale byte, in two factors
// where it is past the type's range (e > 7); NaN for a NaN block.
__device__ __forceinline__ uint32_t factor(int byte, uint32_t &second) {
  second = 0;
  if (byte == kScaleNan) return 0x7fff7fffu;
  const int e = byte - 127;
  const int first = min(120 + e, 127);  // e >= -127
  if (e > 7) {
    const uint32_t s = (uint32_t)(120 + e - first + 127) << 7;
    second = s | (s << 16);
  }
  const uint32_t f = (uint32_t)(first + 127) << 7;
  return f | (f << 16);
}

template <bool TMA_DY>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap mdy, const __grid_constant__ CUtensorMap mx,
                 const __nv_bfloat16 *dy, const uint8_t *scales, float *dw, float *partial, Cut cut, int accumulate,
                 int rows, int n, int k, int pitch, int wide, int *status) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t sbase = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t *smem = raw + (sbase - smem_u32(raw));
  constexpr uint32_t oB = kStages * kStageBytes;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + oB + 2 * kBBytes);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + S_COUNT);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar + S_FULL + s, 1);
      mbar_init(bar + S_EMPTY + s, 9);  // the MMAs and the eight converting warps
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar + S_BFULL + b, 8);
      mbar_init(bar + S_BEMPTY + b, 1);
    }
    mbar_init(bar + S_ACC, 1);
    mbar_init(bar + S_ACCFREE, 8);
    *abort_flag = 0;
    fence_barrier_init();
    if (TMA_DY) prefetch_tmap(&mdy);
    prefetch_tmap(&mx);
  }
  if (warp == 2) tmem_alloc(tslot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const long long u0 = cut.begin(blockIdx.x), u1 = cut.begin(blockIdx.x + 1);
  bool ok = true;
  auto wait = [&](int b, uint32_t par) {
    if (ok) ok = mbar_wait(bar + b, par, status, abort_flag);
    return ok;
  };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + b);
  };

  if (warp == 0 && lane == 0) {
    const int total = (int)(u1 - u0);
    int i = 0;
    for (; i < total; ++i) {
      const int s = i % kStages;
      if (i >= kStages && !wait(S_EMPTY + s, (uint32_t)(i / kStages - 1) & 1)) break;
      const long long u = u0 + i, t = u / cut.steps;
      const int r0 = (int)(u - t * cut.steps) * kStep, n0 = (int)(t / cut.tiles_k) * kTn,
                kk = (int)(t % cut.tiles_k) * kTk;
      const uint32_t at = sbase + s * kStageBytes;
      mbar_arrive_expect_tx(bar + S_FULL + s, (TMA_DY ? kABytes : 0) + kCBytes);
      if (TMA_DY) {
        tma_load_2d(at, &mdy, bar + S_FULL + s, n0, r0);
        tma_load_2d(at + kABytes / 2, &mdy, bar + S_FULL + s, n0 + 64, r0);
      }
      tma_load_2d(at + kABytes, &mx, bar + S_FULL + s, kk, r0);
      tma_load_2d(at + kABytes + kCBytes / 2, &mx, bar + S_FULL + s, kk + kBlock, r0);
    }
    for (int j = max(0, i - kStages); j < i; ++j) mbar_drain(bar + S_FULL + j % kStages, (uint32_t)(j / kStages) & 1);
  } else if (warp == 1 && lane == 0) {
    const uint32_t id = make_idesc(kTn, kTk, true, true);
    int i = 0, seg = 0;
    for (long long u = u0; u < u1 && ok; ++seg) {
      const long long end = min(u1, (u / cut.steps + 1) * cut.steps);
      if (seg > 0 && !wait(S_ACCFREE, (seg - 1) & 1)) break;
      tc_fence_after();
      for (long long first = u; u < end; ++u, ++i) {
        const int s = i % kStages, b = i & 1;
        if (!wait(S_FULL + s, (uint32_t)(i / kStages) & 1) || !wait(S_BFULL + b, (uint32_t)(i >> 1) & 1)) break;
        tc_fence_after();
        const uint64_t da = desc_mnmajor(sbase + s * kStageBytes, kStep, 0, 0);
        const uint64_t db = desc_mnmajor(sbase + oB + b * kBBytes, kStep, 0, 0);
#pragma unroll
        for (int j = 0; j < kStep / 16; ++j)
          mma_bf16(tbase, da + (uint64_t)(j * 128), db + (uint64_t)(j * 128), id, u > first || j > 0);
        mma_commit(bar + S_EMPTY + s);
        mma_commit(bar + S_BEMPTY + b);
      }
      if (ok) mma_commit(bar + S_ACC);
    }
  } else if (warp >= 4) {
    // thread: 16 codes of rows r0 + 16 j, always of the same 128-column block
    const int ct = tid - 128, chunk = ct & 15, row0 = ct >> 4, half = chunk >> 3;
    const uint32_t lanes = 32u * (warp & 3);
    int i = 0, seg = 0;
    for (long long u = u0; u < u1 && ok; ++seg) {
      const long long t = u / cut.steps, end = min(u1, (t + 1) * cut.steps);
      const bool whole = u == t * cut.steps && end == (t + 1) * cut.steps, first_seg = u == u0;
      const int n0 = (int)(t / cut.tiles_k) * kTn, kk = (int)(t % cut.tiles_k) * kTk;
      const int blk = kk / kBlock + half;
      const bool has = blk * kBlock < k;
      auto scale_at = [&](long long step, int j) {
        const long long r = step * kStep + row0 + 16 * j;
        return has && r < rows ? (int)__ldg(scales + (size_t)r * pitch + blk) : 127;
      };
      int byte[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) byte[j] = scale_at(u - t * cut.steps, j);
      for (; u < end; ++u, ++i) {
        const int s = i % kStages, b = i & 1;
        if (!wait(S_FULL + s, (uint32_t)(i / kStages) & 1)) break;
        uint4 code[4];
        const uint32_t from = sbase + s * kStageBytes + kABytes + half * (kCBytes / 2) + (chunk & 7) * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ld_shared_v4(from + (row0 + 16 * j) * kBlock, code[j].x, code[j].y, code[j].z, code[j].w);
        int next[4];
        const long long step = u - t * cut.steps;
#pragma unroll
        for (int j = 0; j < 4; ++j) next[j] = u + 1 < end ? scale_at(step + 1, j) : 127;
        if (!TMA_DY) {  // rows that TMA cannot step over: this warp group's own loads into the same layout
          for (int x = ct; x < kStep * kTn; x += 256) {
            const int r = x / kTn, c = x % kTn;
            const long long gr = step * kStep + r;
            const __nv_bfloat16 v = gr < rows && n0 + c < n ? dy[(size_t)gr * n + n0 + c] : __float2bfloat16_rn(0.f);
            *reinterpret_cast<__nv_bfloat16 *>(smem + s * kStageBytes + sw128_offset(r, c, kStep)) = v;
          }
        }
        if (i >= 2 && !wait(S_BEMPTY + b, (uint32_t)((i >> 1) - 1) & 1)) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t second;
          const uint32_t f = factor(byte[j], second);
          const uint32_t w[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * e] = mul_bf16x2(widen(w[e], 0x1404), f);
            o[2 * e + 1] = mul_bf16x2(widen(w[e], 0x3424), f);
          }
          if (second) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(o[e], second);
          }
          const int r = row0 + 16 * j;
          const uint32_t to = sbase + oB + b * kBBytes;
          // the two 16-byte halves in an order that keeps a warp's stores on distinct banks
          const uint32_t a0 = to + sw128_offset(r, 16 * chunk, kStep), a1 = to + sw128_offset(r, 16 * chunk + 8, kStep);
          if (chunk & 4) {
            st_shared_v4(a1, o[4], o[5], o[6], o[7]);
            st_shared_v4(a0, o[0], o[1], o[2], o[3]);
          } else {
            st_shared_v4(a0, o[0], o[1], o[2], o[3]);
            st_shared_v4(a1, o[4], o[5], o[6], o[7]);
          }
          byte[j] = next[j];
        }
        fence_async_smem();
        arrive(S_BFULL + b);
        arrive(S_EMPTY + s);
      }
      if (!wait(S_ACC, seg & 1)) break;
      tc_fence_after();
      // this thread's row of the tile, 128 of its 256 columns: into dw, or into this CTA's partial tile
      const int nr = (int)lanes + lane, c0 = warp < 8 ? 0 : 128;
      float *to = whole ? dw + (size_t)(n0 + nr) * k + kk
                        : partial + ((size_t)blockIdx.x * 2 + (first_seg ? 0 : 1)) * (kTn * kTk) + (size_t)nr * kTk;
      const int left = whole ? (n0 + nr < n ? k - kk : 0) : kTk;
      const bool vec = !whole || wide, add = whole && accumulate;
      for (int c = c0; c < c0 + 128; c += 32) {
        float v[32];
        __syncwarp();
        tmem_ld32(tmem_addr(tbase, lanes, c), v);
        if (vec) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            if (c + e < left) {
              float4 *p = reinterpret_cast<float4 *>(to + c + e);
              float4 x = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
              if (add) {
                const float4 o = *p;
                x.x += o.x; x.y += o.y; x.z += o.z; x.w += o.w;
              }
              *p = x;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c + e < left) to[c + e] = add ? to[c + e] + v[e] : v[e];
        }
      }
      tc_fence_before();
      arrive(S_ACCFREE);
    }
  }
  __syncthreads();
  if (warp == 2) tmem_dealloc(tbase, 256);
}

// dw of the tiles that several CTAs share: one CTA for 32 rows of such a tile.
__global__ void __launch_bounds__(256) wgrad_join_kernel(const float *partial, float *dw, Cut cut, int accumulate, int n,
                                                         int k) {
  const long long t = blockIdx.x, first = t * cut.steps, last = first + cut.steps - 1;
  // the CTA that holds unit u: the largest c with begin(c) <= u
  auto owner = [&](long long u) {
    int c = (int)(u * cut.ctas / cut.units);
    while (cut.begin(c + 1) <= u) ++c;
    while (cut.begin(c) > u) --c;
    return c;
  };
  const int ca = owner(first), cb = owner(last);
  if (ca == cb) return;  // held by one CTA, written in full
  const int n0 = (int)(t / cut.tiles_k) * kTn, kk = (int)(t % cut.tiles_k) * kTk;
  for (int x = threadIdx.x; x < 32 * kTk; x += 256) {
    const int r = blockIdx.y * 32 + x / kTk, c = x % kTk;
    if (n0 + r >= n || kk + c >= k) continue;
    float v = 0.f;
    for (int i = ca; i <= cb; ++i) {
      // a CTA's first segment lies in slot 0; a later one, which begins its tile, in slot 1
      const int slot = cut.begin(i) / cut.steps == t ? 0 : 1;
      v += partial[((size_t)i * 2 + slot) * (kTn * kTk) + (size_t)r * kTk + c];
    }
    float *to = dw + (size_t)(n0 + r) * k + kk + c;
    *to = accumulate ? *to + v : v;
  }
}

}  // namespace

size_t wgrad_workspace(int rows, int n, int k) {
  if (rows == 0 || n == 0 || k == 0) return 0;
  return (size_t)cut_of(rows, n, k).ctas * 2 * kTn * kTk * sizeof(float);
}

cudaError_t wgrad(const void *dy, const void *x_codes, const void *x_scales, float *dw, bool accumulate,
                  void *workspace, int rows, int n, int k, int *status, cudaStream_t st) {
  const Cut cut = cut_of(rows, n, k);
  const bool tma = n % 8 == 0 && (reinterpret_cast<uintptr_t>(dy) & 15) == 0;
  CUtensorMap mdy, mx;
  const uint64_t kp = (uint64_t)blocks_of(k) * kBlock;
  if (!make_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x_codes, rows, kp, kp, kStep, kBlock, false))
    return cudaErrorInvalidValue;
  mdy = mx;
  if (tma && !make_map_2d(&mdy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, rows, n, (uint64_t)n * 2, kStep, 64, true))
    return cudaErrorInvalidValue;
  auto kern = tma ? wgrad_kernel<true> : wgrad_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  {
    ProfScope ps("q8_wgrad", st);
    kern<<<cut.ctas, kThreads, kSmem, st>>>(mdy, mx, static_cast<const __nv_bfloat16 *>(dy),
                                            static_cast<const uint8_t *>(x_scales), dw,
                                            static_cast<float *>(workspace), cut, accumulate ? 1 : 0, rows, n, k,
                                            scale_pitch(k),
                                            k % 4 == 0 && (reinterpret_cast<uintptr_t>(dw) & 15) == 0, status);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || cut.ctas == 1) return e;
  ProfScope ps("q8_wgrad_join", st);
  wgrad_join_kernel<<<dim3((unsigned)(cut.units / cut.steps), kTn / 32), 256, 0, st>>>(
      static_cast<const float *>(workspace), dw, cut, accumulate ? 1 : 0, n, k);
  return cudaGetLastError();
}

}  // namespace q8
}  // namespace slim
