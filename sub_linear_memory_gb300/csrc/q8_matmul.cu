// q8_matmul.cu -- out [rows][n] = a [rows][k] . b [n][k]^T for 8-bit rows a
// (a scale for each row and 128 columns) and a packed weight b (a scale for
// each 128 x 128 block).
//
// The tensor cores multiply e4m3 codes and apply the scales themselves
// (kind::mxf8f6f4, one E8M0 scale for each row and 32 columns: the four 32s of
// a 128-column block read the same byte), so partial sums never leave the fp32
// accumulator between blocks.
#include <algorithm>

#include "kernels.h"
#include "q8.h"
#include "q8_tc.cuh"
#include "tma_host.h"

namespace slim {
namespace q8 {
namespace {

// ---- few output tiles: weights as the MMA's M side, k split over a cluster ------
//
// A tile is 128 weight rows x up to 128 rows of a.  The accumulator's lanes
// are weight rows, so a warp writes 32 neighbouring columns of out, and the
// MMA's N is only as wide as the rows of a (16 for one token).  The CTAs of a
// cluster take a share of k each and add their partial tiles in the order of
// their ranks through distributed shared memory.
namespace sm {

constexpr int kThreads = 256, kStages = 4, kMaxQuads = 48;
enum { S_FULL = 0, S_EMPTY = S_FULL + kStages, S_SF = S_EMPTY + kStages, S_DONE, S_COUNT };
constexpr uint32_t kW = kBlock * kBlock;  // bytes of a weight tile

__host__ __device__ constexpr uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__host__ __device__ constexpr uint32_t stage_bytes(int nt) { return kW + (uint32_t)(nt + 7) / 8 * 1024u; }
// At least 200 KB, so that no other CTA with tensor memory shares the SM: one
// that waited here for the columns of a CTA whose cluster waits elsewhere for
// another's would never get them.
__host__ __device__ constexpr uint32_t smem_bytes(int nt, bool split) {
  return max_u32(200u << 10, 1024u + kStages * stage_bytes(nt) + (split ? (uint32_t)nt * kBlock * 4u : 0u) + 256u);
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
    matmul_small_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap ma,
                        const uint8_t *a_scales, const uint8_t *b_scales, void *out, int rows, int n, int kb,
                        int pitch, int nt, int *status) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t sbase = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t *smem = raw + (sbase - smem_u32(raw));
  const int split = (int)gridDim.x, rank = (int)blockIdx.x;
  const uint32_t sb = stage_bytes(nt);
  float *part = reinterpret_cast<float *>(smem + kStages * sb);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kStages * sb + (split > 1 ? nt * kBlock * 4 : 0));
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + S_COUNT);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = blockIdx.y * kBlock, m0 = blockIdx.z * kBlock;
  const int k0 = (int)((long long)kb * rank / split), k1 = (int)((long long)kb * (rank + 1) / split), nk = k1 - k0;
  const int quads = (nk + 3) / 4;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar + S_FULL + s, 1);
      mbar_init(bar + S_EMPTY + s, 1);
    }
    mbar_init(bar + S_SF, 4);
    mbar_init(bar + S_DONE, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&mw);
    prefetch_tmap(&ma);
  }
  if (warp == 2) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  // TMEM columns: accumulator 0-127, then 8 for each quad of blocks (scale
  // words of the weight rows, of the rows of a)
  constexpr uint32_t t_sf = 128;
  bool ok = true;
  auto wait = [&](int b, uint32_t par) {
    if (ok) ok = mbar_wait(bar + b, par, status, abort_flag);
    return ok;
  };

  if (warp == 0 && lane == 0) {
    int i = 0;
    for (; i < nk; ++i) {
      const int s = i % kStages;
      if (i >= kStages && !wait(S_EMPTY + s, (i / kStages - 1) & 1)) break;
      mbar_arrive_expect_tx(bar + S_FULL + s, kW + (uint32_t)nt * kBlock);
      tma_load_2d(sbase + s * sb, &mw, bar + S_FULL + s, (k0 + i) * kBlock, n0);
      tma_load_2d(sbase + s * sb + kW, &ma, bar + S_FULL + s, (k0 + i) * kBlock, m0);
    }
    for (int j = max(0, i - kStages); j < i; ++j) mbar_drain(bar + S_FULL + j % kStages, (j / kStages) & 1);
  } else if (warp == 1 && lane == 0) {
    if (wait(S_SF, 0)) {
      for (int i = 0; i < nk; ++i) {
        const int s = i % kStages;
        if (!wait(S_FULL + s, (i / kStages) & 1)) break;
        tc_fence_after();
        const uint32_t id = make_idesc_mx8(128, nt, i & 3);
        const uint32_t sf = tbase + t_sf + (i >> 2) * 8;
        const uint64_t da = make_desc(sbase + s * sb, 16u, 1024u, kSwizzle128);
        const uint64_t db = make_desc(sbase + s * sb + kW, 16u, 1024u, kSwizzle128);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_mx8(tbase, da + 2 * j, db + 2 * j, id, sf, sf + 4, i > 0 || j > 0);
        mma_commit(bar + S_EMPTY + s);
      }
    }
    mma_commit(bar + S_DONE);
    mbar_drain(bar + S_DONE, 0);
  } else if (warp >= 4) {
    // scale words of this CTA's blocks; rows past the end take scale 1 (their codes are zero)
    const uint32_t lanes = 32u * (warp & 3);
    const uint8_t *bs = b_scales + (size_t)blockIdx.y * pitch + k0;
    for (int q = 0; q < quads; ++q) {
      uint32_t w = 0, a[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kk = 4 * q + j;
        w |= (kk < nk ? (uint32_t)__ldg(bs + kk) : 127u) << (8 * j);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int m = m0 + 32 * g + lane;
          const bool on = kk < nk && m < rows && 32 * g < nt;
          a[g] |= (on ? (uint32_t)__ldg(a_scales + (size_t)m * pitch + k0 + kk) : 127u) << (8 * j);
        }
      }
      const uint32_t at = tmem_addr(tbase, lanes, t_sf + 8 * q);
      tmem_st4u(at, w, w, w, w);
      tmem_st4u(at + 4, a[0], a[1], a[2], a[3]);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + S_SF);
    const bool full = wait(S_DONE, 0);
    tc_fence_after();
    const int nn = n0 + 32 * (warp & 3) + lane;
    const int cols = min(nt, rows - m0);
    if (full) {
      for (int c = 0; c < cols; c += 16) {
        float v[16];
        tmem_ld16(tmem_addr(tbase, lanes, c), v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (split > 1) {
            part[(c + i) * kBlock + 32 * (warp & 3) + lane] = v[i];
          } else if (c + i < cols && nn < n) {
            const size_t at = (size_t)(m0 + c + i) * n + nn;
            if (F32) static_cast<float *>(out)[at] = v[i];
            else static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v[i]);
          }
        }
      }
    }
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();
    const int cols = min(nt, rows - m0), nl = tid & (kBlock - 1);
    const uint32_t mine = smem_u32(part);
    if (!*abort_flag && n0 + nl < n) {
      for (int c = rank + split * (tid >> 7); c < cols; c += 2 * split) {
        float x = 0.f;
        for (int r = 0; r < split; ++r) x += ld_peer_f32(map_peer(mine + (uint32_t)(c * kBlock + nl) * 4u, r));
        const size_t at = (size_t)(m0 + c) * n + n0 + nl;
        if (F32) static_cast<float *>(out)[at] = x;
        else static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(x);
      }
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  } else {
    __syncthreads();
  }
  if (warp == 2) tmem_dealloc(tbase, 512);
}

template <bool F32>
cudaError_t launch(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales, void *out,
                   int rows, int n, int k, int *status, cudaStream_t st) {
  const int kb = blocks_of(k), tiles_n = blocks_of(n), tiles_m = blocks_of(rows);
  const int nt = rows >= kBlock ? kBlock : (rows + 15) / 16 * 16;
  // k is split until the SMs have a CTA each, two blocks or more to a CTA
  int split = 1;
  while (split < 8 && 2 * split * (long long)tiles_n * tiles_m <= 152 && 4 * split <= kb) split *= 2;
  while (split < 8 && (kb + split - 1) / split > 4 * kMaxQuads - 4) split *= 2;
  CUtensorMap mw, ma;
  const uint64_t kp = (uint64_t)kb * kBlock;
  if (!make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, b_codes, n, kp, kp, kBlock, kBlock, true) ||
      !make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, rows, kp, kp, nt, kBlock, true))
    return cudaErrorInvalidValue;
  auto kern = matmul_small_kernel<F32>;
  const uint32_t smem = smem_bytes(nt, split > 1);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kBlock, true));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split, tiles_n, tiles_m);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ProfScope ps("q8_matmul_small", st);
  e = cudaLaunchKernelEx(&cfg, kern, mw, ma, static_cast<const uint8_t *>(a_scales),
                         static_cast<const uint8_t *>(b_scales), out, rows, n, kb, scale_pitch(k), nt, status);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace sm
}  // namespace

cudaError_t matmul(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales, void *out,
                   bool f32, int rows, int n, int k, int *status, cudaStream_t st) {
  return f32 ? sm::launch<true>(a_codes, a_scales, b_codes, b_scales, out, rows, n, k, status, st)
             : sm::launch<false>(a_codes, a_scales, b_codes, b_scales, out, rows, n, k, status, st);
}

}  // namespace q8
}  // namespace slim
