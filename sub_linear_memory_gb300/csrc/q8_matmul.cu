// q8_matmul.cu -- out [rows][n] = a [rows][k] . b [n][k]^T for 8-bit rows a
// (a scale for each row and 128 columns) and a packed weight b (a scale for
// each 128 x 128 block).
//
// The tensor cores multiply e4m3 codes and apply the scales themselves
// (kind::mxf8f6f4, one E8M0 scale for each row and 32 columns: the four 32s of
// a 128-column block read the same byte), so partial sums need not leave the
// fp32 accumulator between blocks.
//
// Rounding: the tensor cores add into that accumulator with truncation, four
// times a block.  For operands of one sign (|normal| numbers) that takes 1.5e-6
// of the result for k = 4096, 9.9e-6 for 16384 and 1.6e-4 for 131072.  An fp32
// result is therefore the sum, with rounding to nearest, of parts of 32 blocks
// each: 1.5e-6 at every k (8192 x 4096 x 8192 then takes 178 us, 165 with one
// accumulator; 4096 x 4096 x 16384 190 and 171).  A bf16 result keeps one
// accumulator: its own rounding is 2^-8.
#include <algorithm>

#include "kernels.h"
#include "q8.h"
#include "q8_tc.cuh"
#include "tma_host.h"

namespace slim {
namespace q8 {
namespace {

constexpr int kSumBlocks = 32;  // blocks of k that go into one accumulator where out is fp32
// The end of the part of k that starts at block k0 of kb.
template <bool F32> __device__ __forceinline__ int part_end(int k0, int kb) {
  return F32 && kb - k0 > kSumBlocks ? k0 + kSumBlocks : kb;
}

// ---- few rows: weights as the MMA's M side, k split over a cluster ----------------
//
// A tile is 128 weight rows x all rows of a, up to 128.  The accumulator's
// lanes are weight rows, so a warp writes neighbouring columns of out, and the
// MMA's N is only as wide as the rows of a (16 for one token).  What bounds it
// is latency: the CTAs of a cluster take a share of k each, so that the weight
// comes through as many SMs as there are, and add their partial tiles in the
// order of their ranks through distributed shared memory.  In a graph, one
// token: 4.5 us for 1024 x 4096 (12.3 with k in one piece), 4.0 for 4096 x
// 1024; 128 tokens: 8.9 (19.6) and 8.2 (11.6).
namespace sm {

constexpr int kThreads = 256, kStages = 4, kMaxQuads = 48;
enum {
  S_FULL = 0, S_EMPTY = S_FULL + kStages, S_SF = S_EMPTY + kStages, S_PART, S_PARTFREE, S_DONE, S_COUNT
};
constexpr uint32_t kW = kBlock * kBlock;  // bytes of a weight tile

__host__ __device__ constexpr uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
__host__ __device__ constexpr uint32_t stage_bytes(int nt) { return kW + (uint32_t)(nt + 7) / 8 * 1024u; }
// At least 200 KB, so that no other CTA with tensor memory shares the SM: one
// that waited here for the columns of a CTA whose cluster waits elsewhere for
// another's would never get them.
__host__ __device__ constexpr uint32_t smem_bytes(int nt) {
  return max_u32(200u << 10, 1024u + kStages * stage_bytes(nt) + (uint32_t)nt * kBlock * 4u + 256u);
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
    matmul_small_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap ma,
                        const uint8_t *a_scales, const uint8_t *b_scales, void *out, int rows, int n, int kb,
                        int pitch, int nt, int wide, int *status) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t sbase = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t *smem = raw + (sbase - smem_u32(raw));
  const int split = (int)gridDim.x, rank = (int)blockIdx.x;
  const uint32_t sb = stage_bytes(nt);
  float *part = reinterpret_cast<float *>(smem + kStages * sb);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kStages * sb + nt * kBlock * 4);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + S_COUNT);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = blockIdx.y * kBlock;
  const int k0 = (int)((long long)kb * rank / split), k1 = (int)((long long)kb * (rank + 1) / split), nk = k1 - k0;
  const int quads = (nk + 3) / 4;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar + S_FULL + s, 1);
      mbar_init(bar + S_EMPTY + s, 1);
    }
    mbar_init(bar + S_SF, 4);
    mbar_init(bar + S_PART, 1);
    mbar_init(bar + S_PARTFREE, 4);
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
      tma_load_2d(sbase + s * sb + kW, &ma, bar + S_FULL + s, (k0 + i) * kBlock, 0);
    }
    for (int j = max(0, i - kStages); j < i; ++j) mbar_drain(bar + S_FULL + j % kStages, (j / kStages) & 1);
  } else if (warp == 1 && lane == 0) {
    if (wait(S_SF, 0)) {
      for (int i = 0, first = 0, part_no = 0; i < nk; ++i) {
        if (F32 && i - first == kSumBlocks) {  // the accumulator is emptied before the next block starts it anew
          mma_commit(bar + S_PART);
          if (!wait(S_PARTFREE, part_no & 1)) break;
          tc_fence_after();
          first = i;
          ++part_no;
        }
        const int s = i % kStages;
        if (!wait(S_FULL + s, (i / kStages) & 1)) break;
        tc_fence_after();
        const uint32_t id = make_idesc_mx8(128, nt, i & 3);
        const uint32_t sf = tbase + t_sf + (i >> 2) * 8;
        const uint64_t da = make_desc(sbase + s * sb, 16u, 1024u, kSwizzle128);
        const uint64_t db = make_desc(sbase + s * sb + kW, 16u, 1024u, kSwizzle128);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_mx8(tbase, da + 2 * j, db + 2 * j, id, sf, sf + 4, i > first || j > 0);
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
          const int m = 32 * g + lane;
          const bool on = kk < nk && m < rows;
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
    // The parts before the last are added up in shared memory; each thread has
    // a weight row's elements for itself.
    float *mine = part + 32 * (warp & 3) + lane;
    const int parts = F32 ? (nk + kSumBlocks - 1) / kSumBlocks : 1;
    for (int p = 0; p < parts - 1; ++p) {
      wait(S_PART, p & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      for (int c = 0; c < rows; c += 16) {
        float v[16];
        tmem_ld16(tmem_addr(tbase, lanes, c), v);
#pragma unroll
        for (int i = 0; i < 16; ++i) mine[(c + i) * kBlock] = p > 0 ? mine[(c + i) * kBlock] + v[i] : v[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + S_PARTFREE);
    }
    wait(S_DONE, 0);
    tc_fence_after();
    const int nn = n0 + 32 * (warp & 3) + lane;
    if (__all_sync(0xffffffffu, ok)) {
      for (int c = 0; c < rows; c += 16) {
        float v[16];
        tmem_ld16(tmem_addr(tbase, lanes, c), v);
        if (parts > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += mine[(c + i) * kBlock];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (split > 1) {
            mine[(c + i) * kBlock] = v[i];
          } else if (c + i < rows && nn < n) {
            const size_t at = (size_t)(c + i) * n + nn;
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
    // Four neighbouring columns of out a thread; a CTA takes every split-th
    // group of 8 rows.  All loads of a group are under way together: they cross
    // the SMs, and one after the other took most of the kernel (12.3 us for 128
    // rows x 4096 x 1024).
    const int nl = 4 * lane, left = n - n0 - nl;
    const uint32_t tile = smem_u32(part);
    if (!*abort_flag && left > 0) {
      for (int c = 8 * rank + warp; c < rows; c += 8 * split) {
        float v[8][4];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < split) ld_peer_v4(map_peer(tile + (uint32_t)(c * kBlock + nl) * 4u, r), v[r]);
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < split) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[0][e] += v[r][e];
          }
        const size_t at = (size_t)c * n + n0 + nl;
        if (F32) {
          float *to = static_cast<float *>(out) + at;
          if (wide) {
            *reinterpret_cast<float4 *>(to) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e < left) to[e] = v[0][e];
          }
        } else {
          __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(out) + at;
          if (wide) {
            *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (e < left) to[e] = __float2bfloat16_rn(v[0][e]);
          }
        }
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
  const int kb = blocks_of(k), tiles_n = blocks_of(n), nt = (rows + 15) / 16 * 16;
  // k is split until the SMs have a CTA each, two blocks or more to a CTA
  int split = 1;
  while (split < 8 && 2 * split * (long long)tiles_n <= 152 && 4 * split <= kb) split *= 2;
  while (split < 8 && (kb + split - 1) / split > 4 * kMaxQuads - 4) split *= 2;
  CUtensorMap mw, ma;
  const uint64_t kp = (uint64_t)kb * kBlock;
  if (!make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, b_codes, n, kp, kp, kBlock, kBlock, true) ||
      !make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, rows, kp, kp, nt, kBlock, true))
    return cudaErrorInvalidValue;
  // four columns of out in one store
  const int wide = n % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (F32 ? 15 : 7)) == 0;
  auto kern = matmul_small_kernel<F32>;
  const uint32_t smem = smem_bytes(nt);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(kBlock));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split, tiles_n);
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
                         static_cast<const uint8_t *>(b_scales), out, rows, n, kb, scale_pitch(k), nt, wide, status);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace sm

// ---- more rows: a CTA pair for each 256 x 256 tile ---------------------------------
//
// Two SMs work on one tile (cta_group::2), each loads half of either operand,
// so a 128-byte step of k moves 32 KB into each SM's shared memory for 512
// cycles of MMA.  Pairs walk the tiles; one warp loads, one thread of the pair
// issues, four warps put the scale words into tensor memory (512 columns of k
// at a time), four warps turn the finished accumulator into rows of out while
// the next tile is multiplied into the other one.
//
// 65536 x 4096 x 1024: 178 us, 3.09 PFLOP/s; 16384 x 4096 x 4096 154 us, 3.56
// PFLOP/s (1.6 and 1.9 times the measured bf16 rate; a sustained loop meets
// the power limit, 204 us at 1.53 GHz).  What bounds it are the operands' way
// into shared memory, which the MMAs read at the same time, and at short k the
// hand-over between the two accumulators.  Tiles of 192 and 128 columns were
// slower (262 and 306 against 251 us), as they load more for each product.
namespace lg {

constexpr int kThreads = 384, kStages = 6, kTm = 256, kTn = 256;
constexpr uint32_t kA = kBlock * kBlock;
constexpr uint32_t kOut = 4096;  // one warp's 32 rows x 128 bytes of out
enum {
  S_FULL = 0, S_EMPTY = S_FULL + kStages, S_SF = S_EMPTY + kStages, S_SFFREE = S_SF + 2, S_ACC = S_SFFREE + 2,
  S_ACCFREE = S_ACC + 2, S_DONE, S_COUNT
};

constexpr uint32_t kB = kTn / 2 * kBlock, kStage = kA + kB;
constexpr uint32_t kOutAt = kStages * kStage, kBar = kOutAt + 8 * kOut, kSmem = 1024 + kBar + 256;
// Tensor memory: two accumulators, and two sets of 12 scale columns from
// column 480 on.  Two of 256 columns do not fit beside those, so they share 32
// columns, which the epilogue reads first.
constexpr uint32_t kSf = 480, kAcc1 = kSf - kTn;

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                  const __grid_constant__ CUtensorMap mo, const uint8_t *a_scales, const uint8_t *b_scales, void *out,
                  int rows, int n, int kb, int pitch, int tiles_n, int tiles, int tma_out, int *status) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t sbase = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t *smem = raw + (sbase - smem_u32(raw));
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kBar);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + S_COUNT);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar + S_FULL + s, 1);
      mbar_init(bar + S_EMPTY + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar + S_SF + b, 8);  // four warps of each CTA
      mbar_init(bar + S_SFFREE + b, 1);
      mbar_init(bar + S_ACC + b, 1);
    }
    mbar_init(bar + S_ACCFREE, 8);
    mbar_init(bar + S_DONE, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&ma);
    prefetch_tmap(&mb);
    if (tma_out) prefetch_tmap(&mo);
  }
  if (warp == 2) tmem_alloc_pair(tslot, 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  bool ok = true;
  auto wait = [&](int b, uint32_t par) {
    if (ok) ok = mbar_wait(bar + b, par, status, abort_flag);
    return ok;
  };
  auto wait_warp = [&](int b, uint32_t par) {  // called by a whole warp, whose lanes agree on the result
    wait(b, par);
    return ok = __all_sync(0xffffffffu, ok);
  };
  // arrive on the leading CTA's barrier, once for the warp
  auto arrive_leader = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(map_peer(smem_u32(bar + b), 0));
  };

  if (warp == 0 && lane == 0) {
    int i = 0;
    for (int t = pair; t < tiles && ok; t += pairs) {
      const int m0 = t / tiles_n * kTm + (int)rank * kBlock, n0 = t % tiles_n * kTn + (int)rank * (kTn / 2);
      for (int kk = 0; kk < kb; ++kk, ++i) {
        const int s = i % kStages;
        if (i >= kStages && !wait(S_EMPTY + s, (uint32_t)(i / kStages - 1) & 1)) break;
        if (rank == 0) mbar_arrive_expect_tx(bar + S_FULL + s, 2 * kStage);
        const uint32_t full = map_peer(smem_u32(bar + S_FULL + s), 0), at = sbase + s * kStage;
        tma_load_2d_pair(at, &ma, full, kk * kBlock, m0);
        tma_load_2d_pair(at + kA, &mb, full, kk * kBlock, n0);
      }
    }
    if (rank == 0)
      for (int j = max(0, i - kStages); j < i; ++j) mbar_drain(bar + S_FULL + j % kStages, (uint32_t)(j / kStages) & 1);
  } else if (warp == 1 && rank == 0) {
    const bool issues = elect_lane();
    // a tile and a part of k (all of k where out is bf16) for each accumulator
    int i = 0, quad = 0, j = 0;
    for (int t = pair, k0 = 0; t < tiles && ok; ++j) {
      // the accumulator's columns are free: those that it shares with the last
      // one have been read, so all of the one's before that too
      if (j > 0 && !wait_warp(S_ACCFREE, (uint32_t)(j - 1) & 1)) break;
      tc_fence_after();
      const uint32_t acc = tbase + (j & 1 ? kAcc1 : 0);
      const int k1 = part_end<F32>(k0, kb);
      for (int kk = k0; kk < k1; ++kk, ++i) {
        const uint32_t sf = tbase + kSf + 12 * (quad & 1);
        if ((kk & 3) == 0 && !wait_warp(S_SF + (quad & 1), (uint32_t)(quad >> 1) & 1)) break;
        const int s = i % kStages;
        if (!wait_warp(S_FULL + s, (uint32_t)(i / kStages) & 1)) break;
        tc_fence_after();
        const uint32_t id = make_idesc_mx8(kTm, kTn, kk & 3);
        const uint64_t da = make_desc(sbase + s * kStage, 16u, 1024u, kSwizzle128);
        const uint64_t db = make_desc(sbase + s * kStage + kA, 16u, 1024u, kSwizzle128);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (issues) mma_mx8_pair(acc, da + 2 * x, db + 2 * x, id, sf, sf + 4, kk > k0 || x > 0);
        if (issues) mma_commit_pair(bar + S_EMPTY + s);
        if ((kk & 3) == 3 || kk == kb - 1) {
          if (issues) mma_commit_pair(bar + S_SFFREE + (quad & 1));
          ++quad;
        }
        __syncwarp();
      }
      if (ok && issues) mma_commit_pair(bar + S_ACC + (j & 1));
      __syncwarp();
      k0 = k1 < kb ? k1 : 0;
      if (k0 == 0) t += pairs;
    }
    if (issues) mma_commit_pair(bar + S_DONE);
    __syncwarp();
    mbar_drain(bar + S_DONE, 0);
  } else if (warp >= 4 && warp < 8) {
    // scale words of 4 blocks of k at a time: 128 rows of a (this CTA's), kTn
    // rows of b.  The words of the next 4 blocks (of the next tile, at the end
    // of one) are on their way from memory while these wait for their columns:
    // loaded only then, a first load from DRAM would hold up the MMAs.
    const uint32_t at0 = tmem_addr(tbase, 32u * (warp & 3), kSf);
    constexpr uint32_t kOnes = 0x7f7f7f7fu;
    struct Words {
      uint32_t a[4], b[kTn / kBlock];
    };
    auto fetch = [&](int t, int kk, Words &w) {
      const int m0 = t / tiles_n * kTm + (int)rank * kBlock, n0 = t % tiles_n * kTn;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int m = m0 + 32 * g + lane;
        w.a[g] = m < rows ? __ldg(reinterpret_cast<const uint32_t *>(a_scales + (size_t)m * pitch + kk)) : kOnes;
      }
#pragma unroll
      for (int g = 0; g < kTn / kBlock; ++g) {
        const int blk = n0 / kBlock + g;
        w.b[g] = blk * kBlock < n ? __ldg(reinterpret_cast<const uint32_t *>(b_scales + (size_t)blk * pitch + kk)) : kOnes;
      }
    };
    int quad = 0;
    Words now, next;
    if (pair < tiles) fetch(pair, 0, next);
    for (int t = pair; t < tiles && ok; t += pairs) {
      for (int kk = 0; kk < kb; kk += 4, ++quad) {
        now = next;
        if (kk + 4 < kb) fetch(t, kk + 4, next);
        else if (t + pairs < tiles) fetch(t + pairs, 0, next);
        if (quad >= 2 && !wait_warp(S_SFFREE + (quad & 1), (uint32_t)((quad >> 1) - 1) & 1)) break;
        tc_fence_after();
        const uint32_t at = at0 + 12 * (quad & 1);
        const uint32_t b0 = now.b[0], b1 = now.b[1];
        __syncwarp();
        tmem_st4u(at, now.a[0], now.a[1], now.a[2], now.a[3]);
        tmem_st4u(at + 4, b0, b0, b0, b0);
        tmem_st4u(at + 8, b1, b1, b1, b1);
        tmem_st_wait();
        tc_fence_before();
        arrive_leader(S_SF + (quad & 1));
      }
    }
  } else if (warp >= 8) {
    const int w = warp - 8;
    const uint32_t lanes = 32u * w;
    constexpr int kCols = F32 ? 32 : 64;  // 128 bytes of a row of out
    constexpr int kChunks = kTn / kCols;
    int j = 0, turn = 0;
    for (int t = pair, k0 = 0; t < tiles && ok; ++j) {
      const int m0 = t / tiles_n * kTm + (int)rank * kBlock + 32 * w, n0 = t % tiles_n * kTn;
      if (!wait_warp(S_ACC + (j & 1), (uint32_t)(j >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t acc = j & 1 ? kAcc1 : 0;
      // the parts of k after the first are added to out, each once the part
      // before it has been written (single elements: by the same thread)
      const bool add = k0 > 0;
      if (add && tma_out && lane == 0) tma_store_wait_all();
      for (int x = 0; x < kChunks; ++x) {
        // the columns shared with the other accumulator first: the last of the first, the first of the second
        const int c = (j & 1 ? x : kChunks - 1 - x) * kCols;
        float v[kCols];
        __syncwarp();
        if constexpr (F32) tmem_ld32(tmem_addr(tbase, lanes, acc + c), v);
        else tmem_ld32x2(tmem_addr(tbase, lanes, acc + c), tmem_addr(tbase, lanes, acc + c + 32), v, v + 32);
        if (x == 0) {
          tc_fence_before();
          arrive_leader(S_ACCFREE);
        }
        if (m0 >= rows || n0 + c >= n) continue;  // uniform over the warp
        const uint32_t buf = sbase + kOutAt + (2 * w + (turn & 1)) * kOut;
        ++turn;
        // the store that last read this buffer is done reading
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t to = buf + lane * 128u + ((uint32_t)(q ^ (lane & 7)) << 4);
          if constexpr (F32)
            st_shared_v4(to, __float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                         __float_as_uint(v[4 * q + 3]));
          else
            st_bf16x8(to, v + 8 * q);
        }
        if (tma_out) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (add) tma_reduce_add_2d(&mo, buf, n0 + c, m0);
            else tma_store_2d(&mo, buf, n0 + c, m0);
            tma_store_commit();
          }
        } else {  // rows of out that do not start on 16 bytes: coalesced stores of single elements
          __syncwarp();
          const int live = min(32, rows - m0), left = n - n0 - c;
          for (int r = 0; r < live; ++r) {
#pragma unroll
            for (int h = 0; h < kCols / 32; ++h) {
              const int col = lane + 32 * h;
              const uint32_t bytes = (uint32_t)col * (128 / kCols);
              const uint8_t *from = smem + (buf - sbase) + r * 128 + (((bytes >> 4) ^ (r & 7)) << 4) + (bytes & 15);
              const size_t to = (size_t)(m0 + r) * n + n0 + c + col;
              if (col < left) {
                if constexpr (F32) {
                  const float v = *reinterpret_cast<const float *>(from);
                  static_cast<float *>(out)[to] = add ? static_cast<float *>(out)[to] + v : v;
                } else static_cast<__nv_bfloat16 *>(out)[to] = *reinterpret_cast<const __nv_bfloat16 *>(from);
              }
            }
          }
          __syncwarp();
        }
      }
      const int k1 = part_end<F32>(k0, kb);
      k0 = k1 < kb ? k1 : 0;
      if (k0 == 0) t += pairs;
    }
    if (lane == 0) tma_store_wait_all();
  }
  __syncwarp();
  cluster_sync();
  if (warp == 2) tmem_dealloc_pair(tbase, 512);
}

template <bool F32>
cudaError_t launch(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales, void *out,
                   int rows, int n, int k, int *status, cudaStream_t st) {
  constexpr int kSize = F32 ? 4 : 2;
  const int kb = blocks_of(k), tiles_n = (n + kTn - 1) / kTn;
  const long long tiles = (((long long)rows + kTm - 1) / kTm) * tiles_n;
  const uint64_t kp = (uint64_t)kb * kBlock;
  const bool tma_out = (long long)n * kSize % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  CUtensorMap ma, mb, mo;
  if (!make_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, rows, kp, kp, kBlock, kBlock, true) ||
      !make_map_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, b_codes, n, kp, kp, kTn / 2, kBlock, true))
    return cudaErrorInvalidValue;
  mo = ma;
  if (tma_out && !make_map_2d(&mo, F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, rows,
                              n, (uint64_t)n * kSize, 32, 128 / kSize, true))
    return cudaErrorInvalidValue;
  auto kern = matmul_kernel<F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(152, 2 * tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ProfScope ps("q8_matmul", st);
  e = cudaLaunchKernelEx(&cfg, kern, ma, mb, mo, static_cast<const uint8_t *>(a_scales),
                         static_cast<const uint8_t *>(b_scales), out, rows, n, kb, scale_pitch(k), tiles_n, (int)tiles,
                         tma_out ? 1 : 0, status);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lg
}  // namespace

cudaError_t matmul(const void *a_codes, const void *a_scales, const void *b_codes, const void *b_scales, void *out,
                   bool f32, int rows, int n, int k, int *status, cudaStream_t st) {
  // Few rows go to the split kernel, with 128 of them 8.6 us for 1024 x 4096
  // against 13.3 with whole tiles.  Where k is short there is little to split, and
  // what the split kernel does for each row counts, whatever n: for k = 512 and n
  // from 128 to 4096, 65 rows 6.1-6.5 us against 5.2-5.7 with whole tiles, 128 rows
  // 7.9-8.2 against 5.3-5.9; for k = 1024 6.2-6.5 against 6.4-6.9 and 7.4-8.0
  // against 6.6-7.1; for k = 1536 6.4-6.8 against 7.4-8.0 and 7.7-8.3 against
  // 7.6-8.1.  512 rows x 4096 x 1024 took 12.2 against 7.3 when the split kernel
  // took more rows.
  if (rows > kBlock || (rows > kBlock / 2 && k <= 1024))
    return f32 ? lg::launch<true>(a_codes, a_scales, b_codes, b_scales, out, rows, n, k, status, st)
               : lg::launch<false>(a_codes, a_scales, b_codes, b_scales, out, rows, n, k, status, st);
  return f32 ? sm::launch<true>(a_codes, a_scales, b_codes, b_scales, out, rows, n, k, status, st)
             : sm::launch<false>(a_codes, a_scales, b_codes, b_scales, out, rows, n, k, status, st);
}

}  // namespace q8
}  // namespace slim
