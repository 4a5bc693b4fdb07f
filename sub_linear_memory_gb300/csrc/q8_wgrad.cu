// q8_wgrad.cu -- weight gradient from the 8-bit checkpoint of a product's
// input: dw [n][k] (+)= sum over rows of dy[row][n] x[row][k].
//
// The sum runs over rows, across which the scales of x differ, so the tensor
// cores cannot apply them; but code * 2^e is exactly a bf16 number, and dy is
// bf16.  Eight warps turn each tile of codes into bf16 in shared memory (shifts,
// masks and a packed multiply) while the tensor cores (kind::f16, both operands
// MN-major) work on the tiles before.
//
// Tile: a CTA pair (cta_group::2) forms 256 (n) x 256 (k), each CTA loading
// 128 columns of dy and converting one 128-column block of x, so that a code
// is converted once for 256 results.  With one CTA for 128 x 256, 65536 rows x
// 1024 x 4096 took 1098 us, four times the MMAs' time.
//
// Rounding: the tensor cores add into their fp32 accumulator with truncation;
// over the 4096 additions of 65536 rows that lost 4e-5 of the result.  The
// accumulator is therefore emptied every 20 steps (80 additions) into
// registers of the eight warps, which add with rounding to nearest, while the
// MMAs go on in a second accumulator.
//
// Split: the rows are cut into steps of 64.  While there are as many tiles as
// pairs, a pair takes a whole tile.  The remaining tiles, fewer than the pairs,
// are cut along the rows: each into equal parts, one for a pair, and what the
// left-over pairs can take from the end of every tile.  All pairs then have
// the same number of steps, and those on different tiles pass over the same
// rows at the same time, so that dy and x come from DRAM once and for the rest
// from L2 (one even cut of the line of all steps put them at different rows: by
// count 3.2 GB of reads, and 612 us against 534).  Parts of a tile go to the workspace as partial tiles, which a
// second kernel adds in a fixed order.
//
// Bound: 377 us for 65536 x 1024 x 4096, 1.46 PFLOP/s, 77% of the measured bf16
// rate.  A step's MMAs take 512 cycles; the conversion of its codes, on the
// integer pipe and in the shared memory that the MMAs read, holds it to 730.
// Rows of dy that do not start on 16 bytes are loaded element by element by the
// converting warps, which then bound it: 65536 x 1001 x 1024 957 us, against 99
// with 1024 columns.
#include <algorithm>

#include "kernels.h"
#include "q8.h"
#include "q8_tc.cuh"
#include "tma_host.h"

namespace slim {
namespace q8 {
namespace {

constexpr int kPairs = 76;      // one CTA for each of 152 SMs
constexpr int kTn = 256, kTk = 256, kStep = 64;  // a pair's tile and rows of a step
constexpr int kMinSteps = 4;    // per pair: about what writing and joining a partial tile costs
constexpr int kSegSteps = 8;    // a part's own cost, in steps (381 us with 16, 377 with 8, 381 with 24)
constexpr int kWindow = 20;     // steps in one accumulator
constexpr int kThreads = 384;   // codes, MMA, dy, scales; eight warps that convert and add
// Two rings: dy with the converted tiles (freed together by the MMAs), and the
// codes (freed by the converting warps).
constexpr int kBufs = 5, kCodes = 6;
constexpr uint32_t kDBytes = kStep * kBlock * 2, kCBytes = kStep * kBlock, kBBytes = kStep * kBlock * 2;
constexpr uint32_t kTable = kStep * 4;  // scale words of a step's rows
constexpr uint32_t oB = kBufs * kDBytes, oCodes = oB + kBufs * kBBytes, oTable = oCodes + kCodes * kCBytes,
                   oBar = oTable + kCodes * kTable;
enum {
  S_DY = 0, S_BFULL = S_DY + kBufs, S_FREE = S_BFULL + kBufs, S_CODES = S_FREE + kBufs,
  S_CODESFREE = S_CODES + kCodes, S_ACC = S_CODESFREE + kCodes, S_ACCFREE = S_ACC + 2, S_DONE = S_ACCFREE + 2, S_COUNT
};
constexpr uint32_t kSmem = 1024 + oBar + 512;

// One pair's part of a tile: steps [s0, s1), and the workspace slot of its
// partial tile (-1: the whole tile, straight into dw).
struct Seg {
  int tile, s0, s1, slot;
};

struct Cut {
  int steps;          // of a tile
  int tiles_k;        // tiles along k
  int pairs, waves;   // tiles [0, waves * pairs) are taken whole
  int rest;           // tiles after those, each cut into `parts` of `part` steps
  int parts, part;
  int tail, extras;   // and `tail` last steps, shared out over the `extras` left-over pairs

  __host__ __device__ long long tail_begin(int e) const { return (long long)rest * tail * e / extras; }
  // The left-over pair that holds step u of the tails: the last e whose
  // tail_begin(e) = floor(rest tail e / extras) is not past u.
  __host__ __device__ int tail_owner(long long u) const {
    return (int)(((u + 1) * extras - 1) / ((long long)rest * tail));
  }
  // Segment `i` of a pair; false past its last.
  __host__ __device__ bool get(int pair, int i, Seg &s) const {
    if (i < waves) {
      s = Seg{i * pairs + pair, 0, steps, -1};
      return true;
    }
    i -= waves;
    if (pair < parts * rest) {
      const int t = pair % rest, j = pair / rest, s0 = j * part, s1 = s0 + part < steps ? s0 + part : steps;
      s = Seg{waves * pairs + t, s0, s1, t * parts + j};
      return i == 0 && s0 < s1;
    }
    if (tail == 0) return false;
    const int e = pair - parts * rest;
    const long long lo = tail_begin(e), hi = tail_begin(e + 1), t = lo / tail + i, t0 = t * tail;
    const long long a = lo > t0 ? lo : t0, b = hi < t0 + tail ? hi : t0 + tail;
    s = Seg{waves * pairs + (int)t, parts * part + (int)(a - t0), parts * part + (int)(b - t0),
            parts * rest + (int)t + e};
    return a < b;
  }
};

Cut cut_of(int rows, int n, int k) {
  Cut c;
  c.steps = rows / kStep + (rows % kStep != 0);
  c.tiles_k = k / kTk + (k % kTk != 0);
  const long long tiles = (long long)c.tiles_k * (n / kTn + (n % kTn != 0));
  c.pairs = (int)std::min<long long>(kPairs, std::max(tiles, tiles * c.steps / kMinSteps));
  c.waves = (int)(tiles / c.pairs);
  c.rest = (int)(tiles % c.pairs);
  c.parts = c.part = c.tail = c.extras = 0;
  if (c.rest) {
    c.parts = c.pairs / c.rest;
    c.extras = c.pairs - c.parts * c.rest;
    // a left-over pair has parts of several tiles, each of which costs it
    // kSegSteps steps' time to empty and write
    c.part = c.extras ? (int)std::min<long long>(c.steps, ((long long)c.rest * (c.steps + kSegSteps) + c.pairs - 1) / c.pairs)
                      : (c.steps + c.parts - 1) / c.parts;
    c.tail = c.extras ? std::max(0, c.steps - c.parts * c.part) : 0;
  }
  return c;
}

// Partial tiles: one for each part, and of the tail one more than there are
// cuts between its tiles and between the pairs that share it.
int slots_of(const Cut &c) { return c.rest ? c.parts * c.rest + (c.tail ? c.rest + c.extras : 0) : 0; }

// A pair's steps in order.
struct Walk {
  const Cut &cut;
  int pair, rank, i = 0;
  Seg seg{0, 0, 0, -1};
  bool more;
  int step = 0, n0 = 0, blk = 0;  // this CTA's first n and block of k in the tile
  __device__ Walk(const Cut &c, int p, int r) : cut(c), pair(p), rank(r) { enter(); }
  __device__ void enter() {
    more = cut.get(pair, i, seg);
    step = seg.s0;
    n0 = seg.tile / cut.tiles_k * kTn + rank * kBlock;
    blk = seg.tile % cut.tiles_k * 2 + rank;
  }
  __device__ void next() {
    if (++step < seg.s1) return;
    ++i;
    enter();
  }
};

// Four e4m3 codes c0..c3 as bf16 bits, (c0, c2) and (c1, c3): sign, and the
// seven other bits at the bottom of the exponent and the top of the fraction,
// i.e. the value times 2^-120 (the exponent biases are 7 and 127; subnormal
// codes become subnormal bf16 numbers).  Taking alternate codes needs no byte
// permutation (a NaN code, which stands in NaN blocks only, becomes 480: the
// block's factor is NaN), and the left shifts are multiplications, so that the integer
// pipe, which bounds the conversion, has five operations for four codes (with
// a permutation for each pair it had eight, and a step took 1030 cycles).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &even, uint32_t &odd) {
  even = ((w * 16u) & 0x07f007f0u) | ((w * 256u) & 0x80008000u);
  odd = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
}
// The columns of a converted tile are therefore x's in the order 0 2 1 3 of
// each four; the accumulator's columns 4 q + 1 and 4 q + 2 change places when
// the result is written.

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 2^(120 + e) as a pair of equal bf16 numbers for a scale byte, in two factors
// where it is past the type's range (e > 7); NaN for a NaN block.
__device__ __forceinline__ uint32_t factor(int byte, uint32_t &second) {
  second = 0;  // none
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

__device__ __forceinline__ void ld_shared_v2(uint32_t addr, uint32_t &a, uint32_t &b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}

// Asynchronous copies of 4 bytes, tracked by an mbarrier: each lane's arrival
// (part of the barrier's count) comes when its copies have landed.
__device__ __forceinline__ void copy_async4(uint32_t to, const uint8_t *from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <bool TMA_DY>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap mdy, const __grid_constant__ CUtensorMap mx,
                 const __nv_bfloat16 *dy, const uint8_t *scales, float *dw, float *partial, Cut cut, int accumulate,
                 int rows, int n, int k, int pitch, int wide, int *status) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t sbase = (smem_u32(raw) + 1023u) & ~1023u;
  uint8_t *smem = raw + (sbase - smem_u32(raw));
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + oBar);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + S_COUNT);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = (int)blockIdx.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < kCodes; ++s) {
      mbar_init(bar + S_CODES + s, 1 + 32);  // the load and the scales' lanes
      mbar_init(bar + S_CODESFREE + s, 2);  // two converting warps
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(bar + S_DY + b, 1);
      mbar_init(bar + S_BFULL + b, 4);  // two converting warps of each CTA
      mbar_init(bar + S_FREE + b, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar + S_ACC + b, 1);
      mbar_init(bar + S_ACCFREE + b, 16);  // the eight warps of both CTAs
    }
    mbar_init(bar + S_DONE, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (TMA_DY) prefetch_tmap(&mdy);
    prefetch_tmap(&mx);
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
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + b);
  };
  auto arrive_leader = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(map_peer(smem_u32(bar + b), 0));
  };
  // Registers of the launch: 384 x 168.  The warpgroups' shares (64 + 2 x 216,
  // times 128) come to 63488 of these 64512.
  if (warp < 4) {
    regs_dec<64>();
    if (warp == 0 && lane == 0) {
      int i = 0;
      for (Walk p(cut, pair, rank); p.more; p.next(), ++i) {
        const int s = i % kCodes;
        if (i >= kCodes && !wait(S_CODESFREE + s, (uint32_t)(i / kCodes - 1) & 1)) break;
        mbar_arrive_expect_tx(bar + S_CODES + s, kCBytes);
        tma_load_2d(sbase + oCodes + s * kCBytes, &mx, bar + S_CODES + s, p.blk * kBlock, p.step * kStep);
      }
      for (int j = max(0, i - kCodes); j < i; ++j) mbar_drain(bar + S_CODES + j % kCodes, (uint32_t)(j / kCodes) & 1);
    } else if (warp == 2 && lane == 0 && TMA_DY) {
      int i = 0;
      for (Walk p(cut, pair, rank); p.more; p.next(), ++i) {
        const int s = i % kBufs;
        if (i >= kBufs && !wait(S_FREE + s, (uint32_t)(i / kBufs - 1) & 1)) break;
        if (rank == 0) mbar_arrive_expect_tx(bar + S_DY + s, 2 * kDBytes);
        const uint32_t full = map_peer(smem_u32(bar + S_DY + s), 0), at = sbase + s * kDBytes;
        tma_load_2d_pair(at, &mdy, full, p.n0, p.step * kStep);
        tma_load_2d_pair(at + kDBytes / 2, &mdy, full, p.n0 + 64, p.step * kStep);
      }
      if (rank == 0)
        for (int j = max(0, i - kBufs); j < i; ++j) mbar_drain(bar + S_DY + j % kBufs, (uint32_t)(j / kBufs) & 1);
    } else if (warp == 1 && rank == 0) {
      const bool issues = elect_lane();
      const uint32_t id = make_idesc(kTn, kTk, true, true);
      int i = 0, win = 0;
      Seg seg;
      for (int x = 0; ok && cut.get(pair, x, seg); ++x) {
        for (int first = seg.s0; first < seg.s1 && ok; first += kWindow, ++win) {
          if (win >= 2 && !wait_warp(S_ACCFREE + (win & 1), (uint32_t)((win >> 1) - 1) & 1)) break;
          tc_fence_after();
          const uint32_t acc = tbase + (win & 1) * kTk;
          const int end = min(first + kWindow, seg.s1);
          for (int step = first; step < end; ++step, ++i) {
            const int b = i % kBufs;
            if (TMA_DY && !wait_warp(S_DY + b, (uint32_t)(i / kBufs) & 1)) break;
            if (!wait_warp(S_BFULL + b, (uint32_t)(i / kBufs) & 1)) break;
            tc_fence_after();
            const uint64_t da = desc_mnmajor(sbase + b * kDBytes, kStep, 0, 0);
            const uint64_t db = desc_mnmajor(sbase + oB + b * kBBytes, kStep, 0, 0);
#pragma unroll
            for (int j = 0; j < kStep / 16; ++j)
              if (issues)
                mma_bf16_pair(acc, da + (uint64_t)(j * 128), db + (uint64_t)(j * 128), id, step > first || j > 0);
            if (issues) mma_commit_pair(bar + S_FREE + b);
            __syncwarp();
          }
          if (ok && issues) mma_commit_pair(bar + S_ACC + (win & 1));
          __syncwarp();
        }
      }
      if (issues) mma_commit_pair(bar + S_DONE);
      __syncwarp();
      mbar_drain(bar + S_DONE, 0);
    } else if (warp == 3) {
      // The scale words of each step's rows, two rows a lane, copied without
      // passing through registers: the copies' own arrivals complete the
      // barrier, so this warp is as far ahead as the codes.  (Loading the bytes
      // four steps ahead into registers held a step to 930 cycles.)
      int i = 0;
      for (Walk p(cut, pair, rank); p.more && ok; p.next(), ++i) {
        const int s = i % kCodes;
        if (i >= kCodes && !wait_warp(S_CODESFREE + s, (uint32_t)(i / kCodes - 1) & 1)) break;
        const uint32_t to = sbase + oTable + s * kTable;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = p.step * kStep + lane + 32 * h;
          if (r < rows && p.blk * kBlock < k)
            copy_async4(to + (lane + 32 * h) * 4, scales + (size_t)r * pitch + (p.blk & ~3));
        }
        copy_async_arrive(bar + S_CODES + s);
      }
      copy_async_wait();
    }
  } else {
    regs_inc<216>();
    // Two warps convert a step, the next two the next: what a step costs besides
    // its arithmetic (waits, the proxy fence, arrivals) overlaps.  The same
    // warps empty the accumulators, since adding takes them 3% of the time; with
    // four warps for one and eight for the other a step took 990 cycles.
    // Converting, a thread has 16 codes of rows row0 + 8 j.
    const int mate = (warp >> 1) & 3, chunk = lane & 7, row0 = 4 * (warp & 1) + (lane >> 3);
    // A thread's two 8-byte loads and two 16-byte stores of a row, in an order
    // that keeps the lanes served together on distinct banks: half of them
    // begin with the second half.
    const bool swap = ((chunk >> 2) ^ (lane >> 3)) & 1;
    // Adding, it has a row of the tile (a TMEM lane), and 128 of its 256 columns.
    const uint32_t lanes = 32u * (warp & 3);
    const int c0 = warp < 8 ? 0 : 128, nr = rank * kBlock + (int)lanes + lane;
    int i = 0, win = 0;
    Seg seg;
    for (int x = 0; ok && cut.get(pair, x, seg); ++x) {
      const bool whole = seg.slot < 0;
      const int n0 = seg.tile / cut.tiles_k * kTn, blk = seg.tile % cut.tiles_k * 2 + rank;
      float sum[128];
#pragma unroll
      for (int e = 0; e < 128; ++e) sum[e] = 0.f;
      // the next accumulator that is done, into the sums
      auto take = [&] {
        wait_warp(S_ACC + (win & 1), (uint32_t)(win >> 1) & 1);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          float v[32];
          tmem_ld32(tmem_addr(tbase, lanes, (win & 1) * kTk + c0 + c), v);
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[c + e] += v[e];
        }
        tc_fence_before();
        arrive_leader(S_ACCFREE + (win & 1));
        ++win;
      };
      int done = seg.s0 + kWindow;  // the end of the next accumulator to add
      for (int step = seg.s0; step < seg.s1 && ok; ++step, ++i) {
        // kBufs steps on, a step's buffer is free only when the first step of the
        // accumulator after it has been multiplied: no waiting here
        if (step == done + kBufs) {
          take();
          done += kWindow;
        }
        if ((i & 3) != mate) continue;
        const int s = i % kCodes, b = i % kBufs, r0 = step * kStep;
        if (i >= kBufs && !wait_warp(S_FREE + b, (uint32_t)(i / kBufs - 1) & 1)) break;
        if (!TMA_DY) {  // rows that TMA cannot step over: loaded here into the same layout
          const int nn = n0 + rank * kBlock;
          for (int y = 32 * (warp & 1) + lane; y < kStep * kBlock; y += 64) {
            const int r = y / kBlock, c = y % kBlock;
            const __nv_bfloat16 v =
                r0 + r < rows && nn + c < n ? dy[(size_t)(r0 + r) * n + nn + c] : __float2bfloat16_rn(0.f);
            *reinterpret_cast<__nv_bfloat16 *>(smem + b * kDBytes + sw128_offset(r, c, kStep)) = v;
          }
        }
        if (!wait_warp(S_CODES + s, (uint32_t)(i / kCodes) & 1)) break;
        const uint32_t from = sbase + oCodes + s * kCBytes + chunk * 16, to = sbase + oB + b * kBBytes;
        // Everything that waits for memory or for other lanes comes before the
        // arithmetic: between the stores, which keep their order, each shuffle
        // and load would wait for its turn.
        uint32_t w[kStep / 8][4], f[kStep / 8];
#pragma unroll
        for (int j = 0; j < kStep / 8; ++j) {
          const uint32_t at = from + (row0 + 8 * j) * kBlock;
          ld_shared_v2(at ^ (swap ? 8u : 0u), w[j][0], w[j][1]);
          ld_shared_v2(at ^ (swap ? 0u : 8u), w[j][2], w[j][3]);
        }
        // factor of one row a lane (row 4 (warp & 1) + lane % 4 + 8 (lane / 4))
        const int mine = 4 * (warp & 1) + (lane & 3) + 8 * (lane >> 2);
        int byte = 127;
        if (r0 + mine < rows && blk * kBlock < k) byte = smem[oTable + s * kTable + mine * 4 + (blk & 3)];
        uint32_t second;
        const uint32_t first = factor(byte, second);
        const bool twice = __any_sync(0xffffffffu, second != 0);
        if (second == 0) second = 0x3f803f80u;  // one, for the rows that need none
        arrive(S_CODESFREE + s);                // all of the step's codes and scales are in registers
#pragma unroll
        for (int j = 0; j < kStep / 8; ++j) f[j] = __shfl_sync(0xffffffffu, first, 4 * j + (lane >> 3));
#pragma unroll
        for (int j = 0; j < kStep / 8; ++j) {
          const int r = row0 + 8 * j;
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            widen4(w[j][e], o[2 * e], o[2 * e + 1]);
            o[2 * e] = mul_bf16x2(o[2 * e], f[j]);
            o[2 * e + 1] = mul_bf16x2(o[2 * e + 1], f[j]);
          }
          if (twice) {
            const uint32_t g = __shfl_sync(0xffffffffu, second, 4 * j + (lane >> 3));
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = mul_bf16x2(o[e], g);
          }
          const uint32_t at = (to + sw128_offset(r, 16 * chunk, kStep)) ^ (swap ? 16u : 0u);
          st_shared_v4(at, o[0], o[1], o[2], o[3]);
          st_shared_v4(at ^ 16u, o[4], o[5], o[6], o[7]);
        }
        fence_async_smem();
        arrive_leader(S_BFULL + b);
      }
      for (; ok && done - kWindow < seg.s1; done += kWindow) take();
      if (!ok) break;
#pragma unroll
      for (int e = 0; e < 128; e += 4) {  // the columns' own order
        const float u = sum[e + 1];
        sum[e + 1] = sum[e + 2];
        sum[e + 2] = u;
      }
      if (!whole) {
        // a partial tile is [64 groups of 4 columns][256 rows][4]: a warp's
        // stores are whole lines
        float4 *to = reinterpret_cast<float4 *>(partial + (size_t)seg.slot * (kTn * kTk)) + c0 / 4 * kTn + nr;
#pragma unroll
        for (int e = 0; e < 128; e += 4) to[e / 4 * kTn] = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        continue;
      }
      const int kk = seg.tile % cut.tiles_k * kTk + c0, left = n0 + nr < n ? k - kk : 0;
      float *to = dw + (size_t)(n0 + nr) * k + kk;
      if (wide) {
#pragma unroll
        for (int e = 0; e < 128; e += 4) {
          if (e < left) {
            float4 *p = reinterpret_cast<float4 *>(to + e);
            float4 v = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
            if (accumulate) {
              const float4 o = *p;
              v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
            }
            *p = v;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e < left) to[e] = accumulate ? to[e] + sum[e] : sum[e];
      }
    }
  }
  __syncwarp();
  cluster_sync();
  if (warp == 2) tmem_dealloc_pair(tbase, 512);
}

// dw of the tiles that are cut along the rows: 32 rows x 32 columns a CTA, read
// as the partial tiles lie (four columns a thread, a warp along the rows) and
// turned in shared memory, so that loads and stores are whole lines.
__global__ void __launch_bounds__(256) wgrad_join_kernel(const float *partial, float *dw, Cut cut, int accumulate, int n,
                                                         int k) {
  __shared__ float turned[32][36];
  const int t = blockIdx.x, tile = cut.waves * cut.pairs + t;
  const int r0 = (int)blockIdx.y % 8 * 32, q0 = (int)blockIdx.y / 8 * 8;  // first row, first group of four columns
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const float4 *from = reinterpret_cast<const float4 *>(partial) + (size_t)(q0 + q) * kTn + r0 + lane;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int slot) {
    const float4 x = from[(size_t)slot * (kTn * kTk / 4)];
    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
  };
  const int parts = min(cut.parts, (cut.steps + cut.part - 1) / cut.part);
#pragma unroll 4
  for (int j = 0; j < parts; ++j) add(t * cut.parts + j);
  if (cut.tail) {
    // the left-over pairs that hold steps of this tile's tail (fewer than there
    // are steps, so none of them is empty)
    const long long first = (long long)t * cut.tail;
    const int to = cut.tail_owner(first + cut.tail - 1);
    for (int e = cut.tail_owner(first); e <= to; ++e) add(cut.parts * cut.rest + t + e);
  }
  *reinterpret_cast<float4 *>(&turned[lane][4 * q]) = v;
  __syncthreads();
  const int r = threadIdx.x >> 3, c = threadIdx.x % 8 * 4;
  const int nn = tile / cut.tiles_k * kTn + r0 + r, kk = tile % cut.tiles_k * kTk + 4 * q0 + c;
  if (nn >= n) return;
  float *to = dw + (size_t)nn * k + kk;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (kk + e < k) to[e] = accumulate ? to[e] + turned[r][c + e] : turned[r][c + e];
}

}  // namespace

size_t wgrad_workspace(int rows, int n, int k) {
  if (rows == 0 || n == 0 || k == 0) return 0;
  return (size_t)slots_of(cut_of(rows, n, k)) * kTn * kTk * sizeof(float);
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * cut.pairs);
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
  {
    ProfScope ps("q8_wgrad", st);
    e = cudaLaunchKernelEx(&cfg, kern, mdy, mx, static_cast<const __nv_bfloat16 *>(dy),
                           static_cast<const uint8_t *>(x_scales), dw, static_cast<float *>(workspace), cut,
                           accumulate ? 1 : 0, rows, n, k, scale_pitch(k),
                           k % 4 == 0 && (reinterpret_cast<uintptr_t>(dw) & 15) == 0 ? 1 : 0, status);
    if (e == cudaSuccess) e = cudaGetLastError();
  }
  if (e != cudaSuccess || cut.rest == 0) return e;
  ProfScope ps("q8_wgrad_join", st);
  wgrad_join_kernel<<<dim3((unsigned)cut.rest, kTn * kTk / 1024), 256, 0, st>>>(
      static_cast<const float *>(workspace), dw, cut, accumulate ? 1 : 0, n, k);
  return cudaGetLastError();
}

}  // namespace q8
}  // namespace slim
