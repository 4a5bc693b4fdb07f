// decay_tc.cu -- linear attention with a decay on the tensor cores: bf16 rows, heads of 64 or
// 128 columns.
//
// A block (one an SM) goes through its share of the tiles (decay.h), 128 rows
// at a time, for one operator  out_i = sum lambda^(i-j) (a_i . b_j) c_j + lambda^(i+1) a_i X.
// For each tile (and each query head of a group: a "unit") four products run
// on tcgen05 with fp32 sums in tensor memory:
//   scores   S = a b^T            128 x 128 x D
//   read     R = a X              128 x D x D     (X: the state as bf16)
//   within   W = (S . decay) c    128 x D x 128   (the weighted scores as bf16, from tensor memory)
//   update   U = b~^T c           D x D x 128     (b~: the rows with their weight to the tile's end)
// and out = read factor * R + within factor * W, state = lambda^n state + U.
// The weights lambda^(i-j) are formed as products of two powers of at most 1,
// so that nothing overflows however strong the decay.
//
// Roundings: out is rounded once; weighted scores and X are bf16 operands,
// each off by 2^-9 of a term in the mean square, like the result itself.  The
// state stays in fp32 registers, and b~ enters as two bf16 numbers (high part
// and remainder, 2^-17), because states are results in fp32 too.
//
// Four roles: one warp loads tiles by TMA into a ring, one issues the MMAs,
// and three warpgroups form the weighted scores, write the results, and keep
// the state.  The bound is memory: 128 rows of four arrays take 2900 cycles of
// this SM's share of HBM at D = 64 (5800 at 128), the products of a unit 1400
// (2700).
#include <cuda.h>

#include "decay_common.cuh"
#include "kernels.h"
#include "q8_tc.cuh"
#include "tma_host.h"

namespace slim {
namespace decay {
namespace {

using namespace tc;
using q8::elect_lane;
using q8::regs_dec;
using q8::regs_inc;

constexpr int kTile = 128, kThreads = 512;

template <int D> struct Cfg {
  static constexpr uint32_t kSlot = kTile * D * 2;     // a tile of one operand
  static constexpr int kSlots = D == 64 ? 8 : 4;
  static constexpr int kBuffers = D == 64 ? 2 : 1;     // of scores, b~, X and updates
  static constexpr uint32_t kWeighted = 2 * kSlot;     // b~: high parts and remainders
  static constexpr uint32_t kState = D * D * 2;
  static constexpr uint32_t kExchange = D == 64 ? 16384 : 0;
  static constexpr uint32_t kBytes = 1024 + kSlots * kSlot + kBuffers * (kWeighted + kState) + kExchange + 512;
  // tensor memory columns
  static constexpr uint32_t tScores = 0, tRead = 128 * kBuffers, tWithin = tRead + D, tUpdate = tWithin + D;
  static_assert(tUpdate + kBuffers * D <= 512, "tensor memory");
};

struct Args {
  CUtensorMap maps[4];
  Work work;
  const float *log_decay;
  int *status;
  int mixes;
  Mix mix[3];
  signed char a[3], b[3], c[3];  // the operands' maps
};

// Zero-based phase counters of a ring or of a barrier.
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ void next(int slots) {
    if (++slot == (uint32_t)slots) slot = 0, phase ^= 1;
  }
};

template <int D> __global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ Args p) {
  using C = Cfg<D>;
  extern __shared__ char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  char *generic = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t slots = base, weighted = slots + C::kSlots * C::kSlot, state = weighted + C::kBuffers * C::kWeighted,
                 exchange = state + C::kBuffers * C::kState;
  uint64_t *bars = reinterpret_cast<uint64_t *>(generic + (exchange - base) + C::kExchange);
  uint64_t *full = bars, *empty = full + C::kSlots, *turned = empty + C::kSlots, *scored = turned + C::kSlots,
           *ready = scored + 2, *done = ready + 2, *taken = done + 1, *added = taken + 1, *whole = added + 2, *known = whole + 2, *drain = known + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
  const int part = blockIdx.x / p.mixes, which = blockIdx.x - part * p.mixes;
  const Mix &m = p.mix[which];
  const Work &w = p.work;
  const bool total = m.totals != nullptr, sums = m.b_heads > 1;
  const int groups = max(m.a_heads, m.b_heads);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 2);   // the MMAs, the rows' warpgroup
      mbar_init(turned + i, 1);  // what the MMAs need of the rows' warpgroup
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(scored + i, 1);
      mbar_init(ready + i, 4);
      mbar_init(added + i, 1);
      mbar_init(whole + i, 1);
      mbar_init(known + i, 1);
    }
    mbar_init(done, 1);
    mbar_init(taken, 4);
    mbar_init(drain, 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  if (warp == 0 && lane < 4) prefetch_tmap(p.maps + lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // A wait that has run out anywhere in the block lets every later one pass
  // at once: the roles go through the rest of their loops, without loads and
  // MMAs, so that none is missed at a barrier of its warpgroup.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    return !*abort && mbar_wait(bar, parity, p.status, abort);
  };

  Walk walk(w, part, m.rev);
  Piece pc;
  if (wg == 0) {
    regs_dec<96>();
    if (warp == 0) {
      // ---- loads: b, a, c of each unit -------------------------------------------
      const CUtensorMap *maps[3] = {p.maps + p.b[which], p.maps + (total ? 0 : p.a[which]), p.maps + p.c[which]};
      const int b_heads = m.b_heads, a_heads = m.a_heads;
      Ring r;
      while (walk.next(w, pc)) {
        if ((total && !piece_has_total(m, pc)) || pc.rows == 0) continue;
        for (int k = 0; k < pc.t1 - pc.t0; ++k) {
          const int row = pc.row0 + (m.rev ? pc.t1 - 1 - k : pc.t0 + k) * kTile;
          for (int g = 0; g < groups; ++g) {
            const int hb = pc.head * b_heads + (b_heads > 1 ? g : 0), ha = pc.head * a_heads + (a_heads > 1 ? g : 0);
#pragma unroll
            for (int o = 0; o < 3; ++o) {
              if (o == 1 && total) continue;
              const bool ok = __all_sync(0xffffffffu, wait(empty + r.slot, r.phase ^ 1));
              if (ok && elect_lane()) {
                mbar_arrive_expect_tx(full + r.slot, C::kSlot);
                for (int x = 0; x < D / 64; ++x)
                  tma_load_3d(generic + r.slot * C::kSlot + x * 16384, maps[o], full + r.slot, x * 64, o == 1 ? ha : hb, row);
              }
              __syncwarp();
              r.next(C::kSlots);
            }
          }
        }
      }
    } else if (warp == 1) {
      // ---- MMAs ------------------------------------------------------------------
      const uint32_t id_scores = make_idesc(128, 128, false, false), id_state = make_idesc(128, D, false, true),
                     id_update = make_idesc(128, D, true, true);
      // The warp runs converged and one lane issues: descriptors are a constant and a slot's offset, in uniform
      // registers.  Formed by the issuing lane alone they took three times as long as the MMAs.
      const bool issues = elect_lane();
      const uint64_t rows_k = desc_kmajor(slots, kTile, 0, 0), rows_mn = desc_mnmajor(slots, kTile, 0, 0),
                     weighted_mn = desc_mnmajor(weighted, kTile, 0, 0), state_mn = desc_mnmajor(state, D, 0, 0);
      constexpr uint32_t kSlotStep = C::kSlot >> 4;
      bool alive = true;
      auto agree = [&](bool ok) { alive = alive && __all_sync(0xffffffffu, ok); };
      // A unit's slots, as the ring gives them: b, a, c (b, c).
      struct Unit {
        uint32_t b, pb, a, pa, c, pc;
      };
      auto unit_at = [&](Ring &t) {
        Unit u{};
        u.b = t.slot, u.pb = t.phase;
        t.next(C::kSlots);
        if (!total) {
          u.a = t.slot, u.pa = t.phase;
          t.next(C::kSlots);
        }
        u.c = t.slot, u.pc = t.phase;
        t.next(C::kSlots);
        return u;
      };
      uint32_t scored_units = 0;
      auto scores = [&](const Unit &u) {
        const uint32_t buffer = scored_units++ % C::kBuffers, d = tmem + C::tScores + buffer * 128;
        if (!alive) return;
        tc_fence_after();
        const uint64_t a = rows_k + u.a * kSlotStep, b = rows_k + u.b * kSlotStep;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t at = (s >> 2) * kTile * 8u + (s & 3) * 2u;
          if (issues) mma_bf16(d, a + at, b + at, id_scores, s > 0);
        }
        if (issues) mma_commit(scored + buffer);
        if (issues) mma_commit(empty + u.b);
        __syncwarp();
      };
      Ring r;  // the first load of the unit behind those whose scores are issued
      Unit now{}, then{};
      bool ahead = false;  // the scores of `then` are issued
      uint32_t unit = 0, outs = 0, tiles = 0, updates = 0;
      while (walk.next(w, pc)) {
        if ((total && !piece_has_total(m, pc)) || pc.rows == 0) continue;
        for (int k = 0; k < pc.t1 - pc.t0; ++k, ++tiles) {
          for (int g = 0; g < groups; ++g, ++unit) {
            const bool last = g == groups - 1, update = sums || last;
            auto read = [&]() {
              if (g == 0) agree(wait(known + tiles % C::kBuffers, (tiles / C::kBuffers) & 1));
              if (total || (g > 0 && sums)) return;
              agree(wait(taken, (outs & 1) ^ 1));
              if (!alive) return;
              tc_fence_after();
              const uint64_t a = rows_k + now.a * kSlotStep, x = state_mn + (tiles % C::kBuffers) * (C::kState >> 4);
#pragma unroll
              for (int s = 0; s < D / 16; ++s) {
                const uint32_t at = (s >> 2) * kTile * 8u + (s & 3) * 2u;
                if (issues) mma_bf16(tmem + C::tRead, a + at, x + s * 128u, id_state, s > 0);
              }
              __syncwarp();
            };
            if (ahead) {
              now = then;
              ahead = false;
            } else {
              now = unit_at(r);
              agree(wait(full + now.b, now.pb));
              if (!total) {
                agree(wait(full + now.a, now.pa));
                scores(now);
              }
            }
            agree(wait(full + now.c, now.pc));
            // the scores of the next unit, if its rows are here: whether there is a next one shows in the barrier
            // alone, which completes no phase without a load
            if (C::kBuffers == 2 && !total) {
              Ring t = r;
              const Unit u = unit_at(t);
              const bool here = mbar_test(full + u.b, u.pb) && mbar_test(full + u.a, u.pa);
              if (__all_sync(0xffffffffu, here) && alive) {
                then = u;
                r = t;
                ahead = true;
                scores(u);
              }
            }
            // with two buffers the update goes first, ahead of the state that this tile reads; with one it would
            // overwrite what the state's warpgroup has yet to take
            if (C::kBuffers == 1) read();
            agree(wait(turned + now.c, now.pc));
            const uint64_t c = rows_mn + now.c * kSlotStep;
            if (update) {
              if (alive) {
                tc_fence_after();
                const bool first = !sums || g == 0;
                const uint32_t d = tmem + C::tUpdate + (tiles % C::kBuffers) * D;
                const uint64_t b = weighted_mn + (updates % C::kBuffers) * (C::kWeighted >> 4);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                  if (issues) mma_bf16(d, b + s * 128u, c + s * 128u, id_update, s > 0 || !first);
                if constexpr (D == 128) {
#pragma unroll
                  for (int s = 0; s < 8; ++s)
                    if (issues) mma_bf16(d, b + kSlotStep + s * 128u, c + s * 128u, id_update, 1);
                }
                if (issues) mma_commit(added + updates % C::kBuffers);
                if (last && issues) mma_commit(whole + tiles % C::kBuffers);
                if (total && issues) mma_commit(empty + now.b);
                if (total && issues) mma_commit(empty + now.c);
                __syncwarp();
              }
              ++updates;
            }
            if (C::kBuffers == 2) read();
            if (!total) {
              const uint32_t buffer = unit % C::kBuffers;
              agree(wait(ready + buffer, (unit / C::kBuffers) & 1));
              if (alive) {
                tc_fence_after();
                const bool first = !sums || g == 0;
#pragma unroll
                for (int s = 0; s < 8; ++s)
                  if (issues)
                    mma_bf16_ta(tmem + C::tWithin, tmem + C::tScores + buffer * 128 + s * 8, c + s * 128u, id_state, s > 0 || !first);
                if (issues) mma_commit(empty + now.a);
                if (issues) mma_commit(empty + now.c);
                if ((last || !sums) && issues) mma_commit(done);
                __syncwarp();
              }
              if (last || !sums) ++outs;
            }
          }
        }
      }
      // what was issued has to end before its tensor memory goes
      if (issues) {
        mma_commit(drain);
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  } else if (wg == 1) {
    // ---- weighted scores: thread t has row t -------------------------------------
    const int t = threadIdx.x - 128, q = t >> 5;
    const uint32_t row_base = tmem_addr(tmem, q * 32, C::tScores);
    uint32_t unit = 0;
    while (walk.next(w, pc)) {
      if (total || pc.rows == 0) continue;
      const float g2 = log2_decay(p.log_decay, pc.head);
      // Powers of lambda: from a column to the block's end that is nearer the rows, and on the diagonal block.
      float2 col[16], diag[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int j0 = 2 * j, j1 = 2 * j + 1;
        col[j] = make_float2(exp2f(g2 * (float)(m.rev ? j0 : 31 - j0)), exp2f(g2 * (float)(m.rev ? j1 : 31 - j1)));
        diag[j] = make_float2(exp2f(g2 * fmaxf(0.f, (float)(m.rev ? j0 - lane : lane - j0))),
                              exp2f(g2 * fmaxf(0.f, (float)(m.rev ? j1 - lane : lane - j1))));
      }
      for (int k = 0; k < pc.t1 - pc.t0; ++k) {
        const int tile = m.rev ? pc.t1 - 1 - k : pc.t0 + k, n = min(kTile, pc.rows - tile * kTile);
        for (int g = 0; g < groups; ++g, ++unit) {
          const uint32_t sb = unit % C::kBuffers, at = row_base + sb * 128;
          wait(scored + sb, (unit / C::kBuffers) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int jb = 0; jb < 4; ++jb) {
            float v[32];
            const bool diagonal = jb == q, live = m.rev ? jb > q : jb < q;
            const int c0 = jb * 32;
            if (diagonal || live) {
              tmem_ld32(at + c0, v);
              if (live) {
                const float away = ex2_ftz(g2 * (float)(m.rev ? c0 - t : t - c0 - 31));
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float2 x = __fmul2_rn(make_float2(v[2 * j], v[2 * j + 1]), __fmul2_rn(col[j], make_float2(away, away)));
                  v[2 * j] = x.x, v[2 * j + 1] = x.y;
                }
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const float d = j & 1 ? diag[j / 2].y : diag[j / 2].x;
                  v[j] = (m.rev ? j >= lane : j <= lane) ? v[j] * d : 0.f;
                }
              }
              if (m.rev && c0 + 32 > n) {
                // chosen, not multiplied with 0: the rows behind the sequence may hold anything
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = c0 + j < n ? v[j] : 0.f;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.f;
            }
            // two numbers to a column: block jb's 16 columns lie where scores of blocks already read were
            float packed[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) packed[j] = __uint_as_float(pack_bf16(v[2 * j], v[2 * j + 1]));
            tmem_st16(at + jb * 16, packed);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + sb);
        }
      }
    }
  } else if (wg == 2) {
    // ---- rows: thread t has row t, of b to weigh it and of the results to write them ----
    regs_dec<80>();
    const int t = threadIdx.x - 256, q = t >> 5;
    const uint32_t row_base = tmem_addr(tmem, q * 32, 0);
    Ring r;
    uint32_t outs = 0, updates = 0;
    // the result that is to be written next
    __nv_bfloat16 *dst = nullptr;
    float read = 0.f;
    bool due = false, mine = false;
    auto write = [&]() {
      if (!due) return;
      due = false;
      wait(done, outs & 1);
      ++outs;
      tc_fence_after();
#pragma unroll 1
      for (int x = 0; x < D; x += 16) {
        float v[16], u[16];
        tmem_ld16x2(row_base + C::tRead + x, row_base + C::tWithin + x, v, u);
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          h[j] = pack_bf16(fmaf(v[2 * j], read, m.within * u[2 * j]), fmaf(v[2 * j + 1], read, m.within * u[2 * j + 1]));
        if (mine) {
          *reinterpret_cast<uint4 *>(dst + x) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4 *>(dst + x + 8) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(taken);
    };
    while (walk.next(w, pc)) {
      if ((total && !piece_has_total(m, pc)) || pc.rows == 0) continue;
      const float g2 = log2_decay(p.log_decay, pc.head);
      for (int k = 0; k < pc.t1 - pc.t0; ++k) {
        const int tile = m.rev ? pc.t1 - 1 - k : pc.t0 + k, n = min(kTile, pc.rows - tile * kTile);
        // rows past n are neither weighed nor written
        const float up = exp2f(g2 * (float)(t + 1)), down = exp2f(g2 * (float)(n - 1 - t)), weight = m.add * (m.rev ? up : down);
        for (int g = 0; g < groups; ++g) {
          uint32_t at[3] = {0, 0, 0}, phase[3] = {0, 0, 0};
#pragma unroll
          for (int o = 0; o < 3; ++o) {
            if (o == 1 && total) continue;
            at[o] = r.slot;
            phase[o] = r.phase;
            r.next(C::kSlots);
          }
          const uint32_t b = slots + at[0] * C::kSlot, c = slots + at[2] * C::kSlot;
          wait(full + at[0], phase[0]);
          if (sums || g == groups - 1) {
            const uint32_t high = weighted + (updates % C::kBuffers) * C::kWeighted, rest = high + C::kSlot;
            if (updates >= C::kBuffers) wait(added + updates % C::kBuffers, (updates / C::kBuffers + 1) & 1);
            ++updates;
#pragma unroll 2
            for (int x = 0; x < D; x += 8) {
              float v[8], lo[8];
              const uint32_t off = sw128_offset(t, x, kTile);
              if (t < n) {
                ld_bf16x8(b + off, v);
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float v0 = v[2 * j] * weight, v1 = v[2 * j + 1] * weight;
                  h[j] = pack_bf16(v0, v1);
                  lo[2 * j] = v0 - __uint_as_float(h[j] << 16);
                  lo[2 * j + 1] = v1 - __uint_as_float(h[j] & 0xffff0000u);
                }
                st_shared_v4(high + off, h[0], h[1], h[2], h[3]);
                st_bf16x8(rest + off, lo);
              } else {
                st_shared_v4(high + off, 0, 0, 0, 0);
                st_shared_v4(rest + off, 0, 0, 0, 0);
              }
            }
          }
          if (!total) wait(full + at[1], phase[1]);
          wait(full + at[2], phase[2]);
          if (t >= n) {
            // rows behind the sequence: 0 times whatever they hold has to be 0
#pragma unroll 1
            for (int x = 0; x < D; x += 8) st_shared_v4(c + sw128_offset(t, x, kTile), 0, 0, 0, 0);
          }
          fence_async_smem();
          named_barrier_sync(2, 128);
          if (t == 0) {
#pragma unroll
            for (int o = 0; o < 3; ++o) {
              if (o == 1 && total) continue;
              mbar_arrive(turned + at[o]);  // every slot's, so that its phases go with the loads'
              mbar_arrive(empty + at[o]);
            }
          }
          // the last unit's result, while the MMAs take what was handed out
          write();
          due = !total && (!sums || g == groups - 1);
          if (due) {
            dst = static_cast<__nv_bfloat16 *>(m.out) + ((long long)pc.row0 + tile * kTile + t) * m.out_row +
                  (long long)(pc.head * m.a_heads + (sums ? 0 : g)) * D;
            read = m.read * (m.rev ? down : up);
            mine = t < n;
          }
        }
      }
    }
    write();
  } else {
    // ---- the state -----------------------------------------------------------------
    // Thread t has row t of it (D = 128), or half of row t % 64: with D = 64
    // the update's rows 0-63 are those of the high parts and 64-127 those of
    // the remainders, so two threads exchange halves and add.
    regs_inc<208>();
    constexpr int kOwn = D == 64 ? 32 : 128;
    const int t = threadIdx.x - 384, q = t >> 5;
    const int srow = D == 64 ? t & 63 : t, scol = D == 64 ? (t >> 6) * 32 : 0;
    const uint32_t row_base = tmem_addr(tmem, q * 32, C::tUpdate);
    constexpr int kBar = 1;
    float s[kOwn];
    uint32_t tiles = 0, summed = 0;  // tiles whose state is published, whose update is in the state
    auto publish = [&]() {  // the state as the operand [x][y]
      const uint32_t buffer = tiles++ % C::kBuffers, x = state + buffer * C::kState;
      if (!total) {
#pragma unroll
        for (int i = 0; i < kOwn; i += 8) st_bf16x8(x + sw128_offset(srow, scol + i, D), s + i);
        fence_async_smem();
      }
      named_barrier_sync(kBar, 128);
      if (t == 0) mbar_arrive(known + buffer);
    };
    // The state takes a tile's update.
    auto take = [&](float keep) {
      wait(whole + summed % C::kBuffers, (summed / C::kBuffers) & 1);
      tc_fence_after();
      const uint32_t from = row_base + (summed % C::kBuffers) * D;
      ++summed;
      if constexpr (D == 64) {
        float u[32], v[32];
        tmem_ld32x2(from, from + 32, u, v);
        const bool low = t >= 64;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float *give = low ? u + 4 * i : v + 4 * i;
          st_shared_v4(exchange + (i * 128 + t) * 16, __float_as_uint(give[0]), __float_as_uint(give[1]),
                       __float_as_uint(give[2]), __float_as_uint(give[3]));
        }
        named_barrier_sync(kBar, 128);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x[4];
          ld_shared_v4f(exchange + (i * 128 + (t ^ 64)) * 16, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[4 * i + j] = fmaf(s[4 * i + j], keep, (low ? v[4 * i + j] : u[4 * i + j]) + x[j]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < D; x += 16) {
          float u[16];
          tmem_ld16(from + x, u);
#pragma unroll
          for (int j = 0; j < 16; ++j) s[x + j] = fmaf(s[x + j], keep, u[j]);
        }
      }
      tc_fence_before();
    };
    while (walk.next(w, pc)) {
      if (total && !piece_has_total(m, pc)) continue;
      const float g2 = log2_decay(p.log_decay, pc.head);
      const float *start = piece_start(w, m, pc, part);
      // in memory [x][y], or transposed: step by step either way from one address
      const int first = m.transposed ? scol * D + srow : srow * D + scol;
      if (!start) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) s[i] = 0.f;
      } else if (m.transposed) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) s[i] = start[first + i * D];
      } else {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) s[i] = start[first + i];
      }
      const int count = pc.rows == 0 ? 0 : pc.t1 - pc.t0;
      for (int k = 0; k < count; ++k) {
        const int tile = m.rev ? pc.t1 - 1 - k : pc.t0 + k, n = min(kTile, pc.rows - tile * kTile);
        publish();
        take(exp2f(g2 * (float)n));
      }
      float *end = piece_end(w, m, pc, part);
      if (end && m.transposed) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) end[first + i * D] = s[i];
      } else if (end) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) end[first + i] = s[i];
      }
    }
  }
  __syncthreads();
  if (*abort && threadIdx.x == 0)  // copies still on their way land before the block leaves
    for (int i = 0; i < C::kSlots; ++i)
      for (uint32_t parity = 0; parity < 2; ++parity) mbar_drain(full + i, parity, 20000000ull);
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D> cudaError_t launch(const Args &a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::kBytes);
  if (e != cudaSuccess) return e;
  tc_kernel<D><<<a.work.parts * a.mixes, kThreads, Cfg<D>::kBytes, st>>>(a);
  return cudaGetLastError();
}

// [tokens][heads][D], rows `row` elements apart; boxes of 128 rows and 64 columns of one head.
bool make_map(CUtensorMap *map, const void *p, int tokens, long long heads, int d, long long row) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)row * 2};
  const cuuint32_t box[3] = {64, 1, kTile};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Heads of 64 or 128 columns whose rows start on 16 bytes, as TMA and 16-byte stores want them.
bool tc_supported(const Launch &l) {
  for (int i = 0; i < l.mixes; ++i) {
    const Mix &m = l.mix[i];
    if (m.x != m.y || (m.x != 64 && m.x != 128)) return false;
    const void *ptrs[4] = {m.a, m.b, m.c, m.out};
    const long long rows[4] = {m.a_row, m.b_row, m.c_row, m.out_row};
    for (int k = 0; k < 4; ++k)
      if ((reinterpret_cast<uintptr_t>(ptrs[k]) & 15) || rows[k] % 8 || rows[k] >= (1ll << 38)) return false;
  }
  return true;
}

cudaError_t mix_tc(const Launch &l, int *status, cudaStream_t st) {
  ProfScope ps(l.mix[0].totals ? "decay_totals" : "decay_mix", st);
  Args a{};
  a.work = l.work;
  a.log_decay = l.log_decay;
  a.status = status;
  a.mixes = l.mixes;
  int used = 0;
  struct { const void *p; int heads; long long row; } seen[4] = {};
  auto map_of = [&](const void *p, int heads, long long row, int d) -> int {
    for (int i = 0; i < used; ++i)
      if (seen[i].p == p && seen[i].heads == heads && seen[i].row == row) return i;
    if (used == 4 || !make_map(a.maps + used, p, l.work.tokens, (long long)heads * l.work.heads, d, row)) return -1;
    seen[used] = {p, heads, row};
    return used++;
  };
  for (int i = 0; i < l.mixes; ++i) {
    const Mix &m = a.mix[i] = l.mix[i];
    a.a[i] = (signed char)(m.totals ? 0 : map_of(m.a, m.a_heads, m.a_row, m.x));
    a.b[i] = (signed char)map_of(m.b, m.b_heads, m.b_row, m.x);
    a.c[i] = (signed char)map_of(m.c, m.b_heads, m.c_row, m.x);
    if (a.a[i] < 0 || a.b[i] < 0 || a.c[i] < 0) return cudaErrorInvalidValue;
  }
  for (int i = used; i < 4; ++i) a.maps[i] = a.maps[0];
  return l.mix[0].x == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace decay
}  // namespace slim
