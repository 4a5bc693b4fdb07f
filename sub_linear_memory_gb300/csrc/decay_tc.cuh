// decay_tc.cuh -- linear attention with a decay on the tensor cores: bf16 rows, heads of 64 or
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
// The weights lambda^(i-j) are products of two powers of at most 1, or come
// from a table of powers, so that nothing overflows however strong the decay.
//
// Roundings: out is rounded once; weighted scores and X are bf16 operands,
// each off by 2^-9 of a term in the mean square, like the result itself.  The
// state stays in fp32 registers, and b~ enters as two bf16 numbers (high part
// and remainder, 2^-17), because states are results in fp32 too.
//
// Roles: one warp loads tiles by TMA into a ring, two issue the MMAs, and
// warpgroups form the weighted scores; weigh b's rows; write the results (at
// D = 64 in a warpgroup of its own); and keep the state.  The floor is memory:
// 128 rows of four arrays take 2900 cycles of this SM's share of HBM at D = 64
// (5800 at 128), the products of a unit 1700 (2700).  Measured over 2^20 rows
// of 8 heads of 64: 2980 cycles a tile, 1600 for the totals, whose two arrays
// take 1450.  At D = 128 a unit takes 7200: tensor memory has room for one
// buffer of scores, and shared memory for five tiles, so that loads, scores,
// weights and products of one unit follow one another.
#pragma once

#include "decay_common.cuh"
#include "decay_tc_args.h"
#include "q8_tc.cuh"

namespace slim {
namespace decay {
namespace {

using namespace tc;
using q8::elect_lane;
using q8::regs_dec;
using q8::regs_inc;

constexpr int kTile = 128;
constexpr uint32_t kGiveUp = 1u << 21;  // tries of a wait, each of which may sleep for a while: a second or more
constexpr int kUnits = 16;  // barriers of units in a row: more than the ring holds

template <int D, bool TOTAL> struct Cfg {
  static constexpr uint32_t kSlot = kTile * D * 2;     // a tile of one operand
  // At D = 64 a warpgroup of its own writes the results; at 128 the state's registers leave none.  Registers of the
  // warpgroups (loads and MMAs, weighted scores, rows, results, state): at most 640 x 96 or 512 x 128 in all.
  static constexpr bool kWriters = D == 64 && !TOTAL;
  static constexpr int kThreads = kWriters ? 640 : 512;
  static constexpr int kRegs0 = kWriters ? 88 : 96, kRegsScores = kWriters ? 112 : 128, kRegsRows = kWriters ? 72 : 80,
                       kRegsState = kWriters ? 120 : 208;
  static constexpr int kSlots = D == 64 ? 9 : 5;
  static constexpr int kBuffers = D == 64 ? 2 : 1;     // of scores, b~, X and updates
  static constexpr uint32_t kRest = kSlot;             // b~: remainders; its high parts take b's place
  static constexpr uint32_t kState = D * D * 2;
  static constexpr uint32_t kExchange = D == 64 ? 16384 : 0;
  static constexpr uint32_t kStage = D == 64 ? kSlot : 0;  // results on their way out; at D = 128 in a's slot
  static constexpr uint32_t kBytes = 1024 + kSlots * kSlot + kBuffers * (kRest + kState) + kExchange + kStage + 1024;
  // tensor memory columns
  static constexpr uint32_t tScores = 0, tRead = 128 * kBuffers, tWithin = tRead + D, tUpdate = tWithin + D;
  static_assert(tUpdate + kBuffers * D <= 512, "tensor memory");
};

// Zero-based phase counters of a ring or of a barrier.
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ void next(int slots) {
    if (++slot == (uint32_t)slots) slot = 0, phase ^= 1;
  }
};

// An MN-major operand's descriptor with another distance between its blocks of 64 columns.
__device__ __forceinline__ uint64_t with_lbo(uint64_t desc, uint32_t bytes) {
  return (desc & ~((uint64_t)0x3FFF << 16)) | (uint64_t)((bytes >> 4) & 0x3FFF) << 16;
}

// TOTAL: the totals of the shares alone.  REV: against time.  GROUPED: more than one query head to a key-value head.
// Compiled apart, because the block's instructions have to fit into the caches (one kernel for all: 1.45 ms, now
// 1.01, for 2^20 rows x 8 heads).
template <int D, bool TOTAL, bool REV, bool GROUPED>
__global__ void __launch_bounds__(Cfg<D, TOTAL>::kThreads, 1) tc_kernel(const __grid_constant__ TcArgs p) {
  using C = Cfg<D, TOTAL>;
  extern __shared__ char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  char *generic = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t slots = base, weighted = slots + C::kSlots * C::kSlot, state = weighted + C::kBuffers * C::kRest,
                 exchange = state + C::kBuffers * C::kState, stage_at = exchange + C::kExchange, bars_at = stage_at + C::kStage;
  uint64_t *bars = reinterpret_cast<uint64_t *>(generic + (bars_at - base));
  uint64_t *full = bars, *turned = full + kUnits, *empty = turned + kUnits, *scored = empty + C::kSlots,
           *ready = scored + 2, *done = ready + 2, *taken = done + 1, *added = taken + 1, *whole = added + 2, *known = whole + 2, *drain = known + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 2);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *powers = reinterpret_cast<float *>(generic + (bars_at - base) + 512);  // lambda^0 .. lambda^127

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
  const int part = blockIdx.x / p.mixes, which = blockIdx.x - part * p.mixes;
  const Mix &m = p.mix[which];
  const Work &w = p.work;
  constexpr bool total = TOTAL, rev = REV, sums = REV && GROUPED;
  const int groups = GROUPED ? max(m.a_heads, m.b_heads) : 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(empty + i, total ? 5 : 6);  // each issuing warp, each warp of the rows' warpgroup
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(full + i, total ? 2 : 3);  // the unit's operands
      mbar_init(turned + i, 1);            // what the MMAs need of the rows' warpgroup
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(scored + i, 1);
      mbar_init(ready + i, 4);
      mbar_init(added + i, 1);
      mbar_init(whole + i, 1);
      mbar_init(known + i, 1);
    }
    mbar_init(done, 2);
    mbar_init(taken, 4);
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
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
    if (*abort) return false;
    // Short, because there are many, and the caches have to hold the instructions of all the roles at once.
#pragma unroll 1
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
      if (i & 255u) continue;
      if (i >= kGiveUp) atomicCAS(p.status, 0, 5), *abort = 1;
      if (*abort) return false;
    }
    return true;
  };

  // A group's heads share b and c, or in reverse a.  These are loaded with the first head and held to the last, where
  // all the tile's loads fit into the ring; slots are taken in turn, so that a load must not wait for one that is held.
  // (Without a stage a's slot is held on, until the next tile's first unit has come.)
  const bool share = !GROUPED || (sums ? 2 * groups + (C::kStage ? 1 : 3) : groups + 2) <= C::kSlots;
  auto loads_bc = [&](int g) { return sums || g == 0 || !share; };
  auto loads_a = [&](int g) { return !total && (!sums || g == 0 || !share); };
  auto ends_bc = [&](int g) { return sums || g == groups - 1 || !share; };
  auto ends_a = [&](int g) { return !sums || g == groups - 1 || !share; };
  // A unit's slots, as the ring gives them.
  struct Unit {
    uint32_t b, a, c;
  };
  auto advance = [&](Unit &u, Ring &r, int g) {
    if (loads_bc(g)) u.b = r.slot, r.next(C::kSlots);
    if (loads_a(g)) u.a = r.slot, r.next(C::kSlots);
    if (loads_bc(g)) u.c = r.slot, r.next(C::kSlots);
  };

  Walk walk(w, part, rev);
  Piece pc;
  if (wg == 0) {
    regs_dec<C::kRegs0>();
    if (warp == 0) {
      // ---- loads: b, a, c of each unit -------------------------------------------
      const CUtensorMap *map_b = p.maps + p.b[which], *map_a = p.maps + (total ? 0 : p.a[which]), *map_c = p.maps + p.c[which];
      const int b_heads = m.b_heads, a_heads = m.a_heads;
      Ring r;
      uint32_t unit = 0;
      while (walk.next(w, pc)) {
        if ((total && !piece_has_total(m, pc)) || pc.rows == 0) continue;
        for (int k = 0; k < pc.t1 - pc.t0; ++k) {
          const int row = pc.row0 + (rev ? pc.t1 - 1 - k : pc.t0 + k) * kTile;
          for (int g = 0; g < groups; ++g, ++unit) {
            uint64_t *bar = full + unit % kUnits;
            const int hb = pc.head * b_heads + (b_heads > 1 ? g : 0), ha = pc.head * a_heads + (a_heads > 1 ? g : 0);
            const bool bc = loads_bc(g), na = loads_a(g);
            if (!total && !(bc && na) && elect_lane()) mbar_arrive_n(bar, na ? 2 : 1);
#pragma unroll 1
            for (int o = 0; o < 3; ++o) {
              if (o == 1 ? !na : !bc) continue;
              const bool ok = __all_sync(0xffffffffu, wait(empty + r.slot, r.phase ^ 1));
              if (ok && elect_lane()) {
                const CUtensorMap *map = o == 0 ? map_b : o == 1 ? map_a : map_c;
                mbar_arrive_expect_tx(bar, C::kSlot);
                for (int x = 0; x < D / 64; ++x)
                  tma_load_3d(generic + r.slot * C::kSlot + x * 16384, map, bar, x * 64, o == 1 ? ha : hb, row);
              }
              __syncwarp();
              r.next(C::kSlots);
            }
          }
        }
      }
    } else if (warp < 3) {
      // ---- MMAs: warp 1 issues scores and products of weighted scores, warp 2 updates and reads ----
      // Two warps, because an MMA holds up its issuing thread while it runs, and each of the waits between
      // them costs some fifty cycles more (one warp for all: 4400 cycles a unit at D = 64, 3000 of them busy).
      // A warp runs converged and one lane issues: descriptors are a constant and a slot's offset, in uniform
      // registers.  Formed by the issuing lane alone they took three times as long as the MMAs.
      const bool issues = elect_lane();
      const uint64_t rows_k = desc_kmajor(slots, kTile, 0, 0), rows_mn = desc_mnmajor(slots, kTile, 0, 0),
                     rest_mn = desc_mnmajor(weighted, kTile, 0, 0), state_mn = desc_mnmajor(state, D, 0, 0);
      constexpr uint32_t kSlotStep = C::kSlot >> 4;
      const uint32_t id_scores = make_idesc(128, 128, false, false), id_state = make_idesc(128, D, false, true),
                     id_update = make_idesc(128, D, true, true);
      bool alive = true;
      auto agree = [&](bool ok) { alive = alive && __all_sync(0xffffffffu, ok); };
      Ring r;
      uint32_t unit = 0, outs = 0, tiles = 0, updates = 0;
      if (warp == 1 && !total) {
        uint32_t scored_units = 0;
        auto scores = [&](const Unit &u, bool release) {
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
          if (release && issues) mma_commit(empty + u.b);
          __syncwarp();
        };
        Unit now{}, then{};
        bool ahead = false;  // the scores of `then` are issued; r is behind it
        while (walk.next(w, pc)) {
          if (pc.rows == 0) continue;
          for (int k = 0; k < pc.t1 - pc.t0; ++k) {
            for (int g = 0; g < groups; ++g, ++unit) {
              const bool last = g == groups - 1;
              if (ahead) {
                now = then;
                ahead = false;
              } else {
                advance(now, r, g);
                agree(wait(full + unit % kUnits, (unit / kUnits) & 1));
                scores(now, ends_bc(g));
              }
              // The scores of the next unit, as soon as its rows are here and until this one's are weighed: whether
              // there is a next one shows in the barrier alone, which completes no phase without loads.
              const uint32_t buffer = unit % C::kBuffers;
              if (C::kBuffers == 2) {
                const uint32_t then_unit = unit + 1;
#pragma unroll 1
                for (int i = 0; i < 4096 && alive; ++i) {
                  if (__all_sync(0xffffffffu, mbar_test(full + then_unit % kUnits, (then_unit / kUnits) & 1))) {
                    then = now;
                    advance(then, r, last ? 0 : g + 1);
                    ahead = true;
                    scores(then, ends_bc(last ? 0 : g + 1));
                    break;
                  }
                  if (__all_sync(0xffffffffu, mbar_test(ready + buffer, (unit / C::kBuffers) & 1))) break;
                }
              }
              agree(wait(turned + unit % kUnits, (unit / kUnits) & 1));
              agree(wait(ready + buffer, (unit / C::kBuffers) & 1));
              if (g == 0 || !sums) agree(wait(taken, (outs & 1) ^ 1));
              if (alive) {
                tc_fence_after();
                const uint64_t c = rows_mn + now.c * kSlotStep;
                const bool first = !sums || g == 0;
#pragma unroll
                for (int s = 0; s < 8; ++s)
                  if (issues)
                    mma_bf16_ta(tmem + C::tWithin, tmem + C::tScores + buffer * 128 + s * 8, c + s * 128u, id_state, s > 0 || !first);
                if (ends_a(g) && issues) mma_commit(empty + now.a);
                if (ends_bc(g) && issues) mma_commit(empty + now.c);
                if ((last || !sums) && issues) mma_commit(done);
                __syncwarp();
              }
              if (last || !sums) ++outs;
            }
          }
        }
      } else if (warp == 2) {
        Unit now{};
        while (walk.next(w, pc)) {
          if ((total && !piece_has_total(m, pc)) || pc.rows == 0) continue;
          for (int k = 0; k < pc.t1 - pc.t0; ++k, ++tiles) {
            for (int g = 0; g < groups; ++g, ++unit) {
              const bool last = g == groups - 1, update = sums || last;
              advance(now, r, g);
              uint64_t *bar = full + unit % kUnits;
              const uint32_t phase = (unit / kUnits) & 1;
              auto read = [&]() {
                if (g == 0) agree(wait(known + tiles % C::kBuffers, (tiles / C::kBuffers) & 1));
                if (total) return;
                if (g == 0 || !sums) {
                  agree(wait(bar, phase));
                  agree(wait(taken, (outs & 1) ^ 1));
                  ++outs;
                  if (alive) {
                    tc_fence_after();
                    const uint64_t a = rows_k + now.a * kSlotStep, x = state_mn + (tiles % C::kBuffers) * (C::kState >> 4);
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                      const uint32_t at = (s >> 2) * kTile * 8u + (s & 3) * 2u;
                      if (issues) mma_bf16(tmem + C::tRead, a + at, x + s * 128u, id_state, s > 0);
                    }
                    if (issues) mma_commit(done);
                  }
                }
                if (ends_a(g) && alive && issues) mma_commit(empty + now.a);
                __syncwarp();
              };
              // with two buffers the update goes first, ahead of the state that this tile reads; with one it would
              // overwrite what the state's warpgroup has yet to take
              if (C::kBuffers == 1) read();
              agree(wait(bar, phase));
              agree(wait(turned + unit % kUnits, phase));
              if (alive) {
                tc_fence_after();
                if (update) {
                  const bool first = !sums || g == 0;
                  const uint32_t d = tmem + C::tUpdate + (tiles % C::kBuffers) * D;
                  const uint64_t c = rows_mn + now.c * kSlotStep, rest = rest_mn + (updates % C::kBuffers) * (C::kRest >> 4),
                                 high = rows_mn + now.b * kSlotStep;
                  // At D = 64 high parts and remainders are one operand of 128 columns, so that one MMA takes both:
                  // its columns 64 to 127 lie as far behind the first as the remainders behind b's slot.
                  const uint64_t both = D == 64 ? with_lbo(high, weighted + (updates % C::kBuffers) * C::kRest - (slots + now.b * C::kSlot)) : high;
#pragma unroll
                  for (int s = 0; s < 8; ++s)
                    if (issues) mma_bf16(d, both + s * 128u, c + s * 128u, id_update, s > 0 || !first);
                  if constexpr (D == 128) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                      if (issues) mma_bf16(d, rest + s * 128u, c + s * 128u, id_update, 1);
                  }
                  if (issues) mma_commit(added + updates % C::kBuffers);
                  if (last && issues) mma_commit(whole + tiles % C::kBuffers);
                }
                if (ends_bc(g) && issues) mma_commit(empty + now.b);
                if (ends_bc(g) && issues) mma_commit(empty + now.c);
                __syncwarp();
              }
              if (update) ++updates;
              if (C::kBuffers == 2) read();
            }
          }
        }
      }
      // what was issued has to end before its tensor memory goes
      if (issues) {
        mma_commit(drain + warp - 1);
        mbar_drain(drain + warp - 1, 0);
      }
      __syncwarp();
    }
  } else if (wg == 1) {
    // ---- weighted scores: thread t has row t -------------------------------------
    if (C::kWriters) regs_inc<C::kRegsScores>();
    const int t = threadIdx.x - 128, q = t >> 5;
    const uint32_t row_base = tmem_addr(tmem, q * 32, C::tScores);
    uint32_t unit = 0;
    while (walk.next(w, pc)) {
      if (total || pc.rows == 0) continue;
      const float g2 = log2_decay(p.log_decay, pc.head);
      named_barrier_sync(3, 128);
      powers[t] = exp2f(g2 * (float)t);
      named_barrier_sync(3, 128);
      float2 col[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) col[j] = make_float2(powers[rev ? 2 * j : 31 - 2 * j], powers[rev ? 2 * j + 1 : 30 - 2 * j]);
      for (int k = 0; k < pc.t1 - pc.t0; ++k) {
        const int tile = rev ? pc.t1 - 1 - k : pc.t0 + k, n = min(kTile, pc.rows - tile * kTile);
        for (int g = 0; g < groups; ++g, ++unit) {
          const uint32_t sb = unit % C::kBuffers, at = row_base + sb * 128;
          wait(scored + sb, (unit / C::kBuffers) & 1);
          tc_fence_after();
          // 32 columns at a time.  Away from the diagonal the weight is a power to the block's nearer end times a
          // column's; on it, and where the sequence ends inside a block, each weight comes from the table.  Rolled:
          // unrolled, the block's code was past the instruction caches, and everything in it three times as slow.
#pragma unroll 1
          for (int c0 = 0; c0 < kTile; c0 += 32) {
            float v[32];
            const bool live = rev ? c0 >= 32 * q && c0 < n : c0 <= 32 * q;
            if (live) {
              tmem_ld32(at + c0, v);
              if (c0 != 32 * q && (!rev || c0 + 32 <= n)) {
                const float away = powers[rev ? c0 - t : t - c0 - 31];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float2 x = __fmul2_rn(make_float2(v[2 * j], v[2 * j + 1]), __fmul2_rn(col[j], make_float2(away, away)));
                  v[2 * j] = x.x, v[2 * j + 1] = x.y;
                }
              } else {
                // chosen, not multiplied with 0: the rows behind the sequence may hold anything
                const int end = rev ? n - c0 : 32, off = rev ? c0 - t : t - c0;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const int apart = rev ? off + j : off - j;
                  v[j] = apart >= 0 && j < end ? v[j] * powers[apart & 127] : 0.f;
                }
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.f;
            }
            // two numbers to a column: they lie where scores already read were
            float packed[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) packed[j] = __uint_as_float(pack_bf16(v[2 * j], v[2 * j + 1]));
            tmem_st16(at + c0 / 2, packed);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + sb);
        }
      }
    }
  } else if (wg == 2 || wg == 4) {
    // ---- rows: thread t has row t, of b to weigh it and of the results to write them ----
    regs_dec<C::kRegsRows>();
    const int t = threadIdx.x & 127, q = t >> 5;
    const bool weighs = wg == 2, results = !total && (!C::kWriters || wg == 4);
    const uint32_t row_base = tmem_addr(tmem, q * 32, 0);
    Ring r;
    Unit now{};
    uint32_t outs = 0, updates = 0, units = 0;
    const CUtensorMap *out_map = p.outs + which;
    // the result that is to be written next
    struct {
      int row, head, n;
      uint32_t slot;
      float read;
    } due{0, 0, -1, 0, 0.f};
    int leaving = -1;
    auto write = [&]() {
      if (due.n < 0) return;
      wait(done, outs & 1);
      ++outs;
      tc_fence_after();
      const bool whole_tile = due.n == kTile;
      // a whole tile goes by TMA, 32 rows from each warp: from a place of its own, or at D = 128 from a's slot, whose
      // rows are not needed any more
      const uint32_t stage = C::kStage ? stage_at : slots + due.slot * C::kSlot;
      if (C::kStage) {
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
      }
      __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(m.out) + ((long long)due.row + t) * m.out_row + (long long)due.head * D;
#pragma unroll 1
      for (int x = 0; x < D; x += 16) {
        float v[16], u[16];
        tmem_ld16x2(row_base + C::tRead + x, row_base + C::tWithin + x, v, u);
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          h[j] = pack_bf16(fmaf(v[2 * j], due.read, m.within * u[2 * j]), fmaf(v[2 * j + 1], due.read, m.within * u[2 * j + 1]));
        if (whole_tile) {
          st_shared_v4(stage + sw128_offset(t, x, kTile), h[0], h[1], h[2], h[3]);
          st_shared_v4(stage + sw128_offset(t, x + 8, kTile), h[4], h[5], h[6], h[7]);
        } else if (t < due.n) {
          *reinterpret_cast<uint4 *>(dst + x) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4 *>(dst + x + 8) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      tc_fence_before();
      if (whole_tile) fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(taken);
        if (whole_tile) {
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_store_3d(out_map, generic + (stage - base) + x * 16384 + q * 4096, x * 64, due.head, due.row + 32 * q);
          tma_store_commit();
          leaving = C::kStage ? -1 : (int)due.slot;
        } else if (!C::kStage) {
          mbar_arrive(empty + due.slot);
        }
      }
      __syncwarp();
      due.n = -1;
    };
    // The slot from which the last tile is stored, given back as late as the ring allows: a store waits its turn
    // among the loads.
    auto give_back = [&]() {
      if (leaving >= 0) {
        tma_store_wait_read();
        mbar_arrive(empty + leaving);
        leaving = -1;
      }
    };
    while (walk.next(w, pc)) {
      if ((total && !piece_has_total(m, pc)) || pc.rows == 0) continue;
      const float g2 = log2_decay(p.log_decay, pc.head);
      const float up = exp2f(g2 * (float)(t + 1)), down_whole = exp2f(g2 * (float)(kTile - 1 - t));
      for (int k = 0; k < pc.t1 - pc.t0; ++k) {
        const int tile = rev ? pc.t1 - 1 - k : pc.t0 + k, n = min(kTile, pc.rows - tile * kTile);
        // rows past n are neither weighed nor written
        const float down = n == kTile ? down_whole : exp2f(g2 * (float)(n - 1 - t)), weight = m.add * (rev ? up : down);
        for (int g = 0; g < groups; ++g, ++units) {
          advance(now, r, g);
          const uint32_t b = slots + now.b * C::kSlot, c = slots + now.c * C::kSlot;
          const bool writes = !total && (!sums || g == groups - 1), update = sums || g == groups - 1;
          if (weighs) {
            if (C::kStage == 0) {  // the ring is short: this unit's b may wait for it
              if (lane == 0) give_back();
              __syncwarp();
            }
            wait(full + units % kUnits, (units / kUnits) & 1);
            if (!total) wait(scored + units % C::kBuffers, (units / C::kBuffers) & 1);  // the scores have read b
            if (update) {
              const uint32_t rest = weighted + (updates % C::kBuffers) * C::kRest, high = b;
              if (updates >= C::kBuffers) wait(added + updates % C::kBuffers, (updates / C::kBuffers + 1) & 1);
              ++updates;
              // a row's sixteen-byte pieces lie at their place in the row's 128 bytes, exclusive-or the row's place in eight
              const uint32_t at_row = (uint32_t)(t >> 3) * 1024u + (uint32_t)(t & 7) * 128u, swap = (uint32_t)(t & 7) << 4;
              if (t < n) {
                // two pieces of eight columns at a time, their loads ahead of the arithmetic
#pragma unroll 1
                for (int x = 0; x < D / 8; x += 2) {
                  const uint32_t half = at_row + (uint32_t)(x >> 3) * (kTile * 128u);
                  uint32_t off[2], raw[8], h[8], l[8];
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    off[i] = half + ((uint32_t)(((x & 7) + i) << 4) ^ swap);
                    ld_shared_v4(b + off[i], raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]);
                  }
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float2 v = __fmul2_rn(make_float2(__uint_as_float(raw[j] << 16), __uint_as_float(raw[j] & 0xffff0000u)),
                                                make_float2(weight, weight));
                    h[j] = pack_bf16(v.x, v.y);
                    // v - h, exactly
                    const float2 r2 = __ffma2_rn(make_float2(__uint_as_float(h[j] << 16), __uint_as_float(h[j] & 0xffff0000u)),
                                                 make_float2(-1.f, -1.f), v);
                    l[j] = pack_bf16(r2.x, r2.y);
                  }
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    st_shared_v4(high + off[i], h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
                    st_shared_v4(rest + off[i], l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
                  }
                }
              } else {
#pragma unroll 1
                for (int x = 0; x < D; x += 8) {
                  st_shared_v4(high + sw128_offset(t, x, kTile), 0, 0, 0, 0);
                  st_shared_v4(rest + sw128_offset(t, x, kTile), 0, 0, 0, 0);
                }
              }
            }
            if (loads_bc(g) && t >= n) {
              // rows behind the sequence: 0 times whatever they hold has to be 0
#pragma unroll 1
              for (int x = 0; x < D; x += 8) st_shared_v4(c + sw128_offset(t, x, kTile), 0, 0, 0, 0);
            }
            if (update || n < kTile) {
              fence_async_smem();
              named_barrier_sync(2, 128);
            }
            if (t == 0) mbar_arrive(turned + units % kUnits);
            if (lane == 0) {
              if (ends_bc(g)) mbar_arrive(empty + now.b);
              if (!total && ends_a(g) && (C::kStage || !writes)) mbar_arrive(empty + now.a);
              if (ends_bc(g)) mbar_arrive(empty + now.c);
            }
          }
          if (!results) continue;
          // where the rows' warpgroup does both, the last unit's result, while the MMAs take what was handed out
          if (!C::kWriters) write();
          if (writes) {
            due.row = pc.row0 + tile * kTile;
            due.head = pc.head * m.a_heads + (sums ? 0 : g);
            due.n = n;
            due.slot = now.a;
            due.read = m.read * (rev ? down : up);
            if (C::kWriters) write();
          }
        }
      }
    }
    write();
    give_back();
    tma_store_wait_all();  // what this thread has stored leaves shared memory before the block does
  } else {
    // ---- the state -----------------------------------------------------------------
    // Thread t has row t of it (D = 128), or half of row t % 64: with D = 64
    // the update's rows 0-63 are those of the high parts and 64-127 those of
    // the remainders, so two threads exchange halves and add.
    regs_inc<C::kRegsState>();
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
        const uint32_t own = t >= 64 ? 32 : 0;
        float u[32];
        tmem_ld32(from + (32 - own), u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4(exchange + (i * 128 + t) * 16, __float_as_uint(u[4 * i]), __float_as_uint(u[4 * i + 1]),
                       __float_as_uint(u[4 * i + 2]), __float_as_uint(u[4 * i + 3]));
        tmem_ld32(from + own, u);
        named_barrier_sync(kBar, 128);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x[4];
          ld_shared_v4f(exchange + (i * 128 + (t ^ 64)) * 16, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[4 * i + j] = fmaf(s[4 * i + j], keep, u[4 * i + j] + x[j]);
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
      } else if ((reinterpret_cast<uintptr_t>(start) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kOwn; i += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(start + first + i);
          s[i] = f.x, s[i + 1] = f.y, s[i + 2] = f.z, s[i + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) s[i] = start[first + i];
      }
      const int count = pc.rows == 0 ? 0 : pc.t1 - pc.t0;
      for (int k = 0; k < count; ++k) {
        const int tile = rev ? pc.t1 - 1 - k : pc.t0 + k, n = min(kTile, pc.rows - tile * kTile);
        publish();
        take(exp2f(g2 * (float)n));
      }
      float *end = piece_end(w, m, pc, part);
      if (end && m.transposed) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) end[first + i * D] = s[i];
      } else if (end && (reinterpret_cast<uintptr_t>(end) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kOwn; i += 4)
          *reinterpret_cast<float4 *>(end + first + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      } else if (end) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) end[first + i] = s[i];
      }
    }
  }
  __syncthreads();
  if (*abort && threadIdx.x == 0)  // copies still on their way land before the block leaves
    for (int i = 0; i < kUnits; ++i)
      for (uint32_t parity = 0; parity < 2; ++parity) mbar_drain(full + i, parity, 20000000ull);
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, bool TOTAL, bool REV, bool GROUPED> cudaError_t launch(const TcArgs &a, cudaStream_t st) {
  using C = Cfg<D, TOTAL>;
  static SharedMemory allowed;
  cudaError_t e = allowed.allow(tc_kernel<D, TOTAL, REV, GROUPED>, C::kBytes);
  if (e != cudaSuccess) return e;
  tc_kernel<D, TOTAL, REV, GROUPED><<<a.work.parts * a.mixes, C::kThreads, C::kBytes, st>>>(a);
  return cudaGetLastError();
}

// Passes of one direction.
template <int D> cudaError_t launch_passes(const TcArgs &a, bool total, bool rev, bool grouped, cudaStream_t st) {
  if (total && !rev) return launch<D, true, false, false>(a, st);  // sums of k v^T: once for all of a group's heads
  if (total) return grouped ? launch<D, true, true, true>(a, st) : launch<D, true, true, false>(a, st);
  if (rev) return grouped ? launch<D, false, true, true>(a, st) : launch<D, false, true, false>(a, st);
  return grouped ? launch<D, false, false, true>(a, st) : launch<D, false, false, false>(a, st);
}

}  // namespace
}  // namespace decay
}  // namespace slim
