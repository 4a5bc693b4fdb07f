// decay_scan.cu -- linear attention with a decay: where each share begins, and
// the state that it starts from.
#include "decay_common.cuh"
#include "kernels.h"

namespace slim {
namespace decay {
namespace {

constexpr int kPrepThreads = 1024;

// Exclusive sums over a block of kPrepThreads; `carry` gains the block's total.
__device__ long long block_exclusive(long long v, long long *warp_sums, long long &carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    long long t = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    warp_sums[lane] = t;
  }
  __syncthreads();
  const long long before = carry + (warp ? warp_sums[warp - 1] : 0) + s - v;
  carry += warp_sums[31];
  __syncthreads();
  return before;
}

// One block: the tiles of all sequences are counted, then a second pass over
// them finds the shares that begin in each; and each sequence's place in the
// cache, which the first of the sequences that name it has.
__global__ void __launch_bounds__(kPrepThreads) prepare_kernel(Prepare p) {
  __shared__ long long warp_sums[32];
  const Work &w = p.work;
  const int t = threadIdx.x;
  if (p.slots) {
    for (int i = t; i < w.seqs; i += kPrepThreads) {
      const int s = p.slots[i];
      if (s >= 0 && s < p.places) p.owner[s] = w.seqs;
    }
    __syncthreads();
    for (int i = t; i < w.seqs; i += kPrepThreads) {
      const int s = p.slots[i];
      if (s >= 0 && s < p.places) atomicMin(p.owner + s, i);
    }
    __syncthreads();
    for (int i = t; i < w.seqs; i += kPrepThreads) {
      const int s = p.slots[i];
      p.place[i] = s >= 0 && s < p.places && atomicAdd(p.owner + s, 0) == i ? s : -1;
    }
  }
  if (!p.where) return;
  long long tiles = 0;
  for (int i = 0; i < w.seqs; i += kPrepThreads)
    block_exclusive(i + t < w.seqs ? tiles_of(w, bounds(w, i + t).y) : 0, warp_sums, tiles);
  const long long all = tiles * w.heads;
  if (t == 0) {
    *p.tiles = tiles;
    p.where[w.parts] = make_int4(w.heads, 0, 0, 0);
  }
  long long carry = 0;
  for (int i = 0; i < w.seqs; i += kPrepThreads) {
    const int n = i + t < w.seqs ? tiles_of(w, bounds(w, i + t).y) : 0;
    const long long first = block_exclusive(n, warp_sums, carry);
    for (int h = 0; h < w.heads && n > 0; ++h) {
      // shares whose first tile f = floor(all c / parts) lies in [at, at + n)
      const long long at = h * tiles + first;
      for (long long c = (at * w.parts + all - 1) / all; c < w.parts; ++c) {
        const long long f = all * c / w.parts;
        if (f >= at + n) break;
        if (f >= at) p.where[c] = make_int4(h, i + t, (int)(f - at), 0);
      }
    }
  }
}

constexpr int kScanThreads = 128;

// Share c's incoming state from those of the shares before it (behind it in
// reverse) in the same sequence.  A block goes along one sequence's shares
// from the one that holds its beginning, for its own elements of the state.
__global__ void __launch_bounds__(kScanThreads) scan_kernel(Scan s) {
  const Work &w = s.work;
  const auto &side = s.side[blockIdx.z];
  const int e = blockIdx.x * kScanThreads + threadIdx.x;
  const int step = side.rev ? -1 : 1;
  int c = blockIdx.y;
  const Place begin = share_begin(w, c), end = share_begin(w, c + 1);
  // the border that this share's total crosses lies inside a sequence, and
  // this share holds that sequence's beginning (its end in reverse)
  const Place edge = side.rev ? begin : end;
  if (edge.tile == 0) return;
  const Place other = side.rev ? end : begin;
  const int2 b = bounds(w, edge.seq);
  const int tiles = tiles_of(w, b.y);
  if (other.head == edge.head && other.seq == edge.seq && other.tile > 0 && other.tile < tiles) return;
  const float g = log2_decay(s.log_decay, edge.head);
  const bool live = e < s.states;
  long long at = side.start ? (side.place ? side.place[edge.seq] : edge.seq) : -1;
  float x = at >= 0 && live ? side.start[((size_t)at * w.heads + edge.head) * s.states + e] : 0.f;
  if (live && side.first) side.first[(size_t)c * s.states + e] = x;
  int from = side.rev ? b.y : 0;  // rows already passed lie before (behind) this one
  Place border = edge;
  while (true) {
    const int to = border.tile * w.tile;
    const float keep = exp2f(g * (float)abs(to - from));
    if (live && to != from) x = fmaf(x, keep, side.totals[(size_t)c * s.states + e]);  // a share may be empty
    c += step;
    if (live) side.incoming[(size_t)c * s.states + e] = x;
    from = to;
    border = share_begin(w, side.rev ? c : c + 1);
    if (border.head != edge.head || border.seq != edge.seq || border.tile == 0) return;
  }
}

}  // namespace

cudaError_t prepare(const Prepare &p, cudaStream_t st) {
  ProfScope ps("decay_prepare", st);
  prepare_kernel<<<1, kPrepThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t scan(const Scan &s, cudaStream_t st) {
  ProfScope ps("decay_scan", st);
  const dim3 grid((s.states + kScanThreads - 1) / kScanThreads, s.work.parts, s.sides);
  scan_kernel<<<grid, kScanThreads, 0, st>>>(s);
  return cudaGetLastError();
}

}  // namespace decay
}  // namespace slim
