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

// One block: the tiles of all sequences are counted, then each share finds
// the sequence that it begins in; and each sequence's place in the cache,
// which the first of the sequences that name it has.
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
  // first[i]: the tiles before sequence i, in shared memory where they fit
  __shared__ long long near[kPrepThreads];
  long long *first = w.seqs <= kPrepThreads ? near : p.first;
  long long tiles = 0;
  for (int i = 0; i < w.seqs; i += kPrepThreads) {
    const long long before = block_exclusive(i + t < w.seqs ? tiles_of(w, bounds(w, i + t).y) : 0, warp_sums, tiles);
    if (i + t < w.seqs) first[i + t] = before;
  }
  __syncthreads();
  const long long all = tiles * w.heads;
  for (int c = t; c <= w.parts; c += kPrepThreads) {
    const long long f = all * c / w.parts;
    const int head = (int)(f / tiles);
    const long long r = f - head * tiles;
    int lo = 0, hi = head < w.heads ? w.seqs - 1 : 0;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= r) lo = mid; else hi = mid - 1;
    }
    p.where[c] = make_int4(head, lo, head < w.heads ? (int)(r - first[lo]) : 0, 0);
  }
}

constexpr int kScanThreads = 128;

template <int VEC> struct Elements { using Type = float; };
template <> struct Elements<4> { using Type = float4; };
__device__ __forceinline__ float join(float x, float keep, float t) { return fmaf(x, keep, t); }
__device__ __forceinline__ float4 join(float4 x, float keep, float4 t) {
  return make_float4(fmaf(x.x, keep, t.x), fmaf(x.y, keep, t.y), fmaf(x.z, keep, t.z), fmaf(x.w, keep, t.w));
}

// Share c's incoming state from those of the shares before it (behind it in
// reverse) in the same sequence.  A block goes along one sequence's shares
// from the one that holds its beginning, for its own elements of the state,
// VEC to a thread.
template <int VEC> __global__ void __launch_bounds__(kScanThreads) scan_kernel(Scan s) {
  const Work &w = s.work;
  const auto &side = s.side[blockIdx.z];
  using V = typename Elements<VEC>::Type;
  const int e = (blockIdx.x * kScanThreads + threadIdx.x) * VEC;
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
  V x{};
  if (at >= 0 && live) x = *reinterpret_cast<const V *>(side.start + ((size_t)at * w.heads + edge.head) * s.states + e);
  if (live && side.first) *reinterpret_cast<V *>(side.first + (size_t)c * s.states + e) = x;
  int from = side.rev ? b.y : 0;  // rows already passed lie before (behind) this one
  // The sequence's next shares, a block's threads' worth at a time: where each ends, from all threads at once; then
  // along them with eight totals on their way.
  __shared__ int rows[kScanThreads + 1];
  while (true) {
    const int next = side.rev ? c + step * (int)threadIdx.x : c + 1 + (int)threadIdx.x;
    int to = -1;  // behind the sequence
    if (next >= 0 && next <= w.parts) {
      const Place q = share_begin(w, next);
      if (q.head == edge.head && q.seq == edge.seq && q.tile != 0) to = q.tile * w.tile;
    }
    __syncthreads();
    rows[threadIdx.x] = to;
    if (threadIdx.x == 0) rows[kScanThreads] = -1;
    __syncthreads();
    int k = 0;
    for (bool more = true; more;) {
      V t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        t[j] = live && k + j < kScanThreads && rows[k + j] >= 0
                   ? *reinterpret_cast<const V *>(side.totals + (size_t)(c + step * (k + j)) * s.states + e)
                   : V{};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int here = more ? rows[k] : -1;
        if (here < 0) {
          more = false;
        } else {
          // a share may be empty, and has no total then
          if (here != from) x = join(x, exp2f(g * (float)abs(here - from)), t[j]);
          from = here;
          ++k;
          if (live) *reinterpret_cast<V *>(side.incoming + (size_t)(c + step * k) * s.states + e) = x;
        }
      }
    }
    if (k < kScanThreads) return;
    c += step * kScanThreads;
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
  bool vec = s.states % 4 == 0;  // the workspace's parts are aligned, the caller's states may not be
  for (int i = 0; i < s.sides; ++i) vec = vec && (reinterpret_cast<uintptr_t>(s.side[i].start) & 15) == 0;
  const int each = kScanThreads * (vec ? 4 : 1);
  const dim3 grid((s.states + each - 1) / each, s.work.parts, s.sides);
  if (vec)
    scan_kernel<4><<<grid, kScanThreads, 0, st>>>(s);
  else
    scan_kernel<1><<<grid, kScanThreads, 0, st>>>(s);
  return cudaGetLastError();
}

}  // namespace decay
}  // namespace slim
