// decay_common.cuh -- walking the list of tiles (decay.h).
#pragma once

#include "common.cuh"
#include "decay.h"

namespace slim {
namespace decay {

// log2 of a head's decay: at most 0 (a larger logarithm counts as 0), and finite, so that
// lambda^0 = 1 for lambda = 0 too.  A NaN stays one.
__device__ __forceinline__ float log2_decay(const float *log_decay, int head) {
  float g = log_decay[head] * 1.4426950408889634f;
  g = g > 0.f ? 0.f : g;
  return g < -1e6f ? -1e6f : g;
}

// First row and rows of a sequence, kept inside the tensor whatever cu holds.
__device__ __forceinline__ int2 bounds(const Work &w, int seq) {
  if (!w.cu) return make_int2(seq * w.length, w.length);
  const int a = min(max(w.cu[seq], 0), w.tokens);
  return make_int2(a, min(max(w.cu[seq + 1], a), w.tokens) - a);
}

// An empty sequence has one tile, of no rows, which hands its state on.
__device__ __forceinline__ int tiles_of(const Work &w, int length) { return max(1, (length - 1) / w.tile + 1); }

// The place in the list where share `part` begins.
struct Place {
  int head, seq, tile;
};
__device__ __forceinline__ Place share_begin(const Work &w, int part) {
  if (w.where) {
    const int4 r = w.where[part];
    return Place{r.x, r.y, r.z};
  }
  const int each = tiles_of(w, bounds(w, 0).y);  // all sequences are as long
  const long long tiles = (long long)each * w.seqs, f = tiles * w.heads * part / w.parts;
  const int head = (int)(f / tiles), t = (int)(f - head * tiles);
  return Place{head, t / each, t % each};
}

// A share's part of one sequence: tiles [t0, t1) of `tiles`.
struct Piece {
  int head, seq, t0, t1, tiles, row0, rows;  // the sequence's first row and rows
  __device__ bool begins() const { return t0 == 0; }
  __device__ bool ends() const { return t1 == tiles; }
};

// The pieces of a share, in the direction of time or against it.
struct Walk {
  Place at, last;
  bool rev;
  __device__ Walk(const Work &w, int part, bool reversed) : rev(reversed) {
    at = share_begin(w, part);
    last = share_begin(w, part + 1);
  }
  __device__ bool next(const Work &w, Piece &p) {
    if (at.head == last.head && at.seq == last.seq && at.tile == last.tile) return false;
    if (!rev) {
      const int2 b = bounds(w, at.seq);
      const int n = tiles_of(w, b.y);
      const bool inside = at.head == last.head && at.seq == last.seq;
      p = Piece{at.head, at.seq, at.tile, inside ? last.tile : n, n, b.x, b.y};
      if (inside) {
        at = last;
      } else {
        at.tile = 0;
        if (++at.seq == w.seqs) at.seq = 0, ++at.head;
      }
    } else {
      if (last.tile == 0) {
        if (--last.seq < 0) last.seq = w.seqs - 1, --last.head;
        last.tile = tiles_of(w, bounds(w, last.seq).y);
      }
      const int2 b = bounds(w, last.seq);
      const bool inside = at.head == last.head && at.seq == last.seq;
      p = Piece{last.head, last.seq, inside ? at.tile : 0, last.tile, tiles_of(w, b.y), b.x, b.y};
      last.tile = p.t0;
    }
    return true;
  }
};

// Where a piece's state comes from and goes to (NULL: zero, nowhere).
__device__ __forceinline__ long long place_of(const Mix &m, int seq) { return m.place ? m.place[seq] : seq; }

__device__ __forceinline__ const float *piece_start(const Work &w, const Mix &m, const Piece &p, int part) {
  const size_t n = (size_t)m.x * m.y;
  const bool begins = m.rev ? p.ends() : p.begins(), ends = m.rev ? p.begins() : p.ends();
  if (m.totals) return nullptr;
  if (!begins) return m.incoming + part * n;
  if (!ends && m.first) return m.first + part * n;
  const long long at = m.start ? place_of(m, p.seq) : -1;
  return at < 0 ? nullptr : m.start + ((size_t)at * w.heads + p.head) * n;
}

__device__ __forceinline__ float *piece_end(const Work &w, const Mix &m, const Piece &p, int part) {
  const size_t n = (size_t)m.x * m.y;
  const bool ends = m.rev ? p.begins() : p.ends();
  if (m.totals) return m.totals + part * n;
  const long long at = m.end && ends ? place_of(m, p.seq) : -1;
  return at < 0 ? nullptr : m.end + ((size_t)at * w.heads + p.head) * n;
}

// Whether the totals' launch has to go through a piece: it ends (in the
// direction of the pass) at the share's border, inside its sequence.
__device__ __forceinline__ bool piece_has_total(const Mix &m, const Piece &p) { return m.rev ? !p.begins() : !p.ends(); }

}  // namespace decay
}  // namespace slim
