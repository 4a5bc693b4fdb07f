// decay.h -- linear attention with a decay for each head: what its host entry
// points (decay_api.cu) and kernels share.
//
// For a key-value head with decay lambda and its query heads,
//   S_t = lambda S_(t-1) + k_t v_t^T,   o_t = scale q_t^T S_t.
// Every pass is one operator over rows of three operands,
//   out_i = sum_{j <= i} lambda^(i-j) (a_i . b_j) c_j + lambda^(i+1) a_i X,
// X the state (sum of b_j c_j^T, with decay) before the first row:
//   o  = mix(q, k, v), dq = mix(do, v, k) with the transposed state, and in
//   reverse time, with the gradient's state G, dv = mix(k, q, do) and
//   dk = mix(v, do, q) with the transposed G (j >= i; lambda^(n-1-i) a_i X,
//   because the gradient that reaches the state behind row i has not passed
//   that row's decay yet).
//
// Rows are cut into tiles, each sequence from its first row on; the tiles of
// all heads, sequence by sequence, are one list, which is cut into `parts`
// equal shares, one for each block.  A share that ends inside a sequence
// gives its sum (the `total`) to the ones behind it: a first launch forms the
// totals, a second one adds them up along each sequence, and the main launch
// starts every share from the state it needs.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include <atomic>

#include "../../include/slim_attn.h"

namespace slim {
namespace decay {

// A kernel's leave to use more than 48 KB of shared memory, asked for once on
// each device (a call to the driver costs as much as a launch).
class SharedMemory {
 public:
  template <typename K> cudaError_t allow(K kernel, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<size_t> &most = most_[dev & 63];
    if (dev < 64 && most.load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) most.store(bytes, std::memory_order_relaxed);
    return e;
  }

 private:
  std::atomic<size_t> most_[64] = {};
};

// The list of tiles.
struct Work {
  const int *cu;      // [seqs + 1] first rows, or NULL: seqs sequences of `length` rows
  int tokens, seqs, length, heads, tile, parts;
  const int4 *where;  // [parts + 1] (head, sequence, tile, -) of each share, or NULL where it can be computed
};

// One pass of the operator.
struct Mix {
  const void *a, *b, *c;
  void *out;
  long long a_row, b_row, c_row, out_row;  // elements from row to row; heads are dense
  int x, y;            // columns of a and b, of c and out
  int a_heads, b_heads;  // of a (and out), of b and c, for each key-value head: one of them is 1
  int rev;
  float within, read, add;  // factors of the sum inside a tile, of a X, and of the rows added to the state
  int transposed;      // the state in memory is [y][x]
  const float *incoming;  // [parts][x y]: the state a share starts from, where it starts inside a sequence
  const float *first;  // [parts][x y]: the state of the sequence that a share starts and does not end (or NULL: `start`)
  const float *start;  // [places][heads][x y] (or NULL: zero)
  float *end;          // the same places (or NULL)
  const int *place;    // [seqs] the sequence's place, -1 none (or NULL: its number)
  float *totals;       // not NULL: form the totals alone
};

struct Launch {
  Work work;
  const float *log_decay;  // [heads]
  Mix mix[3];
  int mixes;
};

struct Scan {
  Work work;
  const float *log_decay;
  int states;  // dk dv
  struct {
    const float *totals, *start;
    float *incoming, *first;
    const int *place;
    int rev;
  } side[2];
  int sides;
};

struct Prepare {
  Work work;
  int4 *where;
  long long *first;  // [seqs]
  const int *slots;
  int places;
  int *owner, *place;
};

cudaError_t prepare(const Prepare &p, cudaStream_t st);
cudaError_t scan(const Scan &s, cudaStream_t st);
template <typename T> cudaError_t mix_generic(const Launch &l, cudaStream_t st);
int generic_tile(int dk, int dv);
bool tc_supported(const Launch &l);
cudaError_t mix_tc(const Launch &l, int *status, cudaStream_t st);

// One token of each sequence.
struct Step {
  const void *q, *k, *v;
  void *o;
  long long q_row, k_row, v_row, o_row;
  const float *log_decay;
  float *state;
  const int *slots;
  int rows, places, heads, groups, dk, dv;
  float scale;
};
template <typename T> cudaError_t step(const Step &s, cudaStream_t st);

}  // namespace decay
}  // namespace slim
