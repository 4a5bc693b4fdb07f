// decay_generic.cu -- linear attention with a decay on the CUDA cores: fp32 rows, any head
// widths up to 256, any strides.
//
// A block goes through its share of the tiles (decay.h) for 64 of the y
// columns, with the state [x][64] in shared memory in fp32 and everything of
// a tile beside it: for each tile the weighted scores (a b^T, tile x tile),
// their product with c, the product of a with the state, and the rows' sum
// into the state, as register tiles of 4 x 4 or 2 x 4 results a thread.
//
// All products are fp32 FMAs, about 8 x y + 4 tile (x + y) flops a row: at
// x = y = 64 the bound is the FMA rate, not the rows' bytes (a tile of 64
// rows is 2.1 MFLOP against 64 KB).
#include "decay_common.cuh"
#include "kernels.h"

namespace slim {
namespace decay {
namespace {

constexpr int kThreads = 256, kCols = 64, kPitch = kCols + 4;

// Floats from row to row of a and b: an odd number of 16-byte units, so that
// consecutive rows start in different banks.
__host__ __device__ inline int row_pitch(int x) { return ((x + 3) / 4 | 1) * 4; }

template <int TILE> size_t smem_bytes(int x) {
  return sizeof(float) * ((size_t)2 * TILE * row_pitch(x) + TILE * kPitch + TILE * (TILE + 4) + (size_t)x * kPitch + TILE);
}

// rows [row, row + n) of a head into dst (row pitch `pitch`), zeros below and in columns [cols, padded)
template <typename T, int TILE>
__device__ __forceinline__ void load_rows(float *dst, int pitch, int padded, const void *src, long long stride,
                                          long long row, int n, int col0, int cols) {
  const T *p = static_cast<const T *>(src);
  for (int i = threadIdx.x; i < TILE * padded; i += kThreads) {
    const int r = i / padded, c = i - r * padded;
    dst[r * pitch + c] = r < n && c < cols ? to_f32(p[(row + r) * stride + col0 + c]) : 0.f;
  }
}

template <typename T, int TILE>
__global__ void __launch_bounds__(kThreads) mix_kernel(Launch l) {
  extern __shared__ float4 smem4[];
  constexpr int R = TILE / 16;
  const Mix &m = l.mix[blockIdx.z];
  const Work &w = l.work;
  const int y0 = blockIdx.y * kCols, part = blockIdx.x;
  if (y0 >= m.y) return;
  const int ny = min(kCols, m.y - y0);
  const int px = row_pitch(m.x), x4 = (m.x + 3) / 4 * 4;
  float *A = reinterpret_cast<float *>(smem4), *B = A + TILE * px, *C = B + TILE * px, *P = C + TILE * kPitch,
        *S = P + TILE * (TILE + 4), *lam = S + (size_t)m.x * kPitch;  // lam[n] = lambda^n
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int groups = max(m.a_heads, m.b_heads);
  const bool total = m.totals != nullptr;

  Walk walk(w, part, m.rev);
  Piece p;
  while (walk.next(w, p)) {
    if (total && !piece_has_total(m, p)) continue;
    const float g2 = log2_decay(l.log_decay, p.head);
    const float *start = piece_start(w, m, p, part);
    __syncthreads();  // the last piece's state is read
    for (int i = threadIdx.x; i < TILE; i += kThreads) lam[i] = exp2f(g2 * (float)i);
    const float lam1 = exp2f(g2);
    for (int i = threadIdx.x; i < m.x * kCols; i += kThreads) {
      const int r = i / kCols, c = i - r * kCols;
      float v = 0.f;
      if (start && c < ny) v = start[m.transposed ? (size_t)(y0 + c) * m.x + r : (size_t)r * m.y + y0 + c];
      S[r * kPitch + c] = v;
    }
    for (int k = 0; k < p.t1 - p.t0; ++k) {
      const int tile = m.rev ? p.t1 - 1 - k : p.t0 + k;
      const int n = min(TILE, p.rows - tile * TILE);  // 0 in an empty sequence
      const long long row = (long long)p.row0 + (long long)tile * TILE;
      if (n <= 0) break;
      float acc[R][4] = {}, from[R][4] = {};
      for (int g = 0; g < groups; ++g) {
        __syncthreads();
        const int bh = p.head * m.b_heads + (m.b_heads > 1 ? g : 0), ah = p.head * m.a_heads + (m.a_heads > 1 ? g : 0);
        const bool new_b = g == 0 || m.b_heads > 1, new_a = !total && (g == 0 || m.a_heads > 1);
        if (new_b) {
          load_rows<T, TILE>(B, px, x4, m.b, m.b_row, row, n, bh * m.x, m.x);
          load_rows<T, TILE>(C, kPitch, kCols, m.c, m.c_row, row, n, bh * m.y + y0, ny);
        }
        if (new_a) load_rows<T, TILE>(A, px, x4, m.a, m.a_row, row, n, ah * m.x, m.x);
        __syncthreads();
        if (!total) {
          // scores of rows ty + 16 i and tx + 16 j
          float s[R][R] = {};
          for (int k4 = 0; k4 < x4; k4 += 4) {
            float4 av[R], bv[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
              av[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * px + k4);
              bv[i] = *reinterpret_cast<const float4 *>(B + (tx + 16 * i) * px + k4);
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
              for (int j = 0; j < R; ++j) {
                s[i][j] = fmaf(av[i].x, bv[j].x, s[i][j]);
                s[i][j] = fmaf(av[i].y, bv[j].y, s[i][j]);
                s[i][j] = fmaf(av[i].z, bv[j].z, s[i][j]);
                s[i][j] = fmaf(av[i].w, bv[j].w, s[i][j]);
              }
          }
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < R; ++j) {
              const int ri = ty + 16 * i, rj = tx + 16 * j, apart = m.rev ? rj - ri : ri - rj;
              // chosen, not multiplied with 0: what lies outside may be anything
              P[ri * (TILE + 4) + rj] = apart >= 0 && rj < n ? s[i][j] * lam[apart] : 0.f;
            }
          if (new_a) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) from[i][j] = 0.f;
            for (int k1 = 0; k1 < m.x; ++k1) {
              const float4 sv = *reinterpret_cast<const float4 *>(S + k1 * kPitch + 4 * tx);
#pragma unroll
              for (int i = 0; i < R; ++i) {
                const float av = A[(ty + 16 * i) * px + k1];
                from[i][0] = fmaf(av, sv.x, from[i][0]);
                from[i][1] = fmaf(av, sv.y, from[i][1]);
                from[i][2] = fmaf(av, sv.z, from[i][2]);
                from[i][3] = fmaf(av, sv.w, from[i][3]);
              }
            }
          }
          __syncthreads();  // scores are written; the state and b are read
          if (new_a) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
          }
          for (int j4 = 0; j4 < TILE; j4 += 4) {
            float4 cv[4], pv[R];
#pragma unroll
            for (int j = 0; j < 4; ++j) cv[j] = *reinterpret_cast<const float4 *>(C + (j4 + j) * kPitch + 4 * tx);
#pragma unroll
            for (int i = 0; i < R; ++i) pv[i] = *reinterpret_cast<const float4 *>(P + (ty + 16 * i) * (TILE + 4) + j4);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float q[4] = {pv[i].x, pv[i].y, pv[i].z, pv[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                acc[i][0] = fmaf(q[j], cv[j].x, acc[i][0]);
                acc[i][1] = fmaf(q[j], cv[j].y, acc[i][1]);
                acc[i][2] = fmaf(q[j], cv[j].z, acc[i][2]);
                acc[i][3] = fmaf(q[j], cv[j].w, acc[i][3]);
              }
            }
          }
          if (m.a_heads > 1 || g == groups - 1) {
            T *out = static_cast<T *>(m.out);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const int r = ty + 16 * i;
              if (r >= n) continue;
              const float read = m.read * (m.rev ? lam[n - 1 - r] : lam[r] * lam1);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (4 * tx + j < ny)
                  out[(row + r) * m.out_row + (long long)ah * m.y + y0 + 4 * tx + j] =
                      from_f32<T>(fmaf(from[i][j], read, m.within * acc[i][j]));
            }
          }
        }
        if (m.b_heads > 1 || g == groups - 1) {
          // the rows' sum into the state, which decays once a tile
          const float keep = m.b_heads == 1 || g == 0 ? exp2f(g2 * (float)n) : 1.f;
          for (int i = threadIdx.x; i < n * m.x; i += kThreads) {
            const int r = i / m.x, c = i - r * m.x;
            B[r * px + c] *= m.add * (m.rev ? lam[r] * lam1 : lam[n - 1 - r]);
          }
          __syncthreads();
          for (int x0 = ty; x0 < m.x; x0 += 64) {
            float s[4][4] = {};
            for (int j = 0; j < n; ++j) {
              const float4 cv = *reinterpret_cast<const float4 *>(C + j * kPitch + 4 * tx);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float bv = B[j * px + min(x0 + 16 * i, m.x - 1)];
                s[i][0] = fmaf(bv, cv.x, s[i][0]);
                s[i][1] = fmaf(bv, cv.y, s[i][1]);
                s[i][2] = fmaf(bv, cv.z, s[i][2]);
                s[i][3] = fmaf(bv, cv.w, s[i][3]);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (x0 + 16 * i >= m.x) break;
              float4 &sv = *reinterpret_cast<float4 *>(S + (x0 + 16 * i) * kPitch + 4 * tx);
              sv = make_float4(fmaf(sv.x, keep, s[i][0]), fmaf(sv.y, keep, s[i][1]), fmaf(sv.z, keep, s[i][2]),
                               fmaf(sv.w, keep, s[i][3]));
            }
          }
        }
      }
    }
    float *end = piece_end(w, m, p, part);
    __syncthreads();
    if (end)
      for (int i = threadIdx.x; i < m.x * ny; i += kThreads) {
        const int r = i / ny, c = i - r * ny;
        end[m.transposed ? (size_t)(y0 + c) * m.x + r : (size_t)r * m.y + y0 + c] = S[r * kPitch + c];
      }
  }
}

template <typename T, int TILE> cudaError_t launch(const Launch &l, int widest_x, int widest_y, cudaStream_t st) {
  const size_t bytes = smem_bytes<TILE>(widest_x);
  static SharedMemory allowed;
  cudaError_t e = allowed.allow(mix_kernel<T, TILE>, smem_bytes<TILE>(TILE == 64 ? 128 : 256));
  if (e != cudaSuccess) return e;
  const dim3 grid(l.work.parts, (widest_y + kCols - 1) / kCols, l.mixes);
  mix_kernel<T, TILE><<<grid, kThreads, bytes, st>>>(l);
  return cudaGetLastError();
}

}  // namespace

// Rows of a tile: 64, or where a head is wider than 128 columns 32, so that
// a tile and the state fit into shared memory.
int generic_tile(int dk, int dv) { return max(dk, dv) > 128 ? 32 : 64; }

template <typename T> cudaError_t mix_generic(const Launch &l, cudaStream_t st) {
  ProfScope ps(l.mix[0].totals ? "decay_totals_f32" : "decay_mix_f32", st);
  int x = 0, y = 0;
  for (int i = 0; i < l.mixes; ++i) x = max(x, l.mix[i].x), y = max(y, l.mix[i].y);
  return l.work.tile == 64 ? launch<T, 64>(l, x, y, st) : launch<T, 32>(l, x, y, st);
}

template cudaError_t mix_generic<float>(const Launch &, cudaStream_t);
template cudaError_t mix_generic<__nv_bfloat16>(const Launch &, cudaStream_t);

}  // namespace decay
}  // namespace slim
