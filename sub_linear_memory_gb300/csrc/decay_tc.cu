// decay_tc.cu -- linear attention with a decay on the tensor cores: which calls can run there, their tensor maps and
// launches (kernels: decay_tc.cuh).
#include "decay_tc_args.h"
#include "kernels.h"
#include "tma_host.h"

namespace slim {
namespace decay {
namespace {

constexpr int kTile = 128;

// [tokens][heads][D], rows `row` elements apart; boxes of `rows` rows and 64 columns of one head.
bool make_map(CUtensorMap *map, const void *p, int tokens, long long heads, int d, long long row, int rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)row * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
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
  TcArgs all{};
  all.work = l.work;
  all.log_decay = l.log_decay;
  all.status = status;
  int used = 0;
  struct { const void *p; int heads; long long row; } seen[4] = {};
  auto map_of = [&](const void *p, int heads, long long row, int d) -> int {
    for (int i = 0; i < used; ++i)
      if (seen[i].p == p && seen[i].heads == heads && seen[i].row == row) return i;
    if (used == 4 || !make_map(all.maps + used, p, l.work.tokens, (long long)heads * l.work.heads, d, row, kTile)) return -1;
    seen[used] = {p, heads, row};
    return used++;
  };
  for (int rev = 0; rev < 2; ++rev) {
    TcArgs a = all;
    bool total = false, grouped = false;
    for (int i = 0; i < l.mixes; ++i) {
      if (l.mix[i].rev != rev) continue;
      const int n = a.mixes++;
      const Mix &m = a.mix[n] = l.mix[i];
      total = m.totals != nullptr;
      grouped = m.a_heads > 1 || m.b_heads > 1;
      const int ia = total ? 0 : map_of(m.a, m.a_heads, m.a_row, m.x), ib = map_of(m.b, m.b_heads, m.b_row, m.x),
                ic = map_of(m.c, m.b_heads, m.c_row, m.x);
      if (ia < 0 || ib < 0 || ic < 0) return cudaErrorInvalidValue;
      a.a[n] = (signed char)ia, a.b[n] = (signed char)ib, a.c[n] = (signed char)ic;
      if (!total && !make_map(a.outs + n, m.out, l.work.tokens, (long long)m.a_heads * l.work.heads, m.y, m.out_row, 32))
        return cudaErrorInvalidValue;
    }
    if (a.mixes == 0) continue;
    for (int i = 0; i < 4; ++i) a.maps[i] = all.maps[i < used ? i : 0];
    const cudaError_t e = (l.mix[0].x == 64 ? tc_passes_64 : tc_passes_128)(a, total, rev != 0, grouped, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace decay
}  // namespace slim
