// decay_api.cu -- the slim_decay_* entry points of include/slim_attn.h: argument checks, the
// cut into shares, workspace layout and launches.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "decay.h"
#include "kernels.h"

namespace slim {
namespace decay {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxWidth = 256, kMaxGroups = 64;

struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

#define SLIM_TRY(expr)                    \
  do {                                    \
    const slim_status try_st = (expr);    \
    if (try_st != SLIM_OK) return try_st; \
  } while (0)

slim_status finish(cudaError_t err, cudaStream_t st) {
  if (err != cudaSuccess) return SLIM_ERR_CUDA;
#ifdef SLIM_DEBUG
  return slim_attn_sync_status((slim_stream_t)st);
#else
  (void)st;
  return SLIM_OK;
#endif
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int device_sms() {
  static std::atomic<int> known[64] = {};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

slim_status check_shape(const slim_decay_shape *s) {
  if (!s || s->tokens < 0 || s->seqs < 0 || s->heads < 0 || s->groups < 1 || s->dk < 1 || s->dv < 1 || s->places < 0)
    return SLIM_ERR_INVALID_ARG;
  if (s->dk > kMaxWidth || s->dv > kMaxWidth || s->groups > kMaxGroups) return SLIM_ERR_UNSUPPORTED;
  if ((long long)s->heads * s->groups * kMaxWidth >= (1ll << 31)) return SLIM_ERR_UNSUPPORTED;
  return SLIM_OK;
}

// Rows of `cols` dense elements, `row` elements apart.
slim_status check_rows(const void *p, size_t size, int rows, long long row, long long cols) {
  if (!p) return SLIM_ERR_INVALID_ARG;
  if (rows > 1 && row < cols) return SLIM_ERR_INVALID_ARG;
  return aligned(p, size) ? SLIM_OK : SLIM_ERR_UNSUPPORTED;
}

// The cut of the tiles into shares (decay.h).
struct Cut {
  int tile, parts;
  bool joined;  // a share may end inside a sequence
};

Cut cut_tiles(const slim_decay_shape &s, bool equal, int tile, int blocks) {
  const int length = equal ? s.tokens / s.seqs : s.tokens;
  const long long each = length ? (length - 1) / tile + 1 : 1;
  const long long units = s.heads * (equal ? s.seqs * each : (long long)s.tokens / tile + s.seqs);
  if (length <= tile) return Cut{tile, (int)std::min<long long>(units, blocks), false};  // no sequence has two tiles
  return Cut{tile, (int)std::max<long long>(1, std::min<long long>(units / 2, blocks)), true};
}

Cut generic_cut(const slim_decay_shape &s, bool equal) {
  return cut_tiles(s, equal, generic_tile(s.dk, s.dv), 2 * device_sms());
}

// On the tensor cores a block has an SM, and a tile takes a microsecond or so: shares of two tiles at least.
Cut tc_cut(const slim_decay_shape &s, bool equal) { return cut_tiles(s, equal, 128, device_sms()); }

bool tc_shape(const slim_decay_shape &s) { return s.dk == s.dv && (s.dk == 64 || s.dk == 128); }

// The workspace's parts, in bytes from its start.
struct Layout {
  size_t where, first_tile, owner, place, totals[2], incoming[2], first, bytes;
};

Layout layout(const slim_decay_shape &s, const Cut &c, bool bwd) {
  Layout l{};
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t states = c.joined ? sizeof(float) * (size_t)c.parts * s.dk * s.dv : 0;
  l.where = take(sizeof(int4) * (size_t)(c.parts + 1));
  l.first_tile = take(sizeof(long long) * (size_t)s.seqs);
  l.owner = take(sizeof(int) * (size_t)s.places);
  l.place = take(sizeof(int) * (size_t)s.seqs);
  for (int i = 0; i < (bwd ? 2 : 1); ++i) {
    l.totals[i] = take(states);
    l.incoming[i] = take(states);
  }
  l.first = take(bwd ? 0 : states);
  l.bytes = at;
  return l;
}

struct Call {
  Work work;
  Layout at;
  const int *place;
  char *ws;
  bool joined, tensor;
  template <typename T> T *part(size_t offset) const { return reinterpret_cast<T *>(ws + offset); }
};

// Checks the workspace and finds the shares' beginnings.
slim_status begin(const slim_decay_shape &s, const Cut &c, bool bwd, const int *cu, const int *slots, void *workspace,
                  size_t workspace_bytes, cudaStream_t st, Call &call) {
  call.at = layout(s, c, bwd);
  if (!workspace || workspace_bytes < call.at.bytes) return SLIM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return SLIM_ERR_UNSUPPORTED;
  call.ws = static_cast<char *>(workspace);
  call.joined = c.joined;
  call.work = Work{cu, s.tokens, s.seqs, cu ? 0 : s.tokens / s.seqs, s.heads, c.tile, c.parts, nullptr};
  call.place = nullptr;
  const bool listed = cu && s.seqs > 1;
  if (!listed && !slots) return SLIM_OK;
  Prepare p{call.work, nullptr, nullptr, slots, s.places, nullptr, nullptr};
  if (listed) {
    p.where = call.part<int4>(call.at.where);
    p.first = call.part<long long>(call.at.first_tile);
  }
  if (slots) {
    p.owner = call.part<int>(call.at.owner);
    p.place = call.part<int>(call.at.place);
    call.place = p.place;
  }
  if (prepare(p, st) != cudaSuccess) return SLIM_ERR_CUDA;
  call.work.where = p.where;
  return SLIM_OK;
}

// bf16 rows of the widths and alignment that they take go to the tensor cores (a training pass with 16 heads of 64
// and 2 x 32768 rows: 0.62 ms, 8.8 on the CUDA cores), everything else to the CUDA cores.
template <typename T> slim_status run_mix(const Launch &l, bool tensor, cudaStream_t st) {
  if (!tensor) return finish(mix_generic<T>(l, st), st);
  int *status = device_status_ptr();
  return status ? finish(mix_tc(l, status, st), st) : SLIM_ERR_CUDA;
}

template <typename T>
slim_status run_fwd(const void *q, const void *k, const void *v, const float *log_decay, const int *cu,
                    const float *state_in, float *state_out, const int *slots, void *o, const slim_decay_shape *shape,
                    float scale, void *workspace, size_t workspace_bytes, cudaStream_t st) {
  NvtxRange range("slim_decay_fwd");
  SLIM_TRY(check_shape(shape));
  const slim_decay_shape &s = *shape;
  if (s.seqs == 0 || s.heads == 0) return SLIM_OK;
  if (!cu && s.tokens % s.seqs) return SLIM_ERR_INVALID_ARG;
  if ((state_in || state_out) && !slots && s.places != s.seqs) return SLIM_ERR_INVALID_ARG;
  if (!log_decay) return SLIM_ERR_INVALID_ARG;
  const long long wide = (long long)s.heads * s.groups;
  if (s.tokens) {
    SLIM_TRY(check_rows(q, sizeof(T), s.tokens, s.q_row, wide * s.dk));
    SLIM_TRY(check_rows(k, sizeof(T), s.tokens, s.k_row, (long long)s.heads * s.dk));
    SLIM_TRY(check_rows(v, sizeof(T), s.tokens, s.v_row, (long long)s.heads * s.dv));
    SLIM_TRY(check_rows(o, sizeof(T), s.tokens, s.o_row, wide * s.dv));
    if (o == q || o == k || o == v) return SLIM_ERR_INVALID_ARG;
  }
  if (!aligned(log_decay, 4) || !aligned(cu, 4) || !aligned(slots, 4) || !aligned(state_in, 4) || !aligned(state_out, 4))
    return SLIM_ERR_UNSUPPORTED;
  Launch l{};
  l.log_decay = log_decay;
  l.mixes = 1;
  Mix &m = l.mix[0];
  m = Mix{q, k, v, o, s.q_row, s.k_row, s.v_row, s.o_row, s.dk, s.dv, s.groups, 1, 0, scale, scale, 1.f, 0,
          nullptr, nullptr, state_in, state_out, nullptr, nullptr};
  Call c;
  c.tensor = sizeof(T) == 2 && s.tokens && tc_supported(l);
  SLIM_TRY(begin(s, c.tensor ? tc_cut(s, !cu) : generic_cut(s, !cu), false, cu, state_in || state_out ? slots : nullptr,
                 workspace, workspace_bytes, st, c));
  l.work = c.work;
  m.place = c.place;
  if (c.joined) {
    m.incoming = c.part<float>(c.at.incoming[0]);
    m.first = state_in ? c.part<float>(c.at.first) : nullptr;
    Launch t = l;
    t.mix[0].totals = c.part<float>(c.at.totals[0]);
    t.mix[0].a_heads = 1;
    SLIM_TRY(run_mix<T>(t, c.tensor, st));
    Scan sc{c.work, log_decay, s.dk * s.dv, {}, 1};
    sc.side[0] = {t.mix[0].totals, state_in, c.part<float>(c.at.incoming[0]), state_in ? c.part<float>(c.at.first) : nullptr,
                  c.place, 0};
    SLIM_TRY(finish(scan(sc, st), st));
  }
  return run_mix<T>(l, c.tensor, st);
}

template <typename T>
slim_status run_bwd(const void *q, const void *k, const void *v, const float *log_decay, const int *cu, const void *d_o,
                    const float *state_in, const float *g_in, float *g_out, void *dq, void *dk, void *dv,
                    const slim_decay_shape *shape, float scale, void *workspace, size_t workspace_bytes,
                    cudaStream_t st) {
  NvtxRange range("slim_decay_bwd");
  SLIM_TRY(check_shape(shape));
  const slim_decay_shape &s = *shape;
  if (s.seqs == 0 || s.heads == 0) return SLIM_OK;
  if (!cu && s.tokens % s.seqs) return SLIM_ERR_INVALID_ARG;
  if ((state_in || g_in || g_out) && s.places != s.seqs) return SLIM_ERR_INVALID_ARG;
  if (!log_decay || (g_out && (g_out == g_in || g_out == state_in))) return SLIM_ERR_INVALID_ARG;
  const long long wide = (long long)s.heads * s.groups;
  if (s.tokens) {
    SLIM_TRY(check_rows(q, sizeof(T), s.tokens, s.q_row, wide * s.dk));
    SLIM_TRY(check_rows(k, sizeof(T), s.tokens, s.k_row, (long long)s.heads * s.dk));
    SLIM_TRY(check_rows(v, sizeof(T), s.tokens, s.v_row, (long long)s.heads * s.dv));
    SLIM_TRY(check_rows(d_o, sizeof(T), s.tokens, s.o_row, wide * s.dv));
    SLIM_TRY(check_rows(dq, sizeof(T), s.tokens, s.dq_row, wide * s.dk));
    SLIM_TRY(check_rows(dk, sizeof(T), s.tokens, s.dk_row, (long long)s.heads * s.dk));
    SLIM_TRY(check_rows(dv, sizeof(T), s.tokens, s.dv_row, (long long)s.heads * s.dv));
    for (const void *out : {dq, dk, dv})
      if (out == q || out == k || out == v || out == d_o) return SLIM_ERR_INVALID_ARG;
    if (dq == dk || dq == dv || dk == dv) return SLIM_ERR_INVALID_ARG;
  }
  if (!aligned(log_decay, 4) || !aligned(cu, 4) || !aligned(state_in, 4) || !aligned(g_in, 4) || !aligned(g_out, 4))
    return SLIM_ERR_UNSUPPORTED;
  Launch l{};
  l.log_decay = log_decay;
  l.mixes = 3;
  l.mix[0] = Mix{d_o, v, k, dq, s.o_row, s.v_row, s.k_row, s.dq_row, s.dv, s.dk, s.groups, 1, 0, scale, scale, 1.f, 1,
                 nullptr, nullptr, state_in, nullptr, nullptr, nullptr};
  l.mix[1] = Mix{k, q, d_o, dv, s.k_row, s.q_row, s.o_row, s.dv_row, s.dk, s.dv, 1, s.groups, 1, scale, 1.f, scale, 0,
                 nullptr, nullptr, g_in, g_out, nullptr, nullptr};
  l.mix[2] = Mix{v, d_o, q, dk, s.v_row, s.o_row, s.q_row, s.dk_row, s.dv, s.dk, 1, s.groups, 1, scale, 1.f, scale, 1,
                 nullptr, nullptr, g_in, nullptr, nullptr, nullptr};
  Call c;
  c.tensor = sizeof(T) == 2 && s.tokens && tc_supported(l);
  SLIM_TRY(begin(s, c.tensor ? tc_cut(s, !cu) : generic_cut(s, !cu), true, cu, nullptr, workspace, workspace_bytes, st, c));
  l.work = c.work;
  if (c.joined) {
    l.mix[0].incoming = c.part<float>(c.at.incoming[0]);
    l.mix[1].incoming = l.mix[2].incoming = c.part<float>(c.at.incoming[1]);
    Launch t = l;
    t.mixes = 2;
    t.mix[0] = Mix{nullptr, k, v, nullptr, 0, s.k_row, s.v_row, 0, s.dk, s.dv, 1, 1, 0, 0.f, 0.f, 1.f, 0,
                   nullptr, nullptr, nullptr, nullptr, nullptr, c.part<float>(c.at.totals[0])};
    t.mix[1].totals = c.part<float>(c.at.totals[1]);
    SLIM_TRY(run_mix<T>(t, c.tensor, st));
    Scan sc{c.work, log_decay, s.dk * s.dv, {}, 2};
    sc.side[0] = {t.mix[0].totals, state_in, c.part<float>(c.at.incoming[0]), nullptr, nullptr, 0};
    sc.side[1] = {t.mix[1].totals, g_in, c.part<float>(c.at.incoming[1]), nullptr, nullptr, 1};
    SLIM_TRY(finish(scan(sc, st), st));
  }
  return run_mix<T>(l, c.tensor, st);
}

template <typename T>
slim_status run_step(const void *q, const void *k, const void *v, const float *log_decay, float *state,
                     const int *slots, void *o, const slim_decay_shape *shape, float scale, cudaStream_t st) {
  NvtxRange range("slim_decay_step");
  SLIM_TRY(check_shape(shape));
  const slim_decay_shape &s = *shape;
  const int rows = s.tokens;
  if (!slots && s.places != rows) return SLIM_ERR_INVALID_ARG;
  if (rows == 0 || s.heads == 0) return SLIM_OK;
  if ((long long)rows * s.heads >= (1ll << 31)) return SLIM_ERR_UNSUPPORTED;
  if (!log_decay || (!state && s.places)) return SLIM_ERR_INVALID_ARG;
  const long long wide = (long long)s.heads * s.groups;
  SLIM_TRY(check_rows(q, sizeof(T), rows, s.q_row, wide * s.dk));
  SLIM_TRY(check_rows(k, sizeof(T), rows, s.k_row, (long long)s.heads * s.dk));
  SLIM_TRY(check_rows(v, sizeof(T), rows, s.v_row, (long long)s.heads * s.dv));
  SLIM_TRY(check_rows(o, sizeof(T), rows, s.o_row, wide * s.dv));
  if (o == q || o == k || o == v) return SLIM_ERR_INVALID_ARG;
  if (!aligned(log_decay, 4) || !aligned(slots, 4) || !aligned(state, 4)) return SLIM_ERR_UNSUPPORTED;
  return finish(step<T>(Step{q, k, v, o, s.q_row, s.k_row, s.v_row, s.o_row, log_decay, state, slots, rows, s.places,
                             s.heads, s.groups, s.dk, s.dv, scale},
                        st),
                st);
}

}  // namespace
}  // namespace decay
}  // namespace slim

using namespace slim::decay;

extern "C" {

size_t slim_decay_workspace_bytes(const slim_decay_shape *shape, int equal, int is_bwd) {
  if (check_shape(shape) != SLIM_OK || shape->seqs == 0 || shape->heads == 0) return 0;
  if (equal && shape->tokens % shape->seqs) return 0;
  const size_t bytes = layout(*shape, generic_cut(*shape, equal != 0), is_bwd != 0).bytes;
  return tc_shape(*shape) ? std::max(bytes, layout(*shape, tc_cut(*shape, equal != 0), is_bwd != 0).bytes) : bytes;
}

slim_status slim_decay_fwd(const void *q, const void *k, const void *v, const float *log_decay, const int *cu_seqlens,
                           const float *state_in, float *state_out, const int *slots, void *o,
                           const slim_decay_shape *shape, float scale, void *workspace, size_t workspace_bytes,
                           slim_stream_t stream) {
  return run_fwd<bf16>(q, k, v, log_decay, cu_seqlens, state_in, state_out, slots, o, shape, scale, workspace,
                       workspace_bytes, (cudaStream_t)stream);
}

slim_status slim_decay_fwd_f32(const float *q, const float *k, const float *v, const float *log_decay,
                               const int *cu_seqlens, const float *state_in, float *state_out, const int *slots,
                               float *o, const slim_decay_shape *shape, float scale, void *workspace,
                               size_t workspace_bytes, slim_stream_t stream) {
  return run_fwd<float>(q, k, v, log_decay, cu_seqlens, state_in, state_out, slots, o, shape, scale, workspace,
                        workspace_bytes, (cudaStream_t)stream);
}

slim_status slim_decay_bwd(const void *q, const void *k, const void *v, const float *log_decay, const int *cu_seqlens,
                           const void *d_o, const float *state_in, const float *g_in, float *g_out, void *dq, void *dk,
                           void *dv, const slim_decay_shape *shape, float scale, void *workspace,
                           size_t workspace_bytes, slim_stream_t stream) {
  return run_bwd<bf16>(q, k, v, log_decay, cu_seqlens, d_o, state_in, g_in, g_out, dq, dk, dv, shape, scale, workspace,
                       workspace_bytes, (cudaStream_t)stream);
}

slim_status slim_decay_bwd_f32(const float *q, const float *k, const float *v, const float *log_decay,
                               const int *cu_seqlens, const float *d_o, const float *state_in, const float *g_in,
                               float *g_out, float *dq, float *dk, float *dv, const slim_decay_shape *shape,
                               float scale, void *workspace, size_t workspace_bytes, slim_stream_t stream) {
  return run_bwd<float>(q, k, v, log_decay, cu_seqlens, d_o, state_in, g_in, g_out, dq, dk, dv, shape, scale, workspace,
                        workspace_bytes, (cudaStream_t)stream);
}

slim_status slim_decay_step(const void *q, const void *k, const void *v, const float *log_decay, float *state,
                            const int *slots, void *o, const slim_decay_shape *shape, float scale,
                            slim_stream_t stream) {
  return run_step<bf16>(q, k, v, log_decay, state, slots, o, shape, scale, (cudaStream_t)stream);
}

slim_status slim_decay_step_f32(const float *q, const float *k, const float *v, const float *log_decay, float *state,
                                const int *slots, float *o, const slim_decay_shape *shape, float scale,
                                slim_stream_t stream) {
  return run_step<float>(q, k, v, log_decay, state, slots, o, shape, scale, (cudaStream_t)stream);
}

}  // extern "C"
