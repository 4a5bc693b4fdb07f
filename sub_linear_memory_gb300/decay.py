"""Linear attention with a decay for each head, over packed sequences.

Marshalling for the ``slim_decay_*`` entry points of ``libslim_attn.so``
(argument checks, output and workspace allocations, the current torch
stream); every computation runs in the library's CUDA kernels.

For key-value head h with decay lambda = exp(log_decay[h]) and each query head
that shares it,

    S_t = lambda S_(t-1) + k_t v_t^T,    o_t = scale q_t^T S_t.

A prompt (or a training batch) goes through :func:`attn`, its gradients come
from :func:`attn_bwd`, and one more token of each sequence through
:func:`step`.  Rows are tokens, q [T, Hq, dk], k [T, Hk, dk], v [T, Hk, dv]
with Hq a multiple of Hk, in bf16 or fp32; rows may lie apart (parts of one
projection's rows), the heads of a row may not.  Sequences are rows
[cu_seqlens[i], cu_seqlens[i + 1]), or without ``cu_seqlens`` equal parts of
the T rows.  States are fp32 [places, Hk, dk, dv].
"""
import ctypes

import torch

from . import binding

_lib = binding.raw()
_vp, _i, _sz, _f, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_longlong


class Shape(ctypes.Structure):
    """slim_decay_shape."""
    _fields_ = [(n, _i) for n in ("tokens", "seqs", "heads", "groups", "dk", "dv", "places")] \
        + [(n, _ll) for n in ("q_row", "k_row", "v_row", "o_row", "dq_row", "dk_row", "dv_row")]


_shape = ctypes.POINTER(Shape)
_functions = {}
for _name, _args in (("slim_decay_fwd", [_vp] * 9 + [_shape, _f, _vp, _sz, _vp]),
                     ("slim_decay_bwd", [_vp] * 12 + [_shape, _f, _vp, _sz, _vp]),
                     ("slim_decay_step", [_vp] * 7 + [_shape, _f, _vp])):
    for _dtype, _suffix in ((torch.bfloat16, ""), (torch.float32, "_f32")):
        _fn = getattr(_lib, _name + _suffix)
        _fn.argtypes, _fn.restype = _args, _i
        _functions[_name, _dtype] = (_fn, _name + _suffix)
_lib.slim_decay_workspace_bytes.argtypes = [_shape, _i, _i]
_lib.slim_decay_workspace_bytes.restype = _sz


def _stream(device):
    if device.index != torch._C._cuda_getDevice():
        binding.check_device(device)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _call(name, dtype, *args):
    fn, what = _functions[name, dtype]
    code = fn(*args)
    if code:
        raise binding.SlimError(code, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _row(t, what, shape, like):
    """Elements from row to row of [rows, heads, width], whose heads lie side by side."""
    if t.shape != shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError("%s must be %s in q's dtype on its device; got %s %s" % (what, list(shape), list(t.shape), t.dtype))
    rows, heads, width = shape
    s = t.stride()
    if (width > 1 and s[2] != 1) or (heads > 1 and s[1] != width) or (rows > 1 and s[0] < heads * width):
        raise ValueError("the heads of a row of %s must lie side by side (strides %s)" % (what, list(s)))
    return max(s[0], heads * width) if rows > 1 else heads * width


def _check(q, k, v, log_decay):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float32) or not q.is_cuda:
        raise ValueError("q, k, v must be CUDA bf16 or fp32 [rows, heads, width] tensors")
    rows, hq, dk = q.shape
    hk, dv = v.shape[1:]
    if hk < 1 or hq < 1 or hq % hk or dk < 1 or dv < 1:
        raise ValueError("the query heads must be a multiple of the key-value heads")
    if log_decay.shape != (hk,) or log_decay.dtype != torch.float32 or log_decay.device != q.device \
            or not log_decay.is_contiguous():
        raise ValueError("log_decay must be a contiguous fp32 [%d] tensor on q's device" % hk)
    return Shape(rows, 0, hk, hq // hk, dk, dv, 0, _row(q, "q", (rows, hq, dk), q), _row(k, "k", (rows, hk, dk), q),
                 _row(v, "v", (rows, hk, dv), q))


def _seqs(shape, cu_seqlens, seqs, device):
    if cu_seqlens is None:
        if seqs < 1 or shape.tokens % seqs:
            raise ValueError("%d rows are not %d sequences of one length" % (shape.tokens, seqs))
        shape.seqs = seqs
    else:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.dtype != torch.int32 \
                or cu_seqlens.device != device or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous int32 [sequences + 1] tensor on q's device")
        shape.seqs = cu_seqlens.shape[0] - 1


def _states(shape, device, places, **states):
    """Checks states; the places are the sequences without slots."""
    for what, t in states.items():
        if t is None:
            continue
        if t.dim() != 4 or t.shape[1:] != (shape.heads, shape.dk, shape.dv) or t.dtype != torch.float32 \
                or t.device != device or not t.is_contiguous() or (places is not None and t.shape[0] != places):
            raise ValueError("%s must be a contiguous fp32 [places, heads, dk, dv] tensor on q's device" % what)
        places = t.shape[0]
    shape.places = places or 0


def _slots(slots, n, device):
    if slots is not None and (slots.shape != (n,) or slots.dtype != torch.int32 or slots.device != device
                              or not slots.is_contiguous()):
        raise ValueError("slots must be a contiguous int32 [%d] tensor on q's device" % n)


# What calls of one layout share: the checked slim_decay_shape, the output's shape, and the workspace's bytes.
# The checks and queries cost as much as a short call's kernels.
_known = {}


def _layout(*tensors):
    return tuple(None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors)


def _remember(key, plan):
    if len(_known) >= 4096:
        _known.clear()
    _known[key] = plan
    return plan


def _bytes(shape, cu_seqlens, bwd):
    return _lib.slim_decay_workspace_bytes(ctypes.byref(shape), cu_seqlens is None, bwd)


def _plan_attn(q, k, v, log_decay, cu_seqlens, state_in, state_out, slots, seqs, out):
    key = (0, seqs) + _layout(q, k, v, log_decay, cu_seqlens, state_in, state_out, slots, out)
    plan = _known.get(key)
    if plan is not None:
        return plan
    shape = _check(q, k, v, log_decay)
    _seqs(shape, cu_seqlens, seqs, q.device)
    _slots(slots, shape.seqs, q.device)
    _states(shape, q.device, None if slots is not None else shape.seqs, state_in=state_in, state_out=state_out)
    o = (q.shape[0], q.shape[1], shape.dv)
    shape.o_row = q.shape[1] * shape.dv if out is None else _row(out, "out", o, q)
    return _remember(key, (shape, o, _bytes(shape, cu_seqlens, 0)))


def attn(q, k, v, log_decay, cu_seqlens=None, scale=1.0, state_in=None, state_out=None, slots=None, seqs=1, out=None):
    """o [T, Hq, dv].

    state_in, state_out (one tensor, or two of one shape, or None): the states
    before the first rows and behind the last.  slots: int32 [sequences], each
    sequence's place in the states (without it, sequence i has place i); one
    that names no place, or another's, starts from zero and leaves no state.
    Rows outside every sequence are not written."""
    device = q.device
    stream = _stream(device)
    shape, o, nbytes = _plan_attn(q, k, v, log_decay, cu_seqlens, state_in, state_out, slots, seqs, out)
    if out is None:
        out = torch.empty(o, dtype=q.dtype, device=device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _call("slim_decay_fwd", q.dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(cu_seqlens),
          _ptr(state_in), _ptr(state_out), _ptr(slots), out.data_ptr(), ctypes.byref(shape), scale, ws.data_ptr(), nbytes,
          stream)
    return out


def _plan_bwd(q, k, v, log_decay, do, cu_seqlens, state_in, g_in, g_out, seqs, out):
    key = (1, seqs) + _layout(q, k, v, log_decay, do, cu_seqlens, state_in, g_in, g_out, *(out or ()))
    plan = _known.get(key)
    if plan is not None:
        return plan
    shape = _check(q, k, v, log_decay)
    _seqs(shape, cu_seqlens, seqs, q.device)
    _states(shape, q.device, shape.seqs, state_in=state_in, g_in=g_in, g_out=g_out)
    shape.o_row = _row(do, "do", (q.shape[0], q.shape[1], shape.dv), q)
    dq, dk, dv = out if out is not None else (None, None, None)
    dense = lambda t: t.shape[1] * t.shape[2]
    shape.dq_row = dense(q) if dq is None else _row(dq, "dq", q.shape, q)
    shape.dk_row = dense(k) if dk is None else _row(dk, "dk", k.shape, q)
    shape.dv_row = dense(v) if dv is None else _row(dv, "dv", v.shape, q)
    return _remember(key, (shape, _bytes(shape, cu_seqlens, 1)))


def attn_bwd(q, k, v, log_decay, do, cu_seqlens=None, scale=1.0, state_in=None, g_in=None, g_out=None, seqs=1, out=None):
    """(dq, dk, dv) of :func:`attn`: do is the gradient of o, g_in (or None)
    that of the states behind the last rows; g_out (or None) receives that of
    state_in.  out: buffers for the three, whose rows may lie apart."""
    device = q.device
    stream = _stream(device)
    shape, nbytes = _plan_bwd(q, k, v, log_decay, do, cu_seqlens, state_in, g_in, g_out, seqs, out)
    dq, dk, dv = out if out is not None else (torch.empty(t.shape, dtype=q.dtype, device=device) for t in (q, k, v))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _call("slim_decay_bwd", q.dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(cu_seqlens),
          do.data_ptr(), _ptr(state_in), _ptr(g_in), _ptr(g_out), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
          ctypes.byref(shape), scale, ws.data_ptr(), nbytes, stream)
    return dq, dk, dv


def _plan_step(q, k, v, log_decay, state, slots, out):
    key = (2,) + _layout(q, k, v, log_decay, state, slots, out)
    plan = _known.get(key)
    if plan is not None:
        return plan
    shape = _check(q, k, v, log_decay)
    _slots(slots, shape.tokens, q.device)
    _states(shape, q.device, None if slots is not None else shape.tokens, state=state)
    o = (q.shape[0], q.shape[1], shape.dv)
    shape.o_row = q.shape[1] * shape.dv if out is None else _row(out, "out", o, q)
    return _remember(key, (shape, o))


def step(q, k, v, log_decay, state, slots=None, scale=1.0, out=None):
    """One token of each sequence: q [B, Hq, dk], k [B, Hk, dk], v [B, Hk, dv]
    -> o [B, Hq, dv]; ``state`` is advanced in place.  slots: int32 [B], each
    row's place in it (without it, row i has place i); a row that names no
    place, or an earlier row's, gets zeros."""
    device = q.device
    stream = _stream(device)
    shape, o = _plan_step(q, k, v, log_decay, state, slots, out)
    if out is None:
        out = torch.empty(o, dtype=q.dtype, device=device)
    _call("slim_decay_step", q.dtype, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), state.data_ptr(),
          _ptr(slots), out.data_ptr(), ctypes.byref(shape), scale, stream)
    return out
