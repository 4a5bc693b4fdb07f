"""Group norm of each row's heads, with a gate, and its gradients.

Marshalling for the ``slim_group_norm*`` entry points of ``libslim_attn.so``;
every computation runs in the library's CUDA kernels.  Between an attention
and its output projection,

    y = ((x - mean) rstd gamma + beta) silu(gate)

with mean and rstd over each group (head) of each row.
"""
import ctypes

import torch

from . import binding

_lib = binding.raw()
_vp, _i, _sz, _f, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_longlong

_functions = {}
for _name, _args in (("slim_group_norm", [_vp] * 4 + [_ll, _f, _vp] + [_i] * 3 + [_vp]),
                     ("slim_group_norm_bwd", [_vp] * 5 + [_ll, _f] + [_vp] * 2 + [_ll] + [_vp] * 3 + [_sz] + [_i] * 3 + [_vp])):
    for _dtype, _suffix in ((torch.bfloat16, ""), (torch.float32, "_f32")):
        _fn = getattr(_lib, _name + _suffix)
        _fn.argtypes, _fn.restype = _args, _i
        _functions[_name, _dtype] = (_fn, _name + _suffix)
_lib.slim_group_norm_bwd_workspace_bytes.argtypes = [_i] * 3
_lib.slim_group_norm_bwd_workspace_bytes.restype = _sz


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


def _rows(t, what, like=None):
    if t.dtype not in (torch.bfloat16, torch.float32) or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA bf16 or fp32 [rows, cols] tensor" % what)
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError("%s must have the other rows' shape, dtype and device" % what)


def _gate(t, what, like):
    """Elements from row to row of [rows, cols] whose rows are dense and may lie apart."""
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError("%s must have the other rows' shape, dtype and device" % what)
    s, (rows, cols) = t.stride(), t.shape
    if (cols > 1 and s[1] != 1) or (rows > 1 and s[0] < cols):
        raise ValueError("the rows of %s must be dense (strides %s)" % (what, list(s)))
    return s[0] if rows > 1 else cols


def _check(x, gamma, beta, groups, gate):
    _rows(x, "x")
    rows, cols = x.shape
    for t, what in ((gamma, "gamma"), (beta, "beta")):
        if t.shape != (cols,) or t.dtype != torch.float32 or t.device != x.device or not t.is_contiguous():
            raise ValueError("%s must be a contiguous fp32 [%d] tensor on the rows' device" % (what, cols))
    if groups < 1 or cols % groups:
        raise ValueError("%d columns are not %d groups" % (cols, groups))
    return rows, cols, 0 if gate is None else _gate(gate, "gate", x)


def group_norm(x, gamma, beta, groups, gate=None, eps=1e-5, out=None):
    """y [rows, cols] in x's dtype: the norm of each row's ``groups`` groups of
    consecutive columns, times gamma plus beta, times silu(gate).  The gate's
    rows may lie apart (a part of a projection's rows)."""
    rows, cols, gate_row = _check(x, gamma, beta, groups, gate)
    if out is None:
        out = torch.empty_like(x)
    else:
        _rows(out, "out", x)
    _call("slim_group_norm", x.dtype, x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), _ptr(gate), gate_row, eps, out.data_ptr(),
          rows, cols, groups, _stream(x.device))
    return out


def group_norm_bwd(dy, x, gamma, beta, groups, gate=None, eps=1e-5, dgate=None):
    """(dx, dgate, dgamma, dbeta) of :func:`group_norm`; dgate is None without a gate,
    and else may be a buffer whose rows lie apart."""
    rows, cols, gate_row = _check(x, gamma, beta, groups, gate)
    _rows(dy, "dy", x)
    dx = torch.empty_like(x)
    if gate is None:
        dgate, dgate_row = None, 0
    else:
        dgate = torch.empty_like(x) if dgate is None else dgate
        dgate_row = _gate(dgate, "dgate", x)
    sums = torch.empty((2, cols), dtype=torch.float32, device=x.device)
    nbytes = _lib.slim_group_norm_bwd_workspace_bytes(rows, cols, groups)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _call("slim_group_norm_bwd", x.dtype, dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), _ptr(gate),
          gate_row, eps, dx.data_ptr(), _ptr(dgate), dgate_row, sums[0].data_ptr(), sums[1].data_ptr(), ws.data_ptr(), nbytes, rows, cols,
          groups, _stream(x.device))
    return dx, dgate, sums[0], sums[1]
