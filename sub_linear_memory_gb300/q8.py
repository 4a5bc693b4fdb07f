"""The rest of a layer in 8 bits: norm, projections, activation, checkpoints.

Marshalling for the ``slim_q8_*`` entry points of ``libslim_attn.so`` (argument
checks, output and workspace allocations, the current torch stream); every
computation runs in the library's CUDA kernels.

An 8-bit matrix is a :class:`Q8`: e4m3 codes, padded with zeros to whole blocks
of 128 columns, and one power-of-two scale byte for each row (each 128 rows of
a packed weight) and 128 columns: value = code * 2^(scale - 127).  One training
pass through a projection with its norm and activation:

    h, y, rstd, h8 = rms_norm(x, gamma, res=r, checkpoint=True)
    z = matmul(y, w)                          # w, wt = pack_weight(weight)
    a, z8 = gelu(z)                           # kept: y, h8, z8 (8 bits), rstd
    ...
    dz, dz8 = gelu_bwd(da, z8, quantized=True)
    dw = wgrad(dz, y)
    dh, dgamma = rms_norm_bwd(matmul(dz8, wt), h8, rstd, gamma, dres=dh_after)
"""
import ctypes
from typing import NamedTuple

import torch

from . import binding

_lib = binding.raw()
_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float

BLOCK = 128

_SIGNATURES = {
    "slim_q8_quantize": [_vp] * 3 + [_i] * 2 + [_vp],
    "slim_q8_dequantize": [_vp] * 3 + [_i] * 3 + [_vp],
    "slim_q8_pack_weight": [_vp] * 5 + [_i] * 2 + [_vp],
    "slim_q8_rms_norm": [_vp] * 3 + [_f] + [_vp] * 6 + [_i] * 2 + [_vp],
    "slim_q8_rms_norm_bwd": [_vp] * 10 + [_sz] + [_i] * 2 + [_vp],
    "slim_q8_gelu": [_vp] * 5 + [_i] * 2 + [_vp],
    "slim_q8_gelu_bwd": [_vp] * 6 + [_i] * 2 + [_vp],
    "slim_q8_matmul": [_vp] * 5 + [_i] * 3 + [_vp],
}
for _name, _args in _SIGNATURES.items():
    for _fn in (getattr(_lib, _name), getattr(_lib, _name + "_f32")):
        _fn.argtypes, _fn.restype = _args, _i
_lib.slim_q8_wgrad.argtypes = [_vp] * 4 + [_i, _vp, _sz] + [_i] * 3 + [_vp]
_lib.slim_q8_wgrad.restype = _i
_lib.slim_q8_codes_bytes.argtypes = [_i] * 2
_lib.slim_q8_scales_bytes.argtypes = [_i] * 3
_lib.slim_q8_rms_norm_bwd_workspace_bytes.argtypes = [_i] * 2
_lib.slim_q8_wgrad_workspace_bytes.argtypes = [_i] * 3
for _name in ("codes_bytes", "scales_bytes", "rms_norm_bwd_workspace_bytes", "wgrad_workspace_bytes"):
    getattr(_lib, "slim_q8_" + _name).restype = _sz


class Q8(NamedTuple):
    """An 8-bit matrix of ``cols`` columns.  codes: torch.float8_e4m3fn
    [rows, 128 * blocks]; scales: torch.uint8 [rows (or ceil(rows / 128)),
    4 * ceil(blocks / 4)]; block_rows: 1, or 128 for a packed weight.  Codes
    made elsewhere: NaN codes stand only under scale 255 (``wgrad`` takes others
    for 480)."""

    codes: torch.Tensor
    scales: torch.Tensor
    cols: int
    block_rows: int = 1

    @property
    def rows(self):
        return self.codes.shape[0]


def empty(rows, cols, block_rows=1, device=None):
    """An uninitialised Q8 of the given size."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    nb = -(-cols // BLOCK)
    return Q8(torch.empty((rows, nb * BLOCK), dtype=torch.float8_e4m3fn, device=dev),
              torch.empty((-(-rows // block_rows), -(-nb // 4) * 4), dtype=torch.uint8, device=dev), cols, block_rows)


def _stream(device):
    # the device's number and the stream's handle alone: torch.cuda's functions around them cost
    # more than a small kernel's launch
    if device.index != torch._C._cuda_getDevice():
        binding.check_device(device)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _ptr(t):
    return None if t is None else t.data_ptr()


_TYPES = (torch.bfloat16, torch.float32)


def _rows(t, what, like=None):
    """A dense CUDA bf16 or fp32 matrix; like: one of the same shape, type and device."""
    if t.dtype not in _TYPES or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA bf16 or fp32 [rows, cols] tensor" % what)
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError("%s must have the other rows' shape, dtype and device" % what)


def _vector(t, n, device, what):
    if t.shape != (n,) or t.dtype != torch.float32 or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous fp32 [%d] tensor on the rows' device" % (what, n))


def _mat(q, what, block_rows=1, rows=None, cols=None, device=None):
    nb = -(-q.cols // BLOCK)
    r = q.codes.shape[0]
    if q.block_rows != block_rows or q.codes.dtype != torch.float8_e4m3fn or q.scales.dtype != torch.uint8 \
            or q.codes.shape != (r, nb * BLOCK) or q.scales.shape != (-(-r // block_rows), -(-nb // 4) * 4) \
            or not q.codes.is_contiguous() or not q.scales.is_contiguous() or q.scales.device != q.codes.device \
            or not q.codes.is_cuda:
        raise ValueError("%s must be a Q8 with one scale for each %d row(s) and 128 columns" % (what, block_rows))
    if (rows is not None and r != rows) or (cols is not None and q.cols != cols) \
            or (device is not None and q.codes.device != device):
        raise ValueError("%s does not have the other arguments' sizes and device" % what)


_functions = {(_name, _dtype): (getattr(_lib, _name + _suffix), _name + _suffix)
              for _name in _SIGNATURES for _dtype, _suffix in ((torch.bfloat16, ""), (torch.float32, "_f32"))}


def _call(name, dtype, *args):
    fn, what = _functions[name, dtype]
    code = fn(*args)
    if code:
        raise binding.SlimError(code, what)


def quantize(x, out=None):
    """The 8 bits of x [rows, cols] (bf16 or fp32)."""
    _rows(x, "x")
    rows, cols = x.shape
    if out is None:
        out = empty(rows, cols, device=x.device)
    else:
        _mat(out, "out", 1, rows, cols, x.device)
    _call("slim_q8_quantize", x.dtype, x.data_ptr(), out.codes.data_ptr(), out.scales.data_ptr(), rows, cols, _stream(x.device))
    return out


def dequantize(q, dtype=torch.bfloat16, out=None):
    """The values of a Q8 (rows or packed weight) as bf16, exactly, or fp32."""
    _mat(q, "q", q.block_rows if q.block_rows in (1, BLOCK) else 1)
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    elif out.shape != (q.rows, q.cols) or out.device != q.codes.device:
        raise ValueError("out must be [rows, cols] on q's device")
    _rows(out, "out")
    _call("slim_q8_dequantize", out.dtype, q.codes.data_ptr(), q.scales.data_ptr(), out.data_ptr(), q.rows, q.cols,
          q.block_rows, _stream(out.device))
    return out


def pack_weight(w, transpose=True):
    """The packed weight of w [n, k] (bf16 or fp32) and, for the data gradient,
    that of its transpose (None without ``transpose``): the same values."""
    _rows(w, "w")
    n, k = w.shape
    q = empty(n, k, BLOCK, w.device)
    qt = empty(k, n, BLOCK, w.device) if transpose else None
    _call("slim_q8_pack_weight", w.dtype, w.data_ptr(), q.codes.data_ptr(), q.scales.data_ptr(),
          _ptr(qt and qt.codes), _ptr(qt and qt.scales), n, k, _stream(w.device))
    return q, qt


def rms_norm(x, gamma, res=None, eps=1e-5, checkpoint=False):
    """h = x + res, rstd = (mean h^2 + eps)^(-1/2), y = 8 bits of h rstd gamma.

    Returns (h, y, rstd, h8): h in x's dtype (x itself without ``res``), y a
    Q8, rstd fp32 [rows], and with ``checkpoint`` the 8 bits of h for the
    backward (else None)."""
    _rows(x, "x")
    rows, cols = x.shape
    _vector(gamma, cols, x.device, "gamma")
    h = x
    if res is not None:
        _rows(res, "res", x)
        h = torch.empty_like(x)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    y = empty(rows, cols, device=x.device)
    h8 = empty(rows, cols, device=x.device) if checkpoint else None
    _call("slim_q8_rms_norm", x.dtype, x.data_ptr(), _ptr(res), gamma.data_ptr(), eps,
          None if res is None else h.data_ptr(), rstd.data_ptr(), y.codes.data_ptr(), y.scales.data_ptr(),
          _ptr(h8 and h8.codes), _ptr(h8 and h8.scales), rows, cols, _stream(x.device))
    return h, y, rstd, h8


def rms_norm_bwd(dy, kept, rstd, gamma, dres=None):
    """(dh, dgamma) of :func:`rms_norm`: dy the gradient at the norm's output,
    ``kept`` h in full or its checkpoint h8, ``dres`` the gradient that reaches
    h by other ways, added to dh."""
    _rows(dy, "dy")
    rows, cols = dy.shape
    _vector(gamma, cols, dy.device, "gamma")
    _vector(rstd, rows, dy.device, "rstd")
    h = hc = hs = None
    if isinstance(kept, Q8):
        _mat(kept, "kept", 1, rows, cols, dy.device)
        hc, hs = kept.codes, kept.scales
    else:
        _rows(kept, "kept", dy)
        h = kept
    if dres is not None:
        _rows(dres, "dres", dy)
    dh = torch.empty_like(dy)
    dgamma = torch.empty(cols, dtype=torch.float32, device=dy.device)
    nbytes = _lib.slim_q8_rms_norm_bwd_workspace_bytes(rows, cols)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)
    _call("slim_q8_rms_norm_bwd", dy.dtype, dy.data_ptr(), _ptr(h), _ptr(hc), _ptr(hs), rstd.data_ptr(),
          gamma.data_ptr(), _ptr(dres), dh.data_ptr(), dgamma.data_ptr(), ws.data_ptr(), nbytes, rows, cols,
          _stream(dy.device))
    return dh, dgamma


def gelu(z, checkpoint=True):
    """(a, z8): the 8 bits of GeLU(z) and, with ``checkpoint``, of z itself
    for the backward (else None)."""
    _rows(z, "z")
    rows, cols = z.shape
    a = empty(rows, cols, device=z.device)
    z8 = empty(rows, cols, device=z.device) if checkpoint else None
    _call("slim_q8_gelu", z.dtype, z.data_ptr(), a.codes.data_ptr(), a.scales.data_ptr(), _ptr(z8 and z8.codes),
          _ptr(z8 and z8.scales), rows, cols, _stream(z.device))
    return a, z8


def gelu_bwd(da, z8, quantized=False):
    """dz = da GeLU'(z) at the checkpointed z; with ``quantized`` (dz, dz8),
    dz8 = quantize(dz) from the same pass (the data gradient's operand)."""
    _rows(da, "da")
    rows, cols = da.shape
    _mat(z8, "z8", 1, rows, cols, da.device)
    dz = torch.empty_like(da)
    dz8 = empty(rows, cols, device=da.device) if quantized else None
    _call("slim_q8_gelu_bwd", da.dtype, da.data_ptr(), z8.codes.data_ptr(), z8.scales.data_ptr(), dz.data_ptr(),
          _ptr(dz8 and dz8.codes), _ptr(dz8 and dz8.scales), rows, cols, _stream(da.device))
    return (dz, dz8) if quantized else dz


def matmul(a, w, dtype=torch.bfloat16, out=None):
    """a . w^T: a a Q8 of rows [rows, k], w a packed weight [n, k]; [rows, n]
    in bf16 or fp32."""
    _mat(a, "a")
    _mat(w, "w", BLOCK, None, a.cols, a.codes.device)
    if out is None:
        out = torch.empty((a.rows, w.rows), dtype=dtype, device=a.codes.device)
    elif out.shape != (a.rows, w.rows) or out.device != a.codes.device:
        raise ValueError("out must be [rows, n] on a's device")
    _rows(out, "out")
    _call("slim_q8_matmul", out.dtype, a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(),
          w.scales.data_ptr(), out.data_ptr(), a.rows, w.rows, a.cols, _stream(out.device))
    return out


def wgrad(dy, x, dw=None, accumulate=False):
    """dw [n, k] (fp32) = dy^T . x for dy [rows, n] (bf16) and the 8-bit rows x
    [rows, k]; with ``accumulate`` added to ``dw``."""
    _rows(dy, "dy")
    if dy.dtype != torch.bfloat16:
        raise ValueError("dy must be bf16")
    rows, n = dy.shape
    _mat(x, "x", 1, rows, None, dy.device)
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        dw = torch.empty((n, x.cols), dtype=torch.float32, device=dy.device)
    if dw.shape != (n, x.cols) or dw.dtype != torch.float32 or dw.device != dy.device or not dw.is_contiguous():
        raise ValueError("dw must be a contiguous fp32 [n, k] tensor on dy's device")
    nbytes = _lib.slim_q8_wgrad_workspace_bytes(rows, n, x.cols)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)
    code = _lib.slim_q8_wgrad(dy.data_ptr(), x.codes.data_ptr(), x.scales.data_ptr(), dw.data_ptr(),
                              1 if accumulate else 0, ws.data_ptr(), nbytes, rows, n, x.cols, _stream(dy.device))
    if code:
        raise binding.SlimError(code, "slim_q8_wgrad")
    return dw
