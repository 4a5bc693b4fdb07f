"""AdamW over many tensors in one launch, its states in 32 bits or in 8.

Marshalling for ``slim_adamw``; the step runs in the library's CUDA kernel.

    opt = AdamW(weights, lr=1e-3, bits=8)
    ...
    opt.step(grads)                       # weights change in place
    layer.load(wqkv=weights[0], ...)      # and are packed again
"""
import ctypes

import torch

from . import binding, q8

_lib = binding.raw()
_vp, _i, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float


class _Tensor(ctypes.Structure):
    """slim_adamw_tensor."""
    _fields_ = [(n, _vp) for n in ("param", "grad", "m", "v", "m_scales", "v_scales")] + [("n", ctypes.c_longlong)]


class _Options(ctypes.Structure):
    """slim_adamw_options."""
    _fields_ = [(n, _f) for n in ("lr", "eps", "weight_decay")] + [("bits", _i)] \
        + [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("seed", ctypes.c_ulonglong), ("lr_device", _vp)]


for _fn in (_lib.slim_adamw, _lib.slim_adamw_f32):
    _fn.argtypes, _fn.restype = [ctypes.POINTER(_Tensor), _i, ctypes.POINTER(_Options), _vp, _vp], _i


def _dense(t, what):
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be contiguous CUDA fp32 tensors" % what)


def _fraction(b, what):
    if not 0 <= b < 1:
        raise ValueError("%s must be in [0, 1)" % what)


class AdamW:
    """params: contiguous fp32 CUDA tensors of one device, changed in place.

    ``m`` and ``v`` hold the moments, a tensor for each of params: fp32 of the
    same size, or with bits=8 a one-row :class:`q8.Q8`, where v's holds the
    root of the second moment.  They are made (zero) unless they are given.
    ``count``, int32 [2] on the device, holds the steps done.  lr is a number,
    or a CUDA fp32 tensor of one element that the step reads when it runs (so
    that a captured step can be replayed under another rate).  With bits=8,
    the same seed gives the same roundings."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, bits=32, seed=0, m=None, v=None,
                 count=0):
        self.params = list(params)
        if not self.params:
            raise ValueError("no params")
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32")
        _fraction(betas[0], "betas[0]")
        _fraction(betas[1], "betas[1]")
        if not eps >= 0:
            raise ValueError("eps must be at least 0")
        if not 0 <= seed < 1 << 64:
            raise ValueError("seed must be in [0, 2^64)")
        device = self.params[0].device
        self.lr, self.bits, self.device = lr, bits, device
        for p in self.params:
            _dense(p, "params")
            if p.device != device:
                raise ValueError("params must be on one device")
        self.m = [self._zeros(p) for p in self.params] if m is None else list(m)
        self.v = [self._zeros(p) for p in self.params] if v is None else list(v)
        if len(self.m) != len(self.params) or len(self.v) != len(self.params):
            raise ValueError("m and v must have a tensor for each of params")
        for p, a, b in zip(self.params, self.m, self.v):
            self._check_state(a, p)
            self._check_state(b, p)
        self._refuse_overlaps()
        self.count = torch.tensor([count, 0], dtype=torch.int32, device=device)
        self._options = _Options(0.0, eps, weight_decay, bits, betas[0], betas[1], seed, None)
        self._tensors = (_Tensor * len(self.params))()
        for t, p, a, b in zip(self._tensors, self.params, self.m, self.v):
            t.param, t.n = p.data_ptr(), p.numel()
            if bits == 8:
                t.m, t.m_scales, t.v, t.v_scales = (x.data_ptr() for s in (a, b) for x in s[:2])
            else:
                t.m, t.v = a.data_ptr(), b.data_ptr()

    def _zeros(self, p):
        if self.bits == 32:
            return torch.zeros_like(p)
        state = q8.empty(1, p.numel(), device=p.device)
        state.codes.view(torch.uint8).zero_()
        state.scales.fill_(127)
        return state

    def _check_state(self, s, p):
        if self.bits == 8:
            if not isinstance(s, q8.Q8):
                raise ValueError("a state in 8 bits must be a Q8 of one row")
            q8._mat(s, "a state", 1, 1, p.numel(), p.device)
        else:
            if isinstance(s, q8.Q8):
                raise ValueError("a state in 32 bits must be an fp32 tensor")
            _dense(s, "states")
            if s.numel() != p.numel() or s.device != p.device:
                raise ValueError("a state must have its parameter's size and device")

    def _refuse_overlaps(self):
        parts = [t for s in (self.params, self.m, self.v) for x in s for t in (x[:2] if isinstance(x, q8.Q8) else (x,))]
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in parts if t.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("params and states must not overlap")

    def step(self, grads):
        """One step.  grads: a contiguous tensor for each of params, all bf16 or
        all fp32, or None for a tensor that stays as it is."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError("grads must have a tensor (or None) for each of params")
        dtype = None
        for t, p, g in zip(self._tensors, self.params, grads):
            if g is None:
                t.grad = None
                continue
            if dtype is None:
                dtype = g.dtype
                if dtype not in (torch.bfloat16, torch.float32):
                    raise ValueError("grads must be bf16 or fp32")
            if g.dtype != dtype or g.shape != p.shape or g.device != p.device or not g.is_contiguous():
                raise ValueError("grads must be contiguous, of one dtype, and have the params' shapes and device")
            t.grad = g.data_ptr()
        o = self._options
        if isinstance(self.lr, torch.Tensor):
            if self.lr.dtype != torch.float32 or self.lr.numel() != 1 or self.lr.device != self.device:
                raise ValueError("lr must be a number or a CUDA fp32 tensor of one element")
            o.lr_device = self.lr.data_ptr()
        else:
            o.lr, o.lr_device = self.lr, None
        name = "slim_adamw" if dtype == torch.bfloat16 else "slim_adamw_f32"
        code = getattr(_lib, name)(self._tensors, len(self.params), ctypes.byref(o), self.count.data_ptr(),
                                   self._stream(self.device))
        if code:
            raise binding.SlimError(code, name)

    @staticmethod
    def _stream(device):
        if device.index != torch._C._cuda_getDevice():
            binding.check_device(device)
        return torch._C._cuda_getCurrentRawStream(device.index)
