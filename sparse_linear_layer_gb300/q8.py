"""8-bit activations: matrices of one byte per element with fp32 scales, and
the calls that write and read them (include/snk.h has the definitions).

    kept = pack(x, format="int8", group=128)         # a checkpoint of x
    x2 = unpack(kept)                                # its values
    q, total, rstd = rmsnorm(x, gain, residual=r)    # norm of x + r in 8 bits
    dx, dgain = rmsnorm_backward(dy, total, rstd, gain, dtotal=dr)
    a, kept = gelu(h, keep=True)                     # gelu(h) and h in 8 bits
    dh = gelu_backward(da, kept)

binding.SparseLinear.forward_q8 and backward_weight_q8 take such a matrix as X.
Leading dimensions are rows: a tensor [..., cols] is a matrix of its last
dimension.  Tensors are CUDA tensors, contiguous, float32 / float16 / bfloat16
for activations and float32 for gains and statistics; anything else raises
ValueError.  The arithmetic is libsnk's; nothing falls back to torch.
"""
from __future__ import annotations

import torch

from . import binding

_DTYPES = {torch.float32: binding.SNK_F32, torch.float16: binding.SNK_F16,
           torch.bfloat16: binding.SNK_BF16}
_FORMATS = {"int8": (binding.SNK_Q8_INT8, torch.int8),
            "e4m3": (binding.SNK_Q8_E4M3, torch.float8_e4m3fn)}
_GROUPS = (0, 32, 64, 128, 256)
_F32 = torch.float32
_empty = torch.empty
_lib = None


def _call(name: str, *args):
    """A library call with plain arguments.  (The checks are the caller's: a
    decoding step spends more time in the wrappers than in the kernels, so they
    read each property once.)"""
    global _lib
    if _lib is None:
        _lib = binding.lib()
    status = getattr(_lib, name)(*args)
    if status:
        raise binding.SnkError(status, name)


def _on(stream, device):
    return binding.current_stream(device.index) if stream is None else binding._stream(stream)


def _matrix(t):
    """(type, rows, cols, device) of a contiguous CUDA tensor [..., cols]."""
    shape = t.shape
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"float32, float16 or bfloat16 is needed: got {t.dtype}")
    if not t.is_cuda or not shape or shape[-1] < 1 or not t.is_contiguous():
        raise ValueError(f"a contiguous CUDA tensor [..., cols] with cols >= 1 is needed: got {t.device} "
                         f"{tuple(shape)}, strides {t.stride()}")
    cols = shape[-1]
    return d, t.numel() // cols, cols, t.device


def _like(t, like, name):
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} is contiguous {tuple(like.shape)} {like.dtype} on {like.device}: got "
                         f"{tuple(t.shape)} {t.dtype} {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _f32(t, n, device, name):
    if t.dtype != _F32 or t.numel() != n or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} is contiguous float32 with {n} elements on {device}: got {t.dtype} "
                         f"{tuple(t.shape)} {t.device}")
    return t.data_ptr()


class Q8Tensor:
    """codes (int8, or float8_e4m3fn) [..., cols] and scales float32 [...,
    ceil(cols / group)] (group 0: [..., 1]); it stands for scale * code."""

    __slots__ = ("codes", "scales", "group", "format_id", "rows", "cols")

    def __init__(self, codes, scales, group: int):
        if group not in _GROUPS:
            raise ValueError(f"group is one of {_GROUPS}: got {group}")
        if codes.dtype == torch.int8:
            self.format_id = binding.SNK_Q8_INT8
        elif codes.dtype == torch.float8_e4m3fn:
            self.format_id = binding.SNK_Q8_E4M3
        else:
            raise ValueError(f"codes are int8 or float8_e4m3fn: got {codes.dtype}")
        if not codes.is_cuda or codes.dim() < 1 or codes.shape[-1] < 1 or not codes.is_contiguous():
            raise ValueError(f"codes are a contiguous CUDA tensor [..., cols] with cols >= 1: got {codes.device} "
                             f"{tuple(codes.shape)}, strides {codes.stride()}")
        self.cols = codes.shape[-1]
        self.rows = codes.numel() // self.cols
        _f32(scales, self.rows * (-(-self.cols // group) if group else 1), codes.device, "scales")
        self.codes, self.scales, self.group = codes, scales, group

    @property
    def format(self) -> str:
        return "int8" if self.format_id == binding.SNK_Q8_INT8 else "e4m3"

    @property
    def shape(self):
        return self.codes.shape

    def dequantize(self, dtype=torch.float32):
        return unpack(self, dtype)


def _new(shape, rows, cols, device, format, group):
    """A Q8Tensor to be written."""
    f = _FORMATS.get(format)
    if f is None or group not in _GROUPS:
        raise ValueError(f"format is one of {tuple(_FORMATS)} and group one of {_GROUPS}: got {format!r}, {group}")
    q = Q8Tensor.__new__(Q8Tensor)
    q.format_id = f[0]
    q.rows, q.cols, q.group = rows, cols, group
    q.codes = _empty(shape, dtype=f[1], device=device)
    n = -(-cols // group) if group else 1
    q.scales = _empty((rows, n) if len(shape) == 2 else (*shape[:-1], n), dtype=_F32, device=device)
    return q


def pack(x, format: str = "int8", group: int = 0, stream=None) -> Q8Tensor:
    """x in 8 bits."""
    d, rows, cols, device = _matrix(x)
    q = _new(x.shape, rows, cols, device, format, group)
    _call("snk_q8_pack", x.data_ptr(), d, rows, cols, q.format_id, group, q.codes.data_ptr(), q.scales.data_ptr(),
          _on(stream, device))
    return q


def unpack(q: Q8Tensor, dtype=torch.float32, stream=None):
    """scale * code, rounded to dtype."""
    d = _DTYPES.get(dtype)
    if d is None:
        raise ValueError(f"float32, float16 or bfloat16 is needed: got {dtype}")
    codes = q.codes
    x = _empty(codes.shape, dtype=dtype, device=codes.device)
    _call("snk_q8_unpack", codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, q.format_id, q.group, x.data_ptr(),
          d, _on(stream, codes.device))
    return x


def gelu(x, format: str = "int8", group: int = 0, keep: bool = False, stream=None):
    """x Phi(x) in 8 bits; with keep, also x itself in 8 bits, for
    gelu_backward: (gelu(x), x)."""
    d, rows, cols, device = _matrix(x)
    q = _new(x.shape, rows, cols, device, format, group)
    if not keep:
        _call("snk_gelu_q8", x.data_ptr(), d, rows, cols, q.format_id, group, q.codes.data_ptr(), q.scales.data_ptr(),
              None, None, _on(stream, device))
        return q
    kept = _new(x.shape, rows, cols, device, format, group)
    _call("snk_gelu_q8", x.data_ptr(), d, rows, cols, q.format_id, group, q.codes.data_ptr(), q.scales.data_ptr(),
          kept.codes.data_ptr(), kept.scales.data_ptr(), _on(stream, device))
    return q, kept


def gelu_backward(da, kept: Q8Tensor, out=None, stream=None):
    """The gradient at gelu's input from that at its output, with the input as
    `kept` holds it.  out may be da."""
    d, rows, cols, device = _matrix(da)
    codes = kept.codes
    if da.shape != codes.shape or device != codes.device:
        raise ValueError(f"da is {tuple(codes.shape)} on {codes.device}: got {tuple(da.shape)} {device}")
    if out is None:
        out = torch.empty_like(da)
    else:
        _like(out, da, "out")
    _call("snk_gelu_backward_q8", da.data_ptr(), d, codes.data_ptr(), kept.scales.data_ptr(), rows, cols,
          kept.format_id, kept.group, out.data_ptr(), _on(stream, device))
    return out


def rmsnorm(x, gain, residual=None, eps: float = 1e-5, format: str = "int8", group: int = 0, stream=None):
    """The norm of total = x + residual (x without a residual) times gain, in 8
    bits: (Q8Tensor, total, rstd), rstd [...] the reciprocal root mean square."""
    d, rows, cols, device = _matrix(x)
    shape = x.shape
    g = _f32(gain, cols, device, "gain")
    if residual is None:
        total, res_p, total_p = x, None, None
    else:
        res_p = _like(residual, x, "residual")
        total = torch.empty_like(x)
        total_p = total.data_ptr()
    q = _new(shape, rows, cols, device, format, group)
    rstd = _empty(shape[:-1], dtype=_F32, device=device)
    _call("snk_rmsnorm_q8", x.data_ptr(), res_p, d, g, rows, cols, eps, q.format_id, group, q.codes.data_ptr(),
          q.scales.data_ptr(), total_p, rstd.data_ptr(), _on(stream, device))
    return q, total, rstd


def rmsnorm_backward(dy, total, rstd, gain, dtotal=None, stream=None):
    """(dx, dgain) from the gradient dy (float32) of the norm's output and that
    of total on its other path; dx is the gradient of x and of residual."""
    d, rows, cols, device = _matrix(total)
    dy_p = _f32(dy, rows * cols, device, "dy")
    rstd_p = _f32(rstd, rows, device, "rstd")
    gain_p = _f32(gain, cols, device, "gain")
    dtotal_p = None if dtotal is None else _like(dtotal, total, "dtotal")
    dx = torch.empty_like(total)
    dgain = torch.empty_like(gain)
    scratch = _empty(binding.snk_rmsnorm_backward_scratch(rows, cols), dtype=torch.uint8, device=device)
    _call("snk_rmsnorm_backward", dy_p, total.data_ptr(), d, rstd_p, gain_p, dtotal_p, rows, cols, dx.data_ptr(),
          dgain.data_ptr(), scratch.data_ptr(), _on(stream, device))
    return dx, dgain
