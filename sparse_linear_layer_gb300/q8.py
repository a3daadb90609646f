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


def _shape(t):
    """(rows, cols) of a contiguous CUDA tensor [..., cols]."""
    if not t.is_cuda or not t.is_contiguous() or t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"a contiguous CUDA tensor [..., cols] with cols >= 1 is needed: got {t.device} "
                         f"{tuple(t.shape)}, strides {t.stride()}")
    cols = t.shape[-1]
    return t.numel() // cols, cols


def _dtype(t):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"float32, float16 or bfloat16 is needed: got {t.dtype}")
    return d


def _same(t, like, name):
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} has the shape, type and device of {tuple(like.shape)} {like.dtype} {like.device}, "
                         f"contiguous: got {tuple(t.shape)} {t.dtype} {t.device}")


def _f32(t, n, like, name):
    if t.dtype != torch.float32 or t.numel() != n or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} is contiguous float32 with {n} elements on {like.device}: got {t.dtype} "
                         f"{tuple(t.shape)} {t.device}")


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
        self.rows, self.cols = _shape(codes)
        _f32(scales, self.rows * (-(-self.cols // group) if group else 1), codes, "scales")
        self.codes, self.scales, self.group = codes, scales, group

    @property
    def format(self) -> str:
        return "int8" if self.format_id == binding.SNK_Q8_INT8 else "e4m3"

    @property
    def shape(self):
        return self.codes.shape

    def require(self, cols: int):
        if self.cols != cols:
            raise ValueError(f"a matrix of {cols} columns is needed: got {tuple(self.codes.shape)}")

    def dequantize(self, dtype=torch.float32):
        return unpack(self, dtype)


def _empty(x, rows, cols, format, group):
    """A new Q8Tensor of x's shape."""
    if format not in _FORMATS or group not in _GROUPS:
        raise ValueError(f"format is one of {tuple(_FORMATS)} and group one of {_GROUPS}: got {format!r}, {group}")
    q = Q8Tensor.__new__(Q8Tensor)
    q.format_id, dtype = _FORMATS[format]
    q.rows, q.cols, q.group = rows, cols, group
    q.codes = torch.empty(x.shape, dtype=dtype, device=x.device)
    q.scales = torch.empty((*x.shape[:-1], -(-cols // group) if group else 1), dtype=torch.float32, device=x.device)
    return q


def pack(x, format: str = "int8", group: int = 0, stream=None) -> Q8Tensor:
    """x in 8 bits."""
    rows, cols = _shape(x)
    d = _dtype(x)
    q = _empty(x, rows, cols, format, group)
    binding.snk_q8_pack(x, d, rows, cols, q.format_id, group, q.codes, q.scales, stream)
    return q


def unpack(q: Q8Tensor, dtype=torch.float32, stream=None):
    """scale * code, rounded to dtype."""
    x = torch.empty(q.codes.shape, dtype=dtype, device=q.codes.device)
    binding.snk_q8_unpack(q.codes, q.scales, q.rows, q.cols, q.format_id, q.group, x, _dtype(x), stream)
    return x


def gelu(x, format: str = "int8", group: int = 0, keep: bool = False, stream=None):
    """x Phi(x) in 8 bits; with keep, also x itself in 8 bits, for
    gelu_backward: (gelu(x), x)."""
    rows, cols = _shape(x)
    d = _dtype(x)
    q = _empty(x, rows, cols, format, group)
    kept = _empty(x, rows, cols, format, group) if keep else None
    binding.snk_gelu_q8(x, d, rows, cols, q.format_id, group, q.codes, q.scales, kept.codes if keep else None,
                        kept.scales if keep else None, stream)
    return (q, kept) if keep else q


def gelu_backward(da, kept: Q8Tensor, out=None, stream=None):
    """The gradient at gelu's input from that at its output, with the input as
    `kept` holds it.  out may be da."""
    if da.shape != kept.codes.shape or da.device != kept.codes.device or not da.is_contiguous():
        raise ValueError(f"da is contiguous {tuple(kept.codes.shape)} on {kept.codes.device}: got {tuple(da.shape)} "
                         f"{da.device}")
    d = _dtype(da)
    if out is None:
        out = torch.empty_like(da)
    else:
        _same(out, da, "out")
    binding.snk_gelu_backward_q8(da, d, kept.codes, kept.scales, kept.rows, kept.cols, kept.format_id, kept.group,
                                 out, stream)
    return out


def rmsnorm(x, gain, residual=None, eps: float = 1e-5, format: str = "int8", group: int = 0, stream=None):
    """The norm of total = x + residual (x without a residual) times gain, in 8
    bits: (Q8Tensor, total, rstd), rstd [...] the reciprocal root mean square."""
    rows, cols = _shape(x)
    d = _dtype(x)
    _f32(gain, cols, x, "gain")
    total = x
    if residual is not None:
        _same(residual, x, "residual")
        total = torch.empty_like(x)
    q = _empty(x, rows, cols, format, group)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    binding.snk_rmsnorm_q8(x, residual, d, gain, rows, cols, eps, q.format_id, group, q.codes, q.scales,
                           None if residual is None else total, rstd, stream)
    return q, total, rstd


def rmsnorm_backward(dy, total, rstd, gain, dtotal=None, stream=None):
    """(dx, dgain) from the gradient dy (float32) of the norm's output and that
    of total on its other path; dx is the gradient of x and of residual."""
    rows, cols = _shape(total)
    d = _dtype(total)
    _f32(dy, rows * cols, total, "dy")
    _f32(rstd, rows, total, "rstd")
    _f32(gain, cols, total, "gain")
    if dtotal is not None:
        _same(dtotal, total, "dtotal")
    dx = torch.empty_like(total)
    dgain = torch.empty_like(gain)
    scratch = torch.empty(binding.snk_rmsnorm_backward_scratch(rows, cols), dtype=torch.uint8, device=total.device)
    binding.snk_rmsnorm_backward(dy, total, d, rstd, gain, dtotal, rows, cols, dx, dgain, scratch, stream)
    return dx, dgain
