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

A call runs on torch's current stream, or on `stream` (a stream or its handle), as
if that were current: new tensors then belong to it.
"""
from __future__ import annotations

import torch

from . import binding

_DTYPES = {torch.float32: binding.SNK_F32, torch.float16: binding.SNK_F16,
           torch.bfloat16: binding.SNK_BF16}
_FORMATS = {"int8": binding.SNK_Q8_INT8, "e4m3": binding.SNK_Q8_E4M3}
_GROUPS = (0, 32, 64, 128, 256)


def _format(name: str) -> int:
    f = _FORMATS.get(name)
    if f is None:
        raise ValueError(f"format is one of {tuple(_FORMATS)}: got {name!r}")
    return f


class Q8Tensor:
    """codes (int8, or float8_e4m3fn) [..., cols] and scales float32 [...,
    ceil(cols / group)] (group 0: [..., 1]); it stands for scale * code."""

    __slots__ = ("codes", "scales", "group")

    def __init__(self, codes, scales, group: int):
        if group not in _GROUPS:
            raise ValueError(f"group is one of {_GROUPS}: got {group}")
        if codes.dtype not in (torch.int8, torch.float8_e4m3fn):
            raise ValueError(f"codes are int8 or float8_e4m3fn: got {codes.dtype}")
        if not codes.is_cuda or codes.dim() < 1 or codes.shape[-1] < 1 or not codes.is_contiguous():
            raise ValueError(f"codes are a contiguous CUDA tensor [..., cols] with cols >= 1: got {codes.device} "
                             f"{tuple(codes.shape)}, strides {codes.stride()}")
        cols = codes.shape[-1]
        n = codes.numel() // cols * (-(-cols // group) if group else 1)
        if scales.dtype != torch.float32 or scales.numel() != n or scales.device != codes.device \
                or not scales.is_contiguous():
            raise ValueError(f"scales are contiguous float32 with {n} elements on {codes.device}: got {scales.dtype} "
                             f"{tuple(scales.shape)} {scales.device}")
        self.codes, self.scales, self.group = codes, scales, group

    @property
    def rows(self) -> int:
        return self.codes.numel() // self.codes.shape[-1]

    @property
    def cols(self) -> int:
        return self.codes.shape[-1]

    @property
    def format_id(self) -> int:
        return binding.SNK_Q8_INT8 if self.codes.dtype == torch.int8 else binding.SNK_Q8_E4M3

    @property
    def format(self) -> str:
        return "int8" if self.codes.dtype == torch.int8 else "e4m3"

    @property
    def shape(self):
        return self.codes.shape

    def dequantize(self, dtype=torch.float32):
        return unpack(self, dtype)


def _wrap(codes, scales, group):
    q = Q8Tensor.__new__(Q8Tensor)   # already checked
    q.codes, q.scales, q.group = codes, scales, group
    return q


def pack(x, format: str = "int8", group: int = 0, stream=None) -> Q8Tensor:
    """x in 8 bits."""
    codes, scales = binding.ops().pack(x, _format(format), group, stream)
    return _wrap(codes, scales, group)


def unpack(q: Q8Tensor, dtype=torch.float32, stream=None):
    """scale * code, rounded to dtype."""
    d = _DTYPES.get(dtype)
    if d is None:
        raise ValueError(f"float32, float16 or bfloat16 is needed: got {dtype}")
    return binding.ops().unpack(q.codes, q.scales, q.group, d, stream)


def gelu(x, format: str = "int8", group: int = 0, keep: bool = False, stream=None):
    """x Phi(x) in 8 bits; with keep, also x itself in 8 bits, for
    gelu_backward: (gelu(x), x)."""
    codes, scales, kept_codes, kept_scales = binding.ops().gelu(x, _format(format), group, keep, stream)
    q = _wrap(codes, scales, group)
    return (q, _wrap(kept_codes, kept_scales, group)) if keep else q


def gelu_backward(da, kept: Q8Tensor, out=None, stream=None):
    """The gradient at gelu's input from that at its output, with the input as
    `kept` holds it.  out may be da."""
    return binding.ops().gelu_backward(da, kept.codes, kept.scales, kept.group, out, stream)


def rmsnorm(x, gain, residual=None, eps: float = 1e-5, format: str = "int8", group: int = 0, stream=None):
    """The norm of total = x + residual (x without a residual) times gain, in 8
    bits: (Q8Tensor, total, rstd), rstd [...] the reciprocal root mean square."""
    codes, scales, total, rstd = binding.ops().rmsnorm(x, gain, residual, eps, _format(format), group, stream)
    return _wrap(codes, scales, group), x if residual is None else total, rstd


def rmsnorm_backward(dy, total, rstd, gain, dtotal=None, stream=None):
    """(dx, dgain) from the gradient dy (float32) of the norm's output and that
    of total on its other path; dx is the gradient of x and of residual."""
    return binding.ops().rmsnorm_backward(dy, total, rstd, gain, dtotal, stream)
