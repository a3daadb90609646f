"""8-bit activations: matrices of one byte per element with fp32 scales, and
the calls that write and read them (include/snk.h has the definitions).

    kept = pack(x, format="int8", group=128)         # a checkpoint of x
    x2 = unpack(kept)                                # its values
    q, total, rstd = rmsnorm(x, gain, residual=r)    # norm of x + r in 8 bits
    dx, dgain = rmsnorm_backward(dy, total, rstd, gain, dtotal=dr)
    a, kept = gelu(h, keep=True)                     # gelu(h) and h in 8 bits
    dh = gelu_backward(da, kept)

    w8 = pack_blocks(w)                              # a dense weight, a scale per 128 x 128 block
    y = matmul(pack(x, "e4m3", 128), w8, bias)       # x w^T + bias on the 8-bit values

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


class Q8Blocks:
    """A dense weight in 8 bits: codes float8_e4m3fn [rows, cols] and scales float32
    [ceil(rows / 128), ceil(cols / 128)], one for each 128 x 128 block; it stands for
    scale * code.  Rows of codes may lie further apart than they are long; those that do
    not start on 16 bytes are copied once, here."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes, scales):
        if codes.dtype != torch.float8_e4m3fn or not codes.is_cuda or codes.dim() != 2 or codes.shape[0] < 1 \
                or codes.shape[1] < 1 or codes.stride(1) != 1 or codes.stride(0) < codes.shape[1]:
            raise ValueError(f"codes are a float8_e4m3fn CUDA tensor [rows, cols], rows and cols >= 1, of contiguous rows: "
                             f"got {codes.dtype} {codes.device} {tuple(codes.shape)}, strides {codes.stride()}")
        shape = tuple(-(-n // 128) for n in codes.shape)
        if scales.dtype != torch.float32 or scales.shape != shape or scales.device != codes.device \
                or not scales.is_contiguous():
            raise ValueError(f"scales are contiguous float32 {shape} on {codes.device}: got {scales.dtype} "
                             f"{tuple(scales.shape)} {scales.device}")
        if codes.stride(0) % 16 or codes.data_ptr() % 16:
            rows = torch.empty(codes.shape[0], -(-codes.shape[1] // 16) * 16, dtype=codes.dtype, device=codes.device)
            rows[:, :codes.shape[1]].copy_(codes)
            codes = rows[:, :codes.shape[1]]
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return self.codes.shape


def _wrap_blocks(codes, scales):
    w = Q8Blocks.__new__(Q8Blocks)
    w.codes, w.scales = codes, scales
    return w


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


def pack_both(x, stream=None):
    """x and x^T in 8 bits (E4M3, groups of 128): (Q8Tensor [rows, cols], Q8Tensor
    [cols, rows]), from one reading of x [..., cols]."""
    codes, scales, codes_t, scales_t, _ = binding.ops().pack_both(x, True, True, False, False, stream)
    return _wrap(codes, scales, 128), _wrap(codes_t, scales_t, 128)


def pack_blocks(w, transposed: bool = False, stream=None):
    """A dense weight w [rows, cols] in 8 bits, one scale per 128 x 128 block; with
    transposed, also w^T: (w, w^T), the same codes and scales."""
    codes, scales, codes_t, scales_t = binding.ops().pack_blocks(w, True, transposed, stream)
    q = _wrap_blocks(codes, scales)
    return (q, _wrap_blocks(codes_t, scales_t)) if transposed else q


def matmul(a: Q8Tensor, b, bias=None, dtype=torch.float32, out=None, stream=None):
    """a b^T + bias in `dtype`: a [..., cols] with format "e4m3" and group 128; b
    [n, cols] the same, or a Q8Blocks; bias [n] float32.  The 8-bit values' products
    and sums are fp32."""
    d = _DTYPES.get(dtype)
    if d is None:
        raise ValueError(f"float32, float16 or bfloat16 is needed: got {dtype}")
    blocks = isinstance(b, Q8Blocks)
    if a.group != 128 or not (blocks or b.group == 128):
        raise ValueError(f"matmul needs groups of 128 columns: got {a.group}" + ("" if blocks else f" and {b.group}"))
    return binding.ops().matmul(a.codes, a.scales, b.codes, b.scales, blocks, bias, d, out, stream)
