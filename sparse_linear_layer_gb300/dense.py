"""The dense part of a model whose MLPs are truly sparse: projections whose products run
on 8-bit matrices, and the loss of the vocabulary head, in pieces of the vocabulary; both
with autograd.

    layer = Q8Linear(768, 2304)                         # x W^T + b and its gradients in 8 bits
    y = layer(x)                                        # (linear_q8(x, weight, bias))
    head = VocabularyHead(768, 50257)
    loss = head(x, target)                              # (linear_cross_entropy(x, weight, target))
    logits = head.logits(x, head.pack())                # of a few tokens, from an 8-bit weight

  "Beyond Masked Sparsity: SNACK Enables Truly Sparse Neural Networks on GPU",
    Tables 4-5: language models whose MLPs are truly sparse layers; the head and
    its loss are this library's.

Everything numeric runs in libsnk's kernels; the native module wires them into autograd
(a Python function took 60 to 100 us more of host time for a forward and a backward pass).
"""
from __future__ import annotations

import torch

from . import binding, q8

_REDUCTIONS = {"none": 0, "sum": 1, "mean": 2}


def linear_cross_entropy(x, weight, target, ignore: int = -100, reduction: str = "mean"):
    """Softmax cross entropy of the logits x weight^T, which are never kept.

    x [..., cols] and weight [vocab, cols] are both float16 or both bfloat16, target [...]
    is int64.  Rows whose target is `ignore` take no part, whatever x holds there; a
    target outside the vocabulary gives NaN.  The loss is float32: one per row for
    reduction "none" (zero for ignored rows), else their sum or their mean over the
    rows that count.  Gradients have the types of x and weight."""
    r = _REDUCTIONS.get(reduction)
    if r is None:
        raise ValueError(f"reduction is one of {tuple(_REDUCTIONS)}: got {reduction!r}")
    return binding.ops().linear_cross_entropy(x, weight, target, ignore, r)


def linear_q8(x, weight, bias=None):
    """x weight^T + bias with the products, and those of the gradients, on 8-bit matrices:
    E4M3 codes with a scale for each 128 columns of a row (x, and the upstream gradient)
    or each 128 x 128 block (weight); for the weight's gradient x and the upstream
    gradient have a scale for each 128 rows of a column.

    x [..., cols], weight [out, cols] and bias [out] are float32, float16 or bfloat16, each
    its own type.  The result and x's gradient have x's type, the others' gradients theirs.
    Sums are fp32; roundings to 8 bits are passed through as the
    identity, and x is kept for the backward pass as one byte per element."""
    return binding.ops().linear_q8(x, weight, bias)


class Q8Linear(torch.nn.Module):
    """linear_q8 as a layer: weight [out_features, in_features] and bias float32, or what
    the layer is converted to (.bfloat16(), .half())."""

    def __init__(self, in_features: int, out_features: int, bias: bool = True, device=None):
        super().__init__()
        device = torch.device(device if device is not None else "cuda")
        self.in_features, self.out_features = in_features, out_features
        self.weight = torch.nn.Parameter(torch.randn(out_features, in_features, device=device) * in_features ** -0.5)
        self.bias = torch.nn.Parameter(torch.zeros(out_features, device=device)) if bias else None

    def forward(self, x):
        return linear_q8(x, self.weight, self.bias)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, bias={self.bias is not None}"


class VocabularyHead(torch.nn.Module):
    """The projection onto the vocabulary: weight [vocab, features] in bfloat16 or float16.

    forward(x, target) is linear_cross_entropy of x (converted to the weight's type).
    logits(x) serves: x and the weight in 8 bits (q8.matmul).  A program that serves packs
    the weight once, w8 = head.pack(), and passes it: logits(x, w8)."""

    def __init__(self, features: int, vocab: int, dtype=torch.bfloat16, ignore: int = -100, device=None):
        super().__init__()
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype is bfloat16 or float16: got {dtype}")
        device = torch.device(device if device is not None else "cuda")
        self.features, self.vocab, self.ignore = features, vocab, ignore
        self.weight = torch.nn.Parameter((torch.randn(vocab, features, device=device) * features ** -0.5).to(dtype))

    def forward(self, x, target, reduction: str = "mean"):
        return linear_cross_entropy(x.to(self.weight.dtype), self.weight, target, self.ignore, reduction)

    def pack(self) -> q8.Q8Blocks:
        """The weight, as it is now, in 8 bits."""
        return q8.pack_blocks(self.weight)

    @torch.no_grad()
    def logits(self, x, weight: q8.Q8Blocks | None = None, dtype=torch.float32):
        """x [..., features], or its 8-bit form (format "e4m3", group 128, as q8.rmsnorm
        writes it): the logits [..., vocab], with `weight` from pack() (else packed here)."""
        if not isinstance(x, q8.Q8Tensor):
            x = q8.pack(x.contiguous(), "e4m3", 128)
        return q8.matmul(x, self.pack() if weight is None else weight, dtype=dtype)

    def extra_repr(self) -> str:
        return f"features={self.features}, vocab={self.vocab}, ignore={self.ignore}"
