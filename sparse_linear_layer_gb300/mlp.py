"""A pre-norm MLP block of two truly sparse layers whose activations are kept in
8 bits:

    total = x + residual
    y     = down(gelu(up(rmsnorm(total) * gain)))

The norm writes its output in 8 bits and the first layer multiplies that; GELU
reads the first layer's output once and writes both its own output and that input
in 8 bits, and the second layer multiplies the former.  The backward pass takes
both layers' weight gradients, and GELU's slope, from the 8-bit matrices, so a
block keeps one byte per activation (with fp32 layers: four) beside the residual
stream.  Roundings to 8 bits are passed through as the identity.

  "Beyond Masked Sparsity: SNACK Enables Truly Sparse Neural Networks on GPU",
    Tables 4-5: the GPT-2 MLP stack (768 -> 3072 -> 768, GELU) with truly
    sparse layers; the norm and the 8-bit activations are this library's.

Everything numeric runs in libsnk's kernels; this file wires them into autograd.
"""
from __future__ import annotations

import torch

from . import q8
from .module import SparseLinear


class _SparseMLPFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gain, up_values, up_bias, down_values, down_bias, block, grad):
        ctx.set_materialize_grads(False)
        # what the backward pass of the inputs that need it reads: the first layer's input, GELU's (for all
        # that lies before GELU), the second layer's input, the norm's
        needs = [grad and need for need in ctx.needs_input_grad[:7]]
        n, total, rstd = q8.rmsnorm(x, gain, residual=residual, eps=block.eps, format=block.format,
                                    group=block.group)
        h = block.up._h.forward_q8(n, up_bias)
        a = q8.gelu(h, format=block.format, group=block.group, keep=any(needs[:5]))
        a, kept = a if any(needs[:5]) else (a, None)
        y = block.down._h.forward_q8(a, down_bias)
        ctx.block, ctx.has_residual, ctx.group = block, residual is not None, n.group
        held = [*((total, rstd, gain) if any(needs[:3]) else (None,) * 3)]
        for q, needed in ((n, any(needs[3:5])), (kept, any(needs[:5])), (a, any(needs[5:]))):
            held += (q.codes, q.scales) if needed else (None, None)
        ctx.save_for_backward(*held)
        return (y, total) if ctx.has_residual else y

    @staticmethod
    def backward(ctx, dy, dtotal=None):
        up, down, needs = ctx.block.up, ctx.block.down, ctx.needs_input_grad
        if dtotal is not None:
            dtotal = dtotal.contiguous()
        if dy is None:   # only total was used
            return (dtotal, dtotal if ctx.has_residual else None) + (None,) * 7
        total, rstd, gain, *codes = ctx.saved_tensors
        n, kept, a = (None if c is None else q8.Q8Tensor(c, s, ctx.group) for c, s in zip(codes[::2], codes[1::2]))
        dy = dy.contiguous()
        dx = dgain = d_up = d_up_bias = d_down = d_down_bias = None
        if any(needs[5:7]):
            d_down, d_down_bias = down._h.backward_weight_q8(a, dy, with_bias=True)
        if any(needs[:5]):
            da = down._h.backward_input(dy)
            dh = q8.gelu_backward(da, kept, out=da)
            if any(needs[3:5]):
                d_up, d_up_bias = up._h.backward_weight_q8(n, dh, with_bias=True)
            if any(needs[:3]):
                dn = up._h.backward_input(dh)
                dx, dgain = q8.rmsnorm_backward(dn, total, rstd, gain, dtotal=dtotal)
        grads = (dx, dx, dgain, d_up, d_up_bias, d_down, d_down_bias)
        return tuple(d if need else None for d, need in zip(grads, needs)) + (None, None)


class SparseMLP(torch.nn.Module):
    """forward(x) gives y; forward(x, residual) gives (y, total), total being
    the residual stream that the next block adds y to.  x and residual [...,
    features] are float32, float16 or bfloat16; y has their type.  format and
    group are those of every 8-bit matrix of the block (see q8)."""

    def __init__(self, features: int, hidden: int, sparsity: float, bias: bool = True, eps: float = 1e-5,
                 format: str = "int8", group: int = 0, seed: int = 0, device=None):
        super().__init__()
        self._join(SparseLinear(features, hidden, sparsity, bias=bias, seed=seed, device=device),
                   SparseLinear(hidden, features, sparsity, bias=bias, seed=seed + 2, device=device), eps, format, group)

    @classmethod
    def from_layers(cls, up: SparseLinear, down: SparseLinear, eps: float = 1e-5, format: str = "int8", group: int = 0):
        """A block of two layers that exist (SparseLinear.from_triple): up features ->
        hidden, down hidden -> features."""
        if (up.in_features, up.out_features) != (down.out_features, down.in_features):
            raise ValueError(f"up and down are features -> hidden and hidden -> features: got {up.in_features} -> "
                             f"{up.out_features} and {down.in_features} -> {down.out_features}")
        self = cls.__new__(cls)
        torch.nn.Module.__init__(self)
        self._join(up, down, eps, format, group)
        return self

    def _join(self, up, down, eps, format, group):
        self.up, self.down = up, down
        self.gain = torch.nn.Parameter(torch.ones(up.in_features, device=up.values.device))
        self.eps, self.format, self.group = eps, format, group

    def forward(self, x, residual=None):
        features = self.up.in_features
        x2 = x.reshape(-1, features).contiguous()
        args = (self.gain, self.up.values, self.up.bias, self.down.values, self.down.bias, self,
                torch.is_grad_enabled())   # (inside the function gradients are off)
        if residual is None:
            return _SparseMLPFn.apply(x2, None, *args).to(x.dtype).reshape(x.shape)
        r2 = residual.reshape(-1, features).contiguous()
        y, total = _SparseMLPFn.apply(x2, r2, *args)
        return y.to(x.dtype).reshape(x.shape), total.reshape(x.shape)

    def sparse_layers(self):
        """The block's layers, for SET."""
        return [self.up, self.down]

    def extra_repr(self) -> str:
        return f"eps={self.eps}, format={self.format!r}, group={self.group}"

    def close(self):
        self.up.close()
        self.down.close()
