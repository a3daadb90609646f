"""The dense part of a model whose MLPs are truly sparse: the loss of its vocabulary head with the gradients, and dense products on
8-bit matrices.

The loss is softmax cross entropy of logits x W^T that are never kept; x and W are in 16 bits. A row whose target is -100 is left
out.

An 8-bit matrix has codes (8-bit floats E4M3) and 32-bit scales: one for each 128 columns of a row, or, of a weight, one for each
128 x 128 block. It stands for scale * code. A group's (block's) scale is its largest magnitude over 448.
"""
import math

import torch

own = False

TINY = 2.0 ** -100  # a group whose largest magnitude is below this is held as zeros
TOP = 448.0
IGNORE = -100
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the loss of one token, as when scoring a continuation step by step: latency
        {"name": "loss, one token", "op": "score", "rows": 1, "cols": 768, "vocab": 50257, "type": "bf16", "ignored": 0.0},
        # evaluation of a few ragged texts, padding left out
        {"name": "loss, ragged evaluation", "op": "score", "rows": 333, "cols": 1000, "vocab": 32003, "type": "f16", "ignored": 0.1},
        # a training step over 8 sequences of 1024 tokens: loss and both gradients
        {"name": "loss training step", "op": "train", "rows": 8192, "cols": 768, "vocab": 50257, "type": "bf16", "ignored": 0.0},
        # a wide model's micro-batch whose prompts are not trained on
        {"name": "loss training step, wide", "op": "train", "rows": 4096, "cols": 4096, "vocab": 65536, "type": "bf16", "ignored": 0.3},
        # one short sequence, where the vocabulary's matrix and its gradient are most of the traffic
        {"name": "loss training step, one text", "op": "train", "rows": 100, "cols": 768, "vocab": 50257, "type": "f16", "ignored": 0.0},
        # the projection before attention, one token of one sequence: latency
        {"name": "product, one token", "op": "matmul", "rows": 1, "cols": 768, "out": 2304, "weight": "blocks", "type": "bf16"},
        # the vocabulary head's logits in a decoding step of 64 sequences
        {"name": "product, logits of 64", "op": "matmul", "rows": 64, "cols": 768, "out": 50257, "weight": "blocks", "type": "f32"},
        # odd sizes: a partial group, a partial block, a partial tile
        {"name": "product, ragged", "op": "matmul", "rows": 333, "cols": 1000, "out": 1001, "weight": "blocks", "type": "f32"},
        # the large layer on a large batch
        {"name": "product, large batch", "op": "matmul", "rows": 8192, "cols": 10000, "out": 10000, "weight": "blocks", "type": "bf16"},
        # a weight gradient: both operands with scales along the tokens
        {"name": "product, weight gradient", "op": "matmul", "rows": 4096, "cols": 16384, "out": 1024, "weight": "rows", "type": "f32"},
        # a dense projection's training step over 32 sequences of 1024 tokens, packing included
        {"name": "linear training step", "op": "linear", "rows": 32768, "cols": 768, "out": 2304, "type": "bf16"},
        # the same with odd sizes, everything in 32 bits
        {"name": "linear training step, ragged", "op": "linear", "rows": 777, "cols": 1000, "out": 1500, "type": "f32"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        n = spread(lo, hi)
        return n if rng.random() < 0.25 else max(8, n // 8 * 8)  # most widths of real models are whole multiples of 8

    op = rng.choice(["score", "train", "matmul", "linear"])
    c = {"op": op}
    if op in ("score", "train"):
        c["cols"], c["vocab"] = width(64, 4096), spread(1000, 131072)
        c["rows"] = spread(1, max(2, min(8192, 300_000_000_000 // (c["cols"] * c["vocab"]), 400_000_000 // c["vocab"])))
        c["type"], c["ignored"] = rng.choice(["bf16", "f16"]), rng.choice([0.0, 0.0, 0.1, 0.5, 0.9])
        return c
    if op == "matmul":
        c["cols"], c["out"] = width(64, 16384), spread(64, 16384)
        c["rows"] = spread(1, min(16384, 500_000_000_000 // (c["cols"] * c["out"])))
        c["weight"], c["type"] = rng.choice(["blocks", "blocks", "rows"]), rng.choice(["bf16", "f16", "f32"])
        return c
    c["cols"], c["out"] = width(64, 8192), width(64, 8192)
    c["rows"] = spread(1, min(32768, 50_000_000_000 // (c["cols"] * c["out"])))
    c["type"] = rng.choice(["bf16", "f16", "f32"])
    return c


def _activations(g, rows, cols, dtype, scale=1.0):
    """Normal values with a few columns far larger than the others, as hidden states have them."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    loud = 1.0 + 9.0 * (torch.rand(cols, device="cuda", generator=g) < 0.01)
    return (x * loud * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, cols = case["op"], case["rows"], case["cols"]
    s = dict(case)
    dtype = TYPES[case["type"]]
    if op in ("score", "train"):
        # a normed state and a head whose logits spread by about 3; a target is right with the model's own odds now and then
        s["x"] = _activations(g, rows, cols, dtype, 0.7)
        s["w"] = (2.0 / math.sqrt(cols) * torch.randn(case["vocab"], cols, device="cuda", generator=g)).to(dtype)
        s["target"] = torch.randint(0, case["vocab"], (rows,), device="cuda", generator=g)
        out = torch.rand(rows, device="cuda", generator=g) < case["ignored"]
        out[0] = False
        s["target"][out] = IGNORE
        if op == "train":
            s["x"].requires_grad_(own)
            s["w"].requires_grad_(own)
    elif op == "matmul":
        s["a"], s["a_scales"] = _pack(_activations(g, rows, cols, torch.float32))
        w = torch.randn(case["out"], cols, device="cuda", generator=g) / math.sqrt(cols)
        s["b"], s["b_scales"] = _pack(w) if case["weight"] == "rows" else _pack_blocks(w)
        del w
        s["bias"] = 0.1 * torch.randn(case["out"], device="cuda", generator=g)
    else:
        s["x"] = _activations(g, rows, cols, dtype)
        s["w"] = torch.randn(case["out"], cols, device="cuda", generator=g) / math.sqrt(cols)
        s["bias"] = 0.1 * torch.randn(case["out"], device="cuda", generator=g)
        s["dy"] = (1e-3 * torch.randn(rows, case["out"], device="cuda", generator=g)).to(dtype)
        for name in ("x", "w", "bias"):
            s[name].requires_grad_(own)
    if own:
        from sparse_linear_layer_gb300 import dense, q8
        s["dense"], s["q8"] = dense, q8
        if op == "matmul":
            s["a8"] = q8.Q8Tensor(s["a"], s["a_scales"], 128)
            s["b8"] = q8.Q8Tensor(s["b"], s["b_scales"], 128) if case["weight"] == "rows" else q8.Q8Blocks(s["b"], s["b_scales"])
    return s


# ------------------------------------------------------------------ plain forms

def _codes(y, most):
    """(codes, scales) of groups whose largest magnitudes are `most`, of a shape that stretches over y's."""
    used = most >= TINY
    inverse = torch.where(used, torch.full_like(most, TOP) / most, 0.0)
    return (y * inverse).to(torch.float8_e4m3fn), torch.where(used, most / torch.full_like(most, TOP), 0.0)


def _filled(y, high, wide):
    """y with zeros below and to the right, up to whole tiles."""
    rows, cols = y.shape
    full = torch.zeros(rows + -rows % high, cols + -cols % wide, device=y.device, dtype=y.dtype)
    full[:rows, :cols] = y
    return full


def _pack(y):
    """A scale for each 128 columns of a row."""
    rows, cols = y.shape
    full = _filled(y.float(), 1, 128).reshape(rows, -1, 128)
    codes, scales = _codes(full, full.abs().amax(2, keepdim=True))
    return codes.reshape(rows, -1)[:, :cols].contiguous(), scales.reshape(rows, -1)


def _pack_blocks(w):
    """A scale for each 128 x 128 block."""
    rows, cols = w.shape
    full = _filled(w.float(), 128, 128)
    high, wide = full.shape
    tiles = full.reshape(high // 128, 128, wide // 128, 128)
    codes, scales = _codes(tiles, tiles.abs().amax((1, 3), keepdim=True))
    return codes.reshape(high, wide)[:rows, :cols].contiguous(), scales.reshape(high // 128, wide // 128)


def _values(codes, scales, blocks):
    if blocks:
        scales = scales.repeat_interleave(128, 0)[:codes.shape[0]]
    return codes.float() * scales.repeat_interleave(128, 1)[:, :codes.shape[1]]


def _plain(s):
    op = s["op"]
    if op in ("score", "train"):
        x, w, target = s["x"].float(), s["w"].float(), s["target"]
        kept = target != IGNORE
        at = torch.where(kept, target, 0)[:, None]
        z = x @ w.T
        most = z.amax(1, keepdim=True)
        p = torch.exp(z - most)
        total = p.sum(1, keepdim=True)
        loss = torch.where(kept, (torch.log(total) + most - z.gather(1, at))[:, 0], 0.0)
        if op == "score":
            return {"loss": loss}
        n = kept.sum()
        del z
        p /= total
        p.scatter_add_(1, at, torch.full_like(total, -1.0))
        p *= kept[:, None] / n
        return {"loss": loss.sum() / n, "dx": (p @ w).to(s["x"].dtype), "dw": (p.T @ x).to(s["w"].dtype)}
    dtype = TYPES[s["type"]]
    if op == "matmul":
        y = _values(s["a"], s["a_scales"], False) @ _values(s["b"], s["b_scales"], s["weight"] == "blocks").T
        return {"y": (y + s["bias"]).to(dtype)}
    w = _values(*_pack_blocks(s["w"]), True)
    y = _values(*_pack(s["x"]), False) @ w.T + s["bias"]
    dx = _values(*_pack(s["dy"]), False) @ w
    dw = _values(*_pack(s["dy"].T), False) @ _values(*_pack(s["x"].T), False).T
    return {"y": y.to(dtype), "dx": dx.to(dtype), "dw": dw, "db": s["dy"].float().sum(0)}


def run(s):
    if not own:
        return _plain(s)
    dense, q8, op = s["dense"], s["q8"], s["op"]
    if op == "score":
        with torch.no_grad():
            return {"loss": dense.linear_cross_entropy(s["x"], s["w"], s["target"], ignore=IGNORE, reduction="none")}
    if op == "train":
        loss = dense.linear_cross_entropy(s["x"], s["w"], s["target"], ignore=IGNORE)
        dx, dw = torch.autograd.grad(loss, (s["x"], s["w"]))
        return {"loss": loss.detach(), "dx": dx, "dw": dw}
    if op == "matmul":
        return {"y": q8.matmul(s["a8"], s["b8"], bias=s["bias"], dtype=TYPES[s["type"]])}
    y = dense.linear_q8(s["x"], s["w"], s["bias"])
    dx, dw, db = torch.autograd.grad(y, (s["x"], s["w"], s["bias"]), s["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw, "db": db}


# ------------------------------------------------------------------ 64 bits

def _grid(v):
    """The nearest code value, halves to even."""
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -6))
    step = torch.ldexp(torch.ones_like(v), e - 4)  # three bits after the leading one
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_rounded(y, high):
    """The values that y's 8-bit form stands for, a scale for each `high` rows and 128 columns. (The factor onto the grid and the
    scale are 32-bit numbers by definition.)"""
    out = torch.zeros_like(y, dtype=torch.float64)
    for c in range(0, y.shape[1], 128):
        part = y[:, c:c + 128].float()
        most = part.abs().max(1).values
        if high > 1:
            most = torch.cat([m.max().expand(m.numel()) for m in most.split(high)])
        most = most[:, None]
        inverse, scale = torch.tensor(TOP, device=y.device) / most, most / torch.tensor(TOP, device=y.device)
        on_grid = (part * inverse).double()
        out[:, c:c + 128] = torch.where(most >= TINY, _grid(on_grid) * scale.double(), 0.0)
    return out


def _exact_values(codes, scales, blocks):
    rows = torch.arange(codes.shape[0], device="cuda") // (128 if blocks else 1)
    cols = torch.arange(codes.shape[1], device="cuda") // 128
    return codes.to(torch.float64) * scales.double()[rows][:, cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("score", "train"):
            x, w, t = s["x"].double(), s["w"].double(), s["target"]
            loss = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
            dx, dw = torch.zeros_like(x), torch.zeros_like(w)
            valid = torch.nonzero(t >= 0)[:, 0]
            for rows in valid.split(2048):
                logits = torch.mm(x[rows], w.t())
                logp = torch.log_softmax(logits, 1)
                del logits
                here = torch.arange(rows.numel(), device="cuda"), t[rows]
                loss[rows] = -logp[here]
                if op == "train":
                    grad = logp.exp_()
                    grad[here] -= 1.0
                    grad /= valid.numel()
                    dx[rows] = torch.mm(grad, w)
                    dw.addmm_(grad.t(), x[rows])
            return {"loss": loss} if op == "score" else {"loss": loss.sum() / valid.numel(), "dx": dx, "dw": dw}
        if op == "matmul":
            a = _exact_values(s["a"], s["a_scales"], False)
            b = _exact_values(s["b"], s["b_scales"], case["weight"] == "blocks")
            return {"y": torch.addmm(s["bias"].double(), a, b.t())}
        w = _exact_rounded(s["w"], 128)
        y = torch.addmm(s["bias"].double(), _exact_rounded(s["x"], 1), w.t())
        dx = torch.mm(_exact_rounded(s["dy"], 1), w)
        dw = torch.mm(_exact_rounded(s["dy"].t(), 1), _exact_rounded(s["x"].t(), 1).t())
        return {"y": y, "dx": dx, "dw": dw, "db": s["dy"].double().sum(0)}


def work(case):
    op, rows, cols = case["op"], case["rows"], case["cols"]
    e = 4 if case["type"] == "f32" else 2
    if op in ("score", "train"):
        held = (rows + case["vocab"]) * cols * e
        product = 2 * rows * cols * case["vocab"] * (1 - case["ignored"])
        if op == "score":
            return {"bytes": held + 12 * rows, "flops": product}
        return {"bytes": 2 * held + 8 * rows + 4, "flops": 3 * product}
    out, groups = case["out"], -(-cols // 128)
    if op == "matmul":
        scales = 4 * groups * (rows + (out if case["weight"] == "rows" else -(-out // 128)))
        return {"bytes": rows * cols + out * cols + scales + 4 * out + e * rows * out, "flops": 2 * rows * cols * out}
    return {"bytes": 2 * e * rows * (cols + out) + 8 * out * (cols + 1), "flops": 6 * rows * cols * out}
