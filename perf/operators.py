"""The 8-bit activation path of a sparse MLP block: root-mean-square norm with the residual's addition and an 8-bit output
(and its gradient), 8-bit activation checkpoints (pack, GELU, restore, GELU's gradient), and the sparse layer's forward and
weight gradient on them.

An 8-bit matrix has codes (int8, or 8-bit floats E4M3) and one 32-bit scale for each group of columns of a row (group 0: the
whole row); it stands for scale * code. Codes of 8-bit floats are returned as they are, beside their scales; int8 codes are
returned as the values they stand for.
"""
import math

import torch

own = False

# Smallest magnitude that a group is scaled by; a group below it is held as zeros.
TINY = 2.0 ** -100
TOP = {"int8": 127.0, "e4m3": 448.0}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # the norm before the MLP in a decoding step of one sequence: latency
        {"name": "norm, one token", "op": "norm", "rows": 1, "cols": 768, "type": "f32", "format": "e4m3", "group": 0},
        # the same norm in a training step over 32 sequences of 1024 tokens, the residual stream in 16 bits
        {"name": "norm, training batch", "op": "norm", "rows": 32768, "cols": 768, "type": "bf16", "format": "e4m3", "group": 128},
        # its gradient for a few ragged sequences of a wide model, the stream in 32 bits
        {"name": "norm gradient, ragged", "op": "norm_grad", "rows": 333, "cols": 5000, "type": "f32"},
        # its gradient in the training step
        {"name": "norm gradient, training", "op": "norm_grad", "rows": 32768, "cols": 768, "type": "bf16"},
        # the MLP's activation for one decoding step of 64 sequences
        {"name": "activation, decoding", "op": "act", "rows": 64, "cols": 3072, "type": "f32", "format": "e4m3", "group": 0},
        # the MLP's activation in a training step: the checkpoint of its input and its output, both in 8 bits
        {"name": "activation, training", "op": "act", "rows": 16384, "cols": 3072, "type": "f32", "format": "e4m3", "group": 128},
        # the activation's gradient from that checkpoint
        {"name": "activation gradient", "op": "act_grad", "rows": 16384, "cols": 3072, "type": "f32", "format": "int8", "group": 128},
        # a layer's input kept for the backward pass in int8 and restored there
        {"name": "checkpoint and restore", "op": "keep", "rows": 4096, "cols": 10000, "type": "f32", "format": "int8", "group": 128},
        # the MLP's first layer in a decoding step of one sequence: skewed rows
        {"name": "forward, one token", "op": "forward", "rows": 1, "out": 3072, "cols": 768, "sparsity": 90, "skew": True,
         "format": "int8", "group": 0},
        # the large layer's forward on a small batch
        {"name": "forward, batch 64", "op": "forward", "rows": 64, "out": 10000, "cols": 10000, "sparsity": 90, "skew": False,
         "format": "int8", "group": 0},
        # its weight gradient from a checkpoint, an odd micro-batch
        {"name": "weight gradient, batch 17", "op": "weight_grad", "rows": 17, "out": 10000, "cols": 10000, "sparsity": 95,
         "skew": False, "format": "e4m3", "group": 128},
        # the same in a large-batch step
        {"name": "weight gradient, batch 512", "op": "weight_grad", "rows": 512, "out": 10000, "cols": 10000, "sparsity": 90,
         "skew": False, "format": "int8", "group": 0},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_grad", "act", "act_grad", "keep", "forward", "weight_grad"])
    c = {"op": op}
    if op in ("forward", "weight_grad"):
        c["out"], c["cols"] = spread(256, 10000), spread(256, 10000)
        c["rows"] = spread(1, 512)
        c["sparsity"] = rng.choice([80, 90, 95, 99])
        if c["sparsity"] == 80 and c["out"] * c["cols"] > 50_000_000:
            c["sparsity"] = 90
        c["skew"] = rng.random() < 0.3 and c["out"] * c["cols"] <= 16_000_000
        c["format"], c["group"] = rng.choice(["int8", "e4m3"]), rng.choice([0, 0, 32, 64, 128, 256])
        return c
    c["cols"] = spread(64, 10000)
    if rng.random() < 0.5:  # half the widths of real models are whole multiples of the group
        c["cols"] = max(64, c["cols"] // 64 * 64)
    c["rows"] = spread(1, min(32768, 24_000_000 // c["cols"]))
    c["type"] = rng.choice(["f32", "bf16", "f16"])
    if op != "norm_grad":
        # int8 codes of computed values may differ by one step where a value lies between two; those of given values do not
        c["format"] = "e4m3" if op in ("norm", "act") else rng.choice(["int8", "e4m3"])
        c["group"] = rng.choice([0, 32, 64, 128, 256])
    return c


def _activations(g, rows, cols, dtype, scale=1.0):
    """Normal values with a few columns far larger than the others, as hidden states have them."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    loud = 1.0 + 9.0 * (torch.rand(cols, device="cuda", generator=g) < 0.01)
    return (x * loud * scale).to(dtype)


def _degrees(case):
    """Entries of each row of W: equal, or falling as rank^-1.2 (rows in a fixed mixed order) up to a full row."""
    out, cols = case["out"], case["cols"]
    nnz = max(1, round(out * cols * (100 - case["sparsity"]) / 100))
    if not case["skew"]:
        return [nnz // out + (1 if r < nnz % out else 0) for r in range(out)]
    weight = [(1 + (r * 7919) % out) ** -1.2 for r in range(out)]
    lo, hi = 0.0, float(nnz) * out
    for _ in range(100):  # the factor at which the capped degrees add up to nnz
        mid = (lo + hi) / 2
        lo, hi = (mid, hi) if sum(min(cols, int(mid * w)) for w in weight) < nnz else (lo, mid)
    return [min(cols, int(lo * w)) for w in weight]


def _support(g, case):
    """Row-major (rows, cols) of a support with the case's row degrees, columns drawn without repetition."""
    out, cols = case["out"], case["cols"]
    degree = torch.tensor(_degrees(case), device="cuda")
    most = int(degree.max())
    order = torch.rand(out, cols, device="cuda", generator=g).topk(most, dim=1).indices
    here = torch.arange(most, device="cuda")[None, :] < degree[:, None]
    order = torch.where(here, order, cols).sort(dim=1).values
    rows = torch.arange(out, device="cuda")[:, None].expand(out, most)
    return rows[order < cols].int().contiguous(), order[order < cols].int().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, cols = case["op"], case["rows"], case["cols"]
    s = dict(case)
    dtype = TYPES[case.get("type", "f32")]
    if op == "norm":
        s["x"] = _activations(g, rows, cols, dtype, 0.3)
        s["residual"] = _activations(g, rows, cols, dtype)
        s["gain"] = 1.0 + 0.1 * torch.randn(cols, device="cuda", generator=g)
    elif op == "norm_grad":
        s["total"] = _activations(g, rows, cols, dtype)
        s["gain"] = 1.0 + 0.1 * torch.randn(cols, device="cuda", generator=g)
        s["rstd"] = 1.0 / torch.sqrt(s["total"].float().square().mean(1) + EPS)
        s["dy"] = 1e-3 * torch.randn(rows, cols, device="cuda", generator=g)
        s["dtotal"] = (1e-3 * torch.randn(rows, cols, device="cuda", generator=g)).to(dtype)
    elif op in ("act", "keep"):
        s["x"] = _activations(g, rows, cols, dtype)
    elif op == "act_grad":
        s["da"] = (1e-3 * torch.randn(rows, cols, device="cuda", generator=g)).to(dtype)
        s["codes"], s["scales"] = _pack(_activations(g, rows, cols, torch.float32), case["format"], case["group"])
    else:
        s["w_rows"], s["w_cols"] = _support(g, case)
        s["values"] = torch.randn(s["w_rows"].numel(), device="cuda", generator=g) / math.sqrt(cols * (100 - case["sparsity"]) / 100)
        s["codes"], s["scales"] = _pack(_activations(g, rows, cols, torch.float32), case["format"], case["group"])
        if op == "forward":
            s["bias"] = 0.1 * torch.randn(case["out"], device="cuda", generator=g)
        else:
            s["dy"] = 1e-3 * torch.randn(rows, case["out"], device="cuda", generator=g)
    if own:
        from sparse_linear_layer_gb300 import binding, q8
        s["q8"] = q8
        if "codes" in s:
            s["kept"] = q8.Q8Tensor(s["codes"], s["scales"], case["group"])
        if "values" in s:
            s["layer"] = binding.SparseLinear(case["out"], cols, s["values"], s["w_rows"], s["w_cols"])
    return s


# ------------------------------------------------------------------ plain forms

def _groups(y, group):
    """[rows, groups, group columns], filled up with zeros."""
    rows, cols = y.shape
    group = group or cols
    fill = -cols % group
    if fill:
        y = torch.cat([y, torch.zeros(rows, fill, device=y.device, dtype=y.dtype)], 1)
    return y.reshape(rows, -1, group)


def _pack(y, format, group):
    rows, cols = y.shape
    y = _groups(y.float(), group)
    most = y.abs().amax(2)
    top = torch.full_like(most, TOP[format])
    used = most >= TINY
    scales = torch.where(used, most / top, 0.0)
    code = y * torch.where(used, top / most, 0.0)[:, :, None]
    code = code.reshape(rows, -1)[:, :cols]
    code = torch.round(code).clamp(-127, 127).to(torch.int8) if format == "int8" else code.to(torch.float8_e4m3fn)
    return code.contiguous(), scales


def _unpack(codes, scales, group):
    cols = codes.shape[1]
    each = scales.repeat_interleave(group or cols, 1)[:, :cols]
    return codes.float() * each


def _plain(s):
    op = s["op"]
    if op == "norm":
        total = s["x"] + s["residual"]
        r = total.float()
        rstd = 1.0 / torch.sqrt(r.square().mean(1) + EPS)
        codes, scales = _pack(r * rstd[:, None] * s["gain"], s["format"], s["group"])
        return {"codes": codes, "scales": scales, "total": total, "rstd": rstd}
    if op == "norm_grad":
        n = s["total"].float() * s["rstd"][:, None]
        gdy = s["dy"] * s["gain"]
        dx = s["rstd"][:, None] * (gdy - n * (gdy * n).mean(1, keepdim=True)) + s["dtotal"].float()
        return {"dx": dx.to(s["total"].dtype), "dgain": (s["dy"] * n).sum(0)}
    if op == "act":
        h = s["x"].float()
        kept, kept_scales = _pack(h, s["format"], s["group"])
        codes, scales = _pack(0.5 * h * (1.0 + torch.erf(h * math.sqrt(0.5))), s["format"], s["group"])
        return {"kept": kept, "kept_scales": kept_scales, "codes": codes, "scales": scales}
    if op == "act_grad":
        h = _unpack(s["codes"], s["scales"], s["group"])
        slope = 0.5 * (1.0 + torch.erf(h * math.sqrt(0.5))) + h * torch.exp(-0.5 * h * h) * (1.0 / math.sqrt(2.0 * math.pi))
        return {"dh": (s["da"].float() * slope).to(s["da"].dtype)}
    if op == "keep":
        codes, scales = _pack(s["x"], s["format"], s["group"])
        return {"scales": scales, "values": _unpack(codes, scales, s["group"]).to(s["x"].dtype)}
    x = _unpack(s["codes"], s["scales"], s["group"])
    at = s["w_rows"].long(), s["w_cols"].long()
    if op == "forward":
        w = torch.zeros(s["out"], s["cols"], device="cuda")
        w[at] = s["values"]
        return {"y": x @ w.T + s["bias"]}
    return {"dw": (s["dy"].T @ x)[at], "db": s["dy"].sum(0)}


def run(s):
    if not own:
        return _plain(s)
    q8, op = s["q8"], s["op"]
    if op == "norm":
        q, total, rstd = q8.rmsnorm(s["x"], s["gain"], residual=s["residual"], eps=EPS, format=s["format"], group=s["group"])
        return {"codes": q.codes, "scales": q.scales, "total": total, "rstd": rstd}
    if op == "norm_grad":
        dx, dgain = q8.rmsnorm_backward(s["dy"], s["total"], s["rstd"], s["gain"], dtotal=s["dtotal"])
        return {"dx": dx, "dgain": dgain}
    if op == "act":
        a, kept = q8.gelu(s["x"], format=s["format"], group=s["group"], keep=True)
        return {"kept": kept.codes, "kept_scales": kept.scales, "codes": a.codes, "scales": a.scales}
    if op == "act_grad":
        return {"dh": q8.gelu_backward(s["da"], s["kept"])}
    if op == "keep":
        kept = q8.pack(s["x"], format=s["format"], group=s["group"])
        return {"scales": kept.scales, "values": q8.unpack(kept, s["x"].dtype)}
    if op == "forward":
        return {"y": s["layer"].forward_q8(s["kept"], s["bias"])}
    dw, db = s["layer"].backward_weight_q8(s["kept"], s["dy"], with_bias=True)
    return {"dw": dw, "db": db}


# ------------------------------------------------------------------ 64 bits

def _grid(v, format):
    """The nearest code value, halves to even."""
    if format == "int8":
        return torch.round(v)
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -6))
    step = torch.ldexp(torch.ones_like(v), e - 4)  # three bits after the leading one
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_pack(y, format, group):
    rows, cols = y.shape
    width = group or cols
    codes, scales = torch.empty_like(y), []
    for c in range(0, cols, width):
        part = y[:, c:c + width]
        most = part.abs().max(1, keepdim=True).values
        scale = torch.where(most >= TINY, most / TOP[format], 0.0)
        codes[:, c:c + width] = torch.where(scale > 0, _grid(part / torch.where(scale > 0, scale, 1.0), format), 0.0)
        scales.append(scale)
    return codes, torch.cat(scales, 1)


def _exact_values(s, group):
    at = torch.arange(s["cols"], device="cuda") // (group or s["cols"])
    return s["codes"].to(torch.float64) * s["scales"].double()[:, at]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = (s["x"].double() + s["residual"].double())
        rounded = total.to(s["x"].dtype).double()
        rstd = (rounded.pow(2).sum(1) / case["cols"] + EPS).rsqrt()
        codes, scales = _exact_pack(rounded * rstd[:, None] * s["gain"].double(), case["format"], case["group"])
        return {"codes": codes, "scales": scales, "total": total, "rstd": rstd}
    if op == "norm_grad":
        # y_j = gain_j r_j / sqrt(mean(r^2) + eps): its Jacobian's transpose, applied to dy
        r, rstd, gdy = s["total"].double(), s["rstd"].double()[:, None], s["dy"].double() * s["gain"].double()
        along = (gdy * r).sum(1, keepdim=True) * rstd ** 3 / case["cols"]
        return {"dx": gdy * rstd - along * r + s["dtotal"].double(), "dgain": torch.einsum("tc,tc->c", s["dy"].double(), r * rstd)}
    if op == "act":
        h = s["x"].double()
        kept, kept_scales = _exact_pack(h, case["format"], case["group"])
        codes, scales = _exact_pack(h * 0.5 * torch.erfc(-h / math.sqrt(2.0)), case["format"], case["group"])
        return {"kept": kept, "kept_scales": kept_scales, "codes": codes, "scales": scales}
    if op == "act_grad":
        h = _exact_values(s, case["group"])
        slope = 0.5 * torch.erfc(-h / math.sqrt(2.0)) + h * torch.exp(-h * h / 2) / math.sqrt(2.0 * math.pi)
        return {"dh": slope * s["da"].double()}
    if op == "keep":
        codes, scales = _exact_pack(s["x"].double(), case["format"], case["group"])
        at = torch.arange(case["cols"], device="cuda") // (case["group"] or case["cols"])
        return {"scales": scales, "values": codes * scales[:, at]}
    x = _exact_values(s, case["group"])
    at = s["w_rows"].long() * case["cols"] + s["w_cols"].long()
    if op == "forward":
        w = torch.zeros(case["out"] * case["cols"], device="cuda", dtype=torch.float64)
        w.scatter_(0, at, s["values"].double())
        return {"y": torch.addmm(s["bias"].double(), x, w.view(case["out"], case["cols"]).T)}
    whole = torch.mm(s["dy"].double().T, x).reshape(-1)
    return {"dw": whole.gather(0, at), "db": s["dy"].double().sum(0)}


def work(case):
    op, rows, cols = case["op"], case["rows"], case["cols"]
    e = 4 if case.get("type", "f32") == "f32" else 2
    n = rows * cols
    scales = 4 * rows * -(-cols // (case.get("group") or cols))
    if op == "norm":
        return {"bytes": n * (3 * e + 1) + scales + 4 * rows + 4 * cols, "flops": 6 * n}
    if op == "norm_grad":
        return {"bytes": n * (4 + 3 * e) + 4 * rows + 8 * cols, "flops": 9 * n}
    if op == "act":
        return {"bytes": n * (e + 2) + 2 * scales, "flops": 8 * n}
    if op == "act_grad":
        return {"bytes": n * (1 + 2 * e) + scales, "flops": 8 * n}
    if op == "keep":
        return {"bytes": n * (2 * e + 2) + 2 * scales, "flops": 4 * n}
    # a stored weight is its value (or gradient) in 32 bits and its column in 16
    nnz = sum(_degrees(case))
    return {"bytes": 6 * nnz + n + scales + 4 * rows * case["out"], "flops": 2 * nnz * rows}
