"""The sparse MLP block on 8-bit activations, and a sparse layer that keeps its
input in 8 bits, against 64-bit references step by step: every step is checked on
the block's own inputs to it (roundings to 8 bits would otherwise carry one
step's difference into the next).  Tolerances: the layers' own (1e-5 * A +
1e-6); the norm's gradient 96 u times the sum of its terms' magnitudes (u =
2^-24) and half a unit of the stream's type; GELU's slope 32 u (1 + |h|)."""
import numpy as np
import pytest

import oracle
from tests import q8_ref as ref
from tests.gpu_util import assert_within, dev, host, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


def triple(layer):
    return host(layer.values.detach()), host(layer.rows), host(layer.cols)


@pytest.mark.parametrize("rows", [1, 6, 130])
@pytest.mark.parametrize("dtype,fmt,group", [("float32", "int8", 0), ("bfloat16", "int8", 64),
                                             ("float32", "e4m3", 128), ("float16", "e4m3", 0)])
def test_block_step_by_step(torch, rows, dtype, fmt, group):
    from sparse_linear_layer_gb300 import q8
    from sparse_linear_layer_gb300.mlp import SparseMLP
    torch.manual_seed(3)
    d, f, eps = 200, 328, 1e-5
    dt = getattr(torch, dtype)
    m = SparseMLP(d, f, 0.9, eps=eps, format=fmt, group=group, seed=5)
    with torch.no_grad():
        m.gain.add_(0.1 * torch.randn_like(m.gain))
        m.up.bias.add_(0.1 * torch.randn_like(m.up.bias))
        m.down.bias.add_(0.1 * torch.randn_like(m.down.bias))
    x = torch.randn(rows, d, device="cuda").to(dt).requires_grad_(True)
    r = torch.randn(rows, d, device="cuda").to(dt).requires_grad_(True)
    gy = torch.randn(rows, d, device="cuda").to(dt)
    gt = torch.randn(rows, d, device="cuda").to(dt)
    y, total = m(x, r)
    torch.autograd.backward((y, total), (gy, gt))
    assert torch.equal(total, (x + r).detach()) and y.dtype == dt

    # the block's own intermediate matrices, from the same calls
    n, _, rstd = q8.rmsnorm(x.detach(), m.gain.detach(), residual=r.detach(), eps=eps, format=fmt, group=group)
    nv = host(q8.unpack(n))
    up, down = triple(m.up), triple(m.down)
    h = m.up._h.forward_q8(n, m.up.bias.detach())
    hr, ah = oracle.forward(f, d, *up, nv, host(m.up.bias.detach()))
    assert_within(host(h), hr, ah, "up")
    a, kept = q8.gelu(h, fmt, group, keep=True)
    av, hk = host(q8.unpack(a)), host(q8.unpack(kept)).astype(np.float64)
    yr, ay = oracle.forward(d, f, *down, av, host(m.down.bias.detach()))
    yb = m.down._h.forward_q8(a, m.down.bias.detach())
    assert_within(host(yb), yr, ay, "down")
    assert torch.equal(yb.to(dt), y)

    dy = gy.float()
    dyh = host(dy)
    dwr, aw, dbr, ab = oracle.backward_weight(d, f, *down[1:], av, dyh)
    assert_within(host(m.down.values.grad), dwr, aw, "down values")
    assert_within(host(m.down.bias.grad), dbr, ab, "down bias")
    da = host(m.down._h.backward_input(dy)).astype(np.float64)
    dar, aa = oracle.backward_input(d, f, *down, dyh)
    assert_within(da, dar, aa, "da")
    dh = q8.gelu_backward(m.down._h.backward_input(dy), kept)
    want = da * ref.gelu_slope(hk)
    assert (np.abs(host(dh) - want) <= 32 * U * np.abs(da) * (1 + np.abs(hk)) + U * np.abs(want) + 1e-40).all()
    dwr, aw, dbr, ab = oracle.backward_weight(f, d, *up[1:], nv, host(dh))
    assert_within(host(m.up.values.grad), dwr, aw, "up values")
    assert_within(host(m.up.bias.grad), dbr, ab, "up bias")
    dn = host(m.up._h.backward_input(dh)).astype(np.float64)
    dnr, an = oracle.backward_input(f, d, *up, host(dh))
    assert_within(dn, dnr, an, "dn")
    f8 = lambda t: t.detach().double().cpu().numpy()
    wx, wg, ax, ag = ref.rmsnorm_backward(dn, f8(total), f8(rstd), f8(m.gain), f8(gt))
    half = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}[dtype]
    for t in (x, r):
        assert (np.abs(f8(t.grad) - wx) <= 96 * U * ax + half * np.abs(wx) + 2.0 ** -25 * (dtype == "float16")).all()
    assert (np.abs(f8(m.gain.grad) - wg) <= (rows + 64) * U * ag + 1e-40).all()
    m.close()


def test_block_without_residual_and_unused_outputs(torch):
    from sparse_linear_layer_gb300.mlp import SparseMLP
    m = SparseMLP(64, 96, 0.5, bias=False, group=32)
    x = torch.randn(2, 3, 64, device="cuda", requires_grad=True)
    y = m(x)
    y.sum().backward()
    alone = x.grad.clone()
    assert y.shape == x.shape and torch.isfinite(alone).all()
    x.grad = None
    r = torch.zeros(2, 3, 64, device="cuda", requires_grad=True)
    y2, total = m(x, r)
    assert torch.equal(y2, y) and torch.equal(total, x)
    y2.sum().backward()
    assert torch.equal(x.grad, alone) and torch.equal(r.grad, alone)
    x.grad = None
    _, total = m(x, r)
    total.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))
    m.close()


def test_training_loss_falls_and_set_restructures(torch):
    """A stack of two blocks on the residual stream; SET restructures the layers."""
    from sparse_linear_layer_gb300.mlp import SparseMLP
    from sparse_linear_layer_gb300.module import SET
    torch.manual_seed(1)
    blocks = torch.nn.ModuleList([SparseMLP(96, 256, 0.8, seed=7 + 10 * i, group=32) for i in range(2)])
    opt = torch.optim.Adam(blocks.parameters(), lr=3e-3)
    algo = SET([s for b in blocks for s in b.sparse_layers()], zeta=0.2, every=20)
    x = torch.randn(48, 96, device="cuda")
    target = torch.randn(48, 96, device="cuda")
    losses = []
    for _ in range(60):
        opt.zero_grad()
        y, total = blocks[0](x, torch.zeros_like(x))
        y, total = blocks[1](y, total)
        loss = ((y + total - target) ** 2).mean()
        loss.backward()
        opt.step()
        algo.step()
        losses.append(float(loss.detach()))
    assert algo.restructures == 3 and losses[-1] < 0.5 * losses[0], losses[::10]
    for b in blocks:
        b.close()


@pytest.mark.parametrize("keep,group", [("int8", 0), ("e4m3", 64)])
def test_layer_that_keeps_its_input_in_8_bits(torch, keep, group):
    from sparse_linear_layer_gb300.module import SparseLinear
    in_f, out_f, b = 300, 200, 9
    full = SparseLinear(in_f, out_f, 0.9, seed=31)
    m = SparseLinear(in_f, out_f, 0.9, seed=31, keep=keep, keep_group=group)
    x = torch.randn(b, in_f, device="cuda")
    g = torch.randn(b, out_f, device="cuda")
    xs = [x.clone().requires_grad_(True) for _ in range(2)]
    ys = [layer(t) for layer, t in ((full, xs[0]), (m, xs[1]))]
    held = [t for t in ys[1].grad_fn.saved_tensors]
    assert [t.element_size() for t in held] == [1, 4] and held[0].shape == (b, in_f)
    for y in ys:
        y.backward(g)
    assert torch.equal(ys[0], ys[1]) and torch.equal(xs[0].grad, xs[1].grad)
    codes, scales = ref.pack(host(x), keep, group)
    v, r, c = triple(m)
    dwr, aw, dbr, ab = oracle.backward_weight(out_f, in_f, r, c, ref.values(codes, scales, group).astype(np.float32),
                                              host(g))
    assert_within(host(m.values.grad), dwr, aw, "values grad")
    assert_within(host(m.bias.grad), dbr, ab, "bias grad")
    with pytest.raises(ValueError):
        SparseLinear(in_f, out_f, 0.9, keep="fp4")
    full.close()
    m.close()
