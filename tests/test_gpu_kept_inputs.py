"""What the block and the layer keep in 8 bits between the passes: in the form of
the forward pass, and only for a backward pass that will read it."""
import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("before,after", [(("int8", 32), (None, 0)), ((None, 0), ("int8", 32)),
                                          (("int8", 0), ("int8", 64)), (("e4m3", 64), ("int8", 0))])
def test_layer_changed_between_the_passes(torch, before, after, bias):
    from sparse_linear_layer_gb300.module import SparseLinear
    layer = SparseLinear(200, 130, 0.9, bias=bias, seed=41, keep=before[0], keep_group=before[1])
    x, gy = torch.randn(7, 200, device="cuda"), torch.randn(7, 130, device="cuda")
    grads = []
    for changed in (False, True):
        xs = x.clone().requires_grad_(True)
        y = layer(xs)
        if changed:
            layer.keep, layer.keep_group = after
        layer.values.grad = None
        y.backward(gy)
        grads.append((xs.grad, layer.values.grad))
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])
    layer.close()


def test_block_changed_between_the_passes(torch):
    from sparse_linear_layer_gb300.mlp import SparseMLP
    block = SparseMLP(96, 200, 0.8, format="int8", group=32, seed=43)
    x, r, gy = (torch.randn(9, 96, device="cuda") for _ in range(3))
    grads = []
    for changed in (False, True):
        xs = x.clone().requires_grad_(True)
        y, _ = block(xs, r)
        if changed:
            block.format, block.group = "e4m3", 0
        block.zero_grad()
        y.backward(gy)
        grads.append([xs.grad] + [p.grad for p in block.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    block.close()


@pytest.fixture
def calls(torch, monkeypatch):
    """The 8-bit matrices that the calls write for a backward pass."""
    from sparse_linear_layer_gb300 import q8
    made = []
    gelu, pack = q8.gelu, q8.pack

    def gelu_seen(*a, keep=False, **k):
        made.extend(["gelu"] * keep)
        return gelu(*a, keep=keep, **k)

    monkeypatch.setattr(q8, "gelu", gelu_seen)
    monkeypatch.setattr(q8, "pack", lambda *a, **k: (made.append("pack"), pack(*a, **k))[1])
    return made


def test_nothing_is_kept_without_a_backward_pass(torch, calls):
    from sparse_linear_layer_gb300.mlp import SparseMLP
    from sparse_linear_layer_gb300.module import SparseLinear
    block = SparseMLP(96, 200, 0.8, seed=45)
    layer = SparseLinear(96, 200, 0.8, seed=47, keep="int8")
    x, r = (torch.randn(9, 96, device="cuda") for _ in range(2))
    with torch.no_grad():
        y0, t0 = block(x, r)
        z0 = layer(x)
        assert not y0.requires_grad and not z0.requires_grad
    with torch.inference_mode():
        block(x)
        layer(x)
    assert calls == []
    y1, t1 = block(x, r)
    z1 = layer(x)
    assert calls == ["gelu", "pack"]
    assert torch.equal(y0, y1) and torch.equal(t0, t1) and torch.equal(z0, z1)
    layer.values.requires_grad_(False)
    layer.bias.requires_grad_(False)
    xs = x.clone().requires_grad_(True)
    layer(xs).sum().backward()   # the input's gradient does not read the input
    assert xs.grad is not None and calls == ["gelu", "pack"]
    block.close()
    layer.close()


@pytest.mark.parametrize("training", [["x"], ["residual"], ["gain"], ["up.values"], ["up.bias"], ["down.values"],
                                      ["down.bias"], ["gain", "down.values"], ["x", "up.values", "down.bias"]])
def test_block_computes_the_gradients_that_are_needed(torch, calls, monkeypatch, training):
    """Of a partly frozen block: the same bits as of the whole one, no checkpoint or
    product that only the frozen parts would read, nothing else set."""
    from sparse_linear_layer_gb300 import binding, q8
    from sparse_linear_layer_gb300.mlp import SparseMLP
    block = SparseMLP(96, 200, 0.8, group=32, seed=49)
    x, r, gy, gt = (torch.randn(9, 96, device="cuda") for _ in range(4))

    def step(names):
        leaves = dict(block.named_parameters(), x=x.clone(), residual=r.clone())
        for k in list(leaves):
            leaves[k].requires_grad_(k in names)
            leaves[k].grad = None
        y, total = block(leaves["x"], leaves["residual"])
        torch.autograd.backward([t for t in (y, total) if t.requires_grad],
                                [g for t, g in ((y, gy), (total, gt)) if t.requires_grad])
        return {k: t.grad for k, t in leaves.items()}

    whole = step(["x", "residual", "gain", "up.values", "up.bias", "down.values", "down.bias"])
    assert all(g is not None for g in whole.values())
    del calls[:]
    made = []
    for cls, names in ((binding.SparseLinear, ("backward_weight_q8", "backward_input")), (q8, ("rmsnorm_backward",))):
        for name in names:
            f = getattr(cls, name)
            monkeypatch.setattr(cls, name, lambda *a, f=f, name=name, **k: (made.append(name), f(*a, **k))[1])
    some = step(training)
    assert {k for k, g in some.items() if g is not None} == set(training)
    assert all(torch.equal(some[k], whole[k]) for k in training)
    stream = bool({"x", "residual", "gain"} & set(training))
    first = bool({"up.values", "up.bias"} & set(training))
    second = bool({"down.values", "down.bias"} & set(training))
    assert calls == ["gelu"] * (stream or first)
    assert made.count("backward_weight_q8") == first + second and made.count("rmsnorm_backward") == stream
    assert made.count("backward_input") == (stream or first) + stream
    block.close()


@pytest.mark.parametrize("keep,group", [("int8", 0), ("e4m3", 64)])
def test_layer_on_an_existing_triple_keeps_its_input(torch, keep, group):
    from sparse_linear_layer_gb300.module import SparseLinear
    a = SparseLinear(200, 130, 0.9, seed=51, keep=keep, keep_group=group)
    b = SparseLinear.from_triple(200, 130, a.values.detach().clone(), a.rows.clone(), a.cols.clone(), keep=keep,
                                 keep_group=group)
    x, gy = torch.randn(7, 200, device="cuda"), torch.randn(7, 130, device="cuda")
    for layer in (a, b):
        y = layer(x)
        assert [t.element_size() for t in y.grad_fn.saved_tensors] == [1, 4]
        y.backward(gy)
    assert torch.equal(a.values.grad, b.values.grad)
    with pytest.raises(ValueError):
        SparseLinear.from_triple(200, 130, a.values.detach(), a.rows, a.cols, keep="int4")
    a.close()
    b.close()


def test_block_of_existing_layers(torch):
    """Skewed triples in a block: the products of its layers on its own 8-bit
    matrices."""
    from sparse_linear_layer_gb300 import q8, synth
    from sparse_linear_layer_gb300.mlp import SparseMLP
    from sparse_linear_layer_gb300.module import SparseLinear

    def layer(out_f, in_f, seed):
        lay = synth.make_layer(out_f, in_f, 90, 0.1, seed, seed + 1, zipf_s=1.2)
        t = [torch.from_numpy(a).cuda() for a in (lay.values, lay.rows, lay.cols)]
        return SparseLinear.from_triple(in_f, out_f, *t)

    up, down = layer(200, 96, 61), layer(96, 200, 63)
    block = SparseMLP.from_layers(up, down, group=32)
    x = torch.randn(9, 96, device="cuda", requires_grad=True)
    y = block(x)
    n, _, _ = q8.rmsnorm(x.detach(), block.gain.detach(), group=32)
    a = q8.gelu(up._h.forward_q8(n, up.bias.detach()), group=32)
    assert torch.equal(y, down._h.forward_q8(a, down.bias.detach()))
    y.sum().backward()
    assert {k for k, p in block.named_parameters() if p.grad is not None} == {
        "gain", "up.values", "up.bias", "down.values", "down.bias"}
    with pytest.raises(ValueError):
        SparseMLP.from_layers(up, up)
    block.close()
