"""A weight gradient of no batch rows is a sum over nothing: zero, not what its
memory held before."""
import pytest

from sparse_linear_layer_gb300 import synth
from tests.gpu_util import make_gpu_layer, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


def spoiled(torch, *sizes):
    """Leave NaN in the blocks that the next tensors of these sizes take."""
    blocks = [torch.full((n,), float("nan"), device="cuda") for n in sizes for _ in range(4)]
    del blocks


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_weight_gradient_on_8_bits(torch, fmt, group):
    from sparse_linear_layer_gb300 import binding, q8
    g = make_gpu_layer(torch, synth.make_layer(70, 50, 80, 0.1, 301, 302))
    x = q8.pack(torch.empty(0, 50, device="cuda"), fmt, group)
    dy = torch.empty(0, 70, device="cuda")
    dw, db = (torch.full((n,), float("nan"), device="cuda") for n in (g.nnz, 70))
    binding.snk_backward_weight_q8(g.handle, x.codes, x.scales, x.format_id, group, dy, 0, dw, db)
    assert (dw == 0).all() and (db == 0).all()
    dw.fill_(float("nan"))
    binding.snk_backward_weight_q8(g.handle, x.codes, x.scales, x.format_id, group, dy, 0, dw)
    assert (dw == 0).all()
    spoiled(torch, g.nnz, 70)
    dw, db = g.backward_weight_q8(x, dy, with_bias=True)
    assert (dw == 0).all() and (db == 0).all()
    g.close()


def test_block(torch):
    from sparse_linear_layer_gb300.mlp import SparseMLP
    block = SparseMLP(96, 160, 0.8)
    x = torch.empty(0, 96, device="cuda", requires_grad=True)
    y, total = block(x, torch.empty(0, 96, device="cuda"))
    spoiled(torch, block.up.nnz, block.down.nnz, 160, 96)
    (y.sum() + total.sum()).backward()
    assert x.grad.shape == (0, 96)
    for p in block.parameters():
        assert (p.grad == 0).all()
    block.close()


def test_layer_that_keeps_8_bits(torch):
    from sparse_linear_layer_gb300.module import SparseLinear
    layer = SparseLinear(96, 160, 0.8, keep="int8")
    y = layer(torch.empty(0, 96, device="cuda"))
    spoiled(torch, layer.nnz, 160)
    y.sum().backward()
    assert (layer.values.grad == 0).all() and (layer.bias.grad == 0).all()
    layer.close()


def test_weight_gradient_in_fp32(torch):
    from sparse_linear_layer_gb300 import binding
    g = make_gpu_layer(torch, synth.make_layer(70, 50, 80, 0.1, 303, 304))
    x, dy = torch.empty(0, 50, device="cuda"), torch.empty(0, 70, device="cuda")
    dw, db = (torch.full((n,), float("nan"), device="cuda") for n in (g.nnz, 70))
    binding.snk_backward_weight(g.handle, x, dy, dw, db)
    assert (dw == 0).all() and (db == 0).all()
    spoiled(torch, g.nnz, 70)
    dw, db = g.backward_weight(x, dy, with_bias=True)
    assert (dw == 0).all() and (db == 0).all()
    g.close()


def test_layer(torch):
    from sparse_linear_layer_gb300.module import SparseLinear
    layer = SparseLinear(96, 160, 0.8)
    y = layer(torch.empty(0, 96, device="cuda"))
    spoiled(torch, layer.nnz, 160)
    y.sum().backward()
    assert (layer.values.grad == 0).all() and (layer.bias.grad == 0).all()
    layer.close()
