"""Forward-mode differentiation is refused, not dropped: a dual tensor needs no gradient, and a result
without a tangent would count as a derivative of zero."""
import pytest

torch = pytest.importorskip("torch")
import torch.autograd.forward_ad as fwd  # noqa: E402

from sparse_linear_layer_gb300 import build, dense  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def inputs(device):
    x, w = torch.randn(4, 16, device=device), torch.randn(8, 16, device=device)
    return x, w, torch.zeros(8, device=device), torch.zeros(4, dtype=torch.int64, device=device)


def refused(device):
    x, w, b, t = inputs(device)
    with fwd.dual_level():
        def dual(v):
            return fwd.make_dual(v, torch.ones_like(v))
        for args in ((dual(x), w, b), (x, dual(w), b), (x, w, dual(b)), (dual(x.clone().requires_grad_()), w, b)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                dense.linear_q8(*args)
        for args in ((dual(x.bfloat16()), w.bfloat16(), t), (x.bfloat16(), dual(w.bfloat16()), t)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                dense.linear_cross_entropy(*args)
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                dense.linear_cross_entropy(*args)


def test_tangents_are_refused():
    refused("cpu")


@pytest.mark.gpu
def test_tangents_are_refused_on_the_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    refused("cuda")
    x, w, b, t = inputs("cuda")
    with fwd.dual_level():   # a level without dual inputs changes nothing, nor do tangents where they are switched off
        assert dense.linear_q8(x, w, b).shape == (4, 8)
        with fwd._set_fwd_grad_enabled(False):
            assert dense.linear_q8(fwd.make_dual(x, torch.ones_like(x)), w, b).shape == (4, 8)
    assert torch.isfinite(dense.linear_cross_entropy(x.bfloat16(), w.bfloat16(), t))
