"""The dense operators at the edges of what their calls take: very long rows and sums, upstream
gradients at the ends of fp32, forward-mode differentiation, layers converted to 16 bits, and the
entry points by the names of the C calls."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_linear_layer_gb300 import dense  # noqa: E402
from tests.gpu_util import need_gpu  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("cols", [11_863_040, 11_863_048, 12_000_000])
def test_loss_of_rows_whose_turns_pass_32_bits(cols):
    """cols / 64 stages in turns of 16: from 11 863 041 columns on the stages' number times the turns is 2^31
    and more.

    Every column holds the same numbers, so that a logit is cols * x w exactly.  Sums of a turn truncate, toward
    zero: 64 steps, each by less than 2^-23 of the turn's sum, then cols / 1024 additions in fp32 and those of the
    target's dot product (cols / 256 a lane) of half a unit of the sum each, which random signs do not average
    where all terms are equal: the logits' relative error is below (64 * 2 + 0.005 * cols) * 2^-24."""
    x = torch.full((2, cols), 2.0 ** -12, device="cuda", dtype=torch.bfloat16)
    w = torch.empty(3, cols, device="cuda", dtype=torch.bfloat16)
    w.copy_(torch.tensor([[0.0], [2.0 ** -12], [-(2.0 ** -11)]], device="cuda"))
    target = torch.tensor([0, 1], device="cuda")
    got = dense.linear_cross_entropy(x, w, target, reduction="none").double()
    z = torch.tensor([0.0, cols * 2.0 ** -24, -cols * 2.0 ** -23], device="cuda", dtype=torch.float64)
    want = z.logsumexp(0) - z[:2]
    tol = 2 * (128 + 0.005 * cols) * 2.0 ** -24 * z.abs().max() + 1e-6
    assert tol < 0.05 and bool(((got - want).abs() <= tol).all()), (got, want, tol)
