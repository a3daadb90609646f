"""One, two and three rows with group scales on both sides of the width from which
the forward reads an fp32 copy of one or two rows instead of the codes."""
import pytest

from sparse_linear_layer_gb300 import synth
from tests.gpu_util import need_gpu
from tests.test_gpu_q8_layer import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.mark.parametrize("fmt,group", [("int8", 32), ("e4m3", 128), ("int8", 0)])
@pytest.mark.parametrize("b", [1, 2, 3])
@pytest.mark.parametrize("in_f", [5999, 6000, 7003])
def test_forward_and_weight_gradient(torch, fmt, group, b, in_f):
    check(torch, synth.make_layer(300, in_f, 95, 0.1, 321, 322), b, fmt, group, 323)
