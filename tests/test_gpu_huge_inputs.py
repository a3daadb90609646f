"""Rows of X near the end of fp32's range: outputs that fp32 holds are finite and
right in the large-batch forward too, whose scaled sums are far larger than they."""
import numpy as np
import pytest

import oracle
from sparse_linear_layer_gb300 import synth
from tests.gpu_util import RTOL_A, dev, host, make_gpu_layer, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.mark.parametrize("large", ["on", "off"])
@pytest.mark.parametrize("kept", [("int8", 0), ("e4m3", 0), ("int8", 32), None])
def test_forward(torch, monkeypatch, large, kept):
    from sparse_linear_layer_gb300 import q8
    monkeypatch.setenv("SNK_LARGE_BATCH", large)
    lay = synth.make_layer(150, 200, 90, 1e-3, 331, 332)
    g = make_gpu_layer(torch, lay)
    x = np.random.default_rng(333).standard_normal((130, 200)).astype(np.float32)
    x[1] *= np.float32(1e33)
    x[2] *= np.float32(1e36)
    x[3] *= np.float32(3e37)
    x[4] *= np.float32(1e-30)
    if kept:
        q = q8.pack(dev(x, torch), *kept)
        x = host(q8.unpack(q))
        y = host(g.forward_q8(q))
    else:
        y = host(g.forward(dev(x, torch)))
    can = oracle.canonicalize(150, 200, lay.values, lay.rows, lay.cols)
    yr, a = oracle.forward(150, 200, can["values"], can["rows"], can["cols"], x, None)
    assert np.isfinite(yr).all() and np.abs(yr).max() > 1e34
    assert (np.abs(y - yr) <= RTOL_A * a + 1e-6).all(), [float(np.abs(y - yr)[r].max()) for r in range(5)]
    g.close()
