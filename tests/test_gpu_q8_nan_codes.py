"""E4M3 has a NaN code.  No call of this library writes it, but a matrix made
elsewhere may hold it (a cast that overflowed): it reaches the outputs whose
entries lie in its column, and no others, on every path."""
import numpy as np
import pytest

import oracle
from sparse_linear_layer_gb300 import synth
from tests.gpu_util import assert_within, dev, host, make_gpu_layer, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.mark.parametrize("large", ["on", "off", ""])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("b", [4, 130])
def test_forward_and_weight_gradient(torch, monkeypatch, large, group, b):
    from sparse_linear_layer_gb300 import q8
    monkeypatch.setenv("SNK_LARGE_BATCH", large)
    lay = synth.make_layer(150, 200, 90, 0.1, 311, 312)
    g = make_gpu_layer(torch, lay)
    rng = np.random.default_rng(313)
    q = q8.pack(dev(rng.standard_normal((b, 200)).astype(np.float32), torch), "e4m3", group)
    codes = q.codes.view(torch.uint8)
    codes[1, 7] = 0x7F
    codes[3, 199] = 0xFF
    x = host(q8.unpack(q))
    assert np.isnan(x).sum() == 2
    dy = rng.standard_normal((b, 150)).astype(np.float32)
    y = g.forward_q8(q)
    dw, db = g.backward_weight_q8(q, dev(dy, torch), with_bias=True)
    can = oracle.canonicalize(150, 200, lay.values, lay.rows, lay.cols)
    v, r, c = can["values"], can["rows"], can["cols"]
    with np.errstate(all="ignore"):
        yr, ay = oracle.forward(150, 200, v, r, c, x, None)
        dwr, aw, dbr, ab = oracle.backward_weight(150, 200, r, c, x, dy)
    assert_within(host(y), yr, ay, "forward_q8")
    assert_within(host(dw), dwr, aw, "backward_weight_q8")
    assert_within(host(db), dbr, ab, "db")
    g.close()
