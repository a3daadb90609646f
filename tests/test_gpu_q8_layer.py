"""The sparse layer's forward and weight gradient on an 8-bit X, against the
oracle on the values that the matrix stands for, within the layer's own
tolerance 1e-5 * A + 1e-6: every batch tile, wide operands (column bands and
the transposed copy), the tensor-core path, and groups whose scale is NaN."""
import numpy as np
import pytest

import oracle
from sparse_linear_layer_gb300 import synth
from tests import q8_ref as ref
from tests.gpu_util import assert_within, dev, host, make_gpu_layer, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


def q8_input(torch, rng, b, cols, fmt, group, spoil=None):
    """An 8-bit matrix on the GPU and its values."""
    from sparse_linear_layer_gb300 import q8
    x = rng.standard_normal((b, cols)).astype(np.float32)
    x *= (1 + 9 * (rng.random(cols) < 0.02)).astype(np.float32)
    if spoil:
        spoil(x)
    q = q8.pack(dev(x, torch), fmt, group)
    with np.errstate(all="ignore"):
        v = host(q8.unpack(q))
    codes, scales = ref.pack(x, fmt, group)
    assert np.array_equal(v, ref.values(codes, scales, group).astype(np.float32), equal_nan=True)
    return q, v


def check(torch, lay, b, fmt, group, seed, spoil=None, bias=True):
    rng = np.random.default_rng(seed)
    g = make_gpu_layer(torch, lay)
    q, x = q8_input(torch, rng, b, lay.in_f, fmt, group, spoil)
    dy = rng.standard_normal((b, lay.out_f)).astype(np.float32)
    bi = (0.1 * rng.standard_normal(lay.out_f)).astype(np.float32) if bias else None
    y = g.forward_q8(q, dev(bi, torch) if bias else None)
    dw, db = g.backward_weight_q8(q, dev(dy, torch), with_bias=True)
    can = oracle.canonicalize(lay.out_f, lay.in_f, lay.values, lay.rows, lay.cols)
    v, r, c = can["values"], can["rows"], can["cols"]
    with np.errstate(all="ignore"):
        yr, ay = oracle.forward(lay.out_f, lay.in_f, v, r, c, x, bi)
        dwr, aw, dbr, ab = oracle.backward_weight(lay.out_f, lay.in_f, r, c, x, dy)
    assert_within(host(y), yr, ay, "forward_q8")
    assert_within(host(dw), dwr, aw, "backward_weight_q8")
    assert_within(host(db), dbr, ab, "db")
    # the same bits again, and on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = g.forward_q8(q, dev(bi, torch) if bias else None)
        dw2 = g.backward_weight_q8(q, dev(dy, torch))
    side.synchronize()
    np.testing.assert_array_equal(host(y).view(np.uint32), host(y2).view(np.uint32))
    np.testing.assert_array_equal(host(dw).view(np.uint32), host(dw2).view(np.uint32))
    g.close()


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 32), ("e4m3", 128), ("int8", 256)])
@pytest.mark.parametrize("b", [1, 2, 3, 4, 7, 8, 16, 17, 33, 64, 65])
def test_batch_tiles(torch, fmt, group, b):
    lay = synth.make_layer(300, 203, 90, 0.1, 201, 202)
    check(torch, lay, b, fmt, group, 203 + b)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 32), ("e4m3", 128)])
@pytest.mark.parametrize("b", [33, 64, 65])
def test_wide_batch_tiles(torch, monkeypatch, fmt, group, b):
    """The 64-row tiles, which a layer of few entries leaves by itself at b > 32."""
    monkeypatch.setenv("SNK_LARGE_BATCH", "off")
    check(torch, synth.make_layer(300, 203, 90, 0.1, 201, 202), b, fmt, group, 203 + b)
    check(torch, synth.make_layer(96, 1003, 95, 0.1, 204, 205), b, fmt, group, 206 + b)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 32), ("e4m3", 64), ("int8", 256)])
@pytest.mark.parametrize("b", [33, 127, 192, 193, 256, 257, 400])
def test_few_entries(torch, fmt, group, b):
    """Layers of few entries at b > 32: passes of 256 (192) batch rows, rows of W
    without entries, long rows, widths that are no whole words."""
    check(torch, synth.make_layer(300, 203, 90, 0.1, 301, 302), b, fmt, group, 303 + b)
    check(torch, synth.make_layer(700, 64, 99, 0.1, 304, 305), b, fmt, group, 306 + b, bias=False)
    check(torch, synth.make_layer(97, 1240, 95, 0.1, 307, 308, zipf_s=1.2), b, fmt, group, 309 + b)


def test_few_entries_and_spoiled_rows(torch):
    def spoil(x):
        x[3] = 0
        x[5, 70] = np.inf
        x[200, 3] = np.nan
        x[7] *= np.float32(1e-20)

    for fmt, group in (("int8", 0), ("e4m3", 32)):
        check(torch, synth.make_layer(150, 200, 99, 0.1, 311, 312), 300, fmt, group, 313, spoil)


@pytest.mark.parametrize("shape", [(1, 1), (1, 700), (700, 1), (97, 1003), (64, 64)])
def test_odd_shapes(torch, shape):
    out_f, in_f = shape
    lay = synth.make_layer(out_f, in_f, 50, 0.1, 211, 212)
    for b in (1, 5, 40):
        check(torch, lay, b, "int8", 0, 213 + b, bias=False)
        check(torch, lay, b, "e4m3", 32, 214 + b)


@pytest.mark.parametrize("b", [8, 16, 33, 64])
@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 128)])
def test_wide_operand(torch, b, fmt, group):
    """in = 10000: the operand of 8 and more columns exceeds shared memory.  At
    80% the weight gradient runs on column bands, at 99% on the transposed copy."""
    check(torch, synth.make_layer(640, 10000, 80, 0.1, 221, 222), b, fmt, group, 223 + b)
    check(torch, synth.make_layer(640, 10001, 99, 0.1, 224, 225), b, fmt, group, 226 + b)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 32), ("e4m3", 64), ("int8", 128),
                                       ("e4m3", 256)])
@pytest.mark.parametrize("b", [1, 2, 3, 4, 5, 8, 11, 16, 20, 33, 64])
def test_many_entries_per_column(torch, b, fmt, group):
    """More than 200 entries per column: wider tiles read the codes too (with groups
    up to 16 columns)."""
    check(torch, synth.make_layer(520, 301, 50, 0.1, 321, 322), b, fmt, group, 323 + b)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 64), ("int8", 128)])
@pytest.mark.parametrize("b", [4, 16])
def test_many_entries_wide_operand(torch, b, fmt, group):
    """Codes (and their scales) beyond shared memory."""
    check(torch, synth.make_layer(420, 15001, 50, 0.1, 331, 332), b, fmt, group, 333 + b)
    check(torch, synth.make_layer(40, 70001, 99, 0.1, 334, 335), b, fmt, group, 336 + b)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 128), ("e4m3", 32)])
@pytest.mark.parametrize("b", [17, 24, 25, 33, 40, 41, 64 + 18])
def test_rows_past_a_tile(torch, monkeypatch, b, fmt, group):
    """Large layers run a few rows more than 16 or 32 as a tile of their own."""
    monkeypatch.setenv("SNK_LARGE_BATCH", "off")
    check(torch, synth.make_layer(4100, 2000, 50, 0.1, 341, 342), b, fmt, group, 343 + b)


def test_groups_of_nan_in_small_batches(torch):
    def spoil(x):
        x[1] = 0
        x[2, 70] = np.inf
        x[3, 250:] = np.nan
        x[4] *= np.float32(1e-20)
        x[5, :100] *= np.float32(1e-5)

    for b in (6, 8, 13, 20):
        for fmt in ("int8", "e4m3"):
            check(torch, synth.make_layer(520, 301, 50, 0.1, 351, 352), b, fmt, 64, 353 + b, spoil)
            check(torch, synth.make_layer(97, 301, 99, 0.1, 354, 355), b, fmt, 32, 356 + b, spoil)


def test_columns_past_16_bits(torch):
    """in > 65536: 32-bit column indices."""
    check(torch, synth.make_layer(40, 70000, 99, 0.1, 231, 232), 3, "int8", 0, 233)
    check(torch, synth.make_layer(40, 70000, 99, 0.1, 231, 232), 9, "e4m3", 64, 234)


def test_zipf_rows(torch):
    lay = synth.make_layer(3072, 768, 90, 0.05, 241, 242, zipf_s=1.2)
    for b in (1, 64):
        check(torch, lay, b, "int8", 0, 243 + b)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 32), ("e4m3", 256)])
@pytest.mark.parametrize("b", [96, 130, 300])
def test_tensor_cores(torch, monkeypatch, fmt, group, b):
    monkeypatch.setenv("SNK_LARGE_BATCH", "on")
    check(torch, synth.make_layer(300, 200, 90, 0.1, 251, 252), b, fmt, group, 253 + b)
    check(torch, synth.make_layer(517, 1003, 95, 0.1, 254, 255), b, fmt, group, 256 + b, bias=False)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 32), ("e4m3", 256)])
@pytest.mark.parametrize("b", [1, 41, 64, 65])
def test_tensor_cores_small_batch(torch, monkeypatch, fmt, group, b):
    monkeypatch.setenv("SNK_LARGE_BATCH", "on")
    check(torch, synth.make_layer(517, 1003, 90, 0.1, 361, 362), b, fmt, group, 363 + b)


@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 128)])
@pytest.mark.parametrize("sparsity,out_f,b", [(90, 4500, 40), (90, 4500, 41), (90, 1500, 96), (95, 1500, 65), (97, 1500, 100),
                                              (98, 1500, 128), (99, 1500, 193)])
def test_choice_by_batch(torch, fmt, group, sparsity, out_f, b):
    """On both sides of the batches where a product takes the tensor cores by itself
    (the forward and the weight gradient each have their own)."""
    check(torch, synth.make_layer(out_f, 5000, sparsity, 0.1, 371, 372), b, fmt, group, 373 + b)


@pytest.mark.parametrize("large", ["on", "off"])
def test_no_entries(torch, monkeypatch, large):
    from sparse_linear_layer_gb300 import binding, q8
    monkeypatch.setenv("SNK_LARGE_BATCH", large)
    z = lambda d: torch.empty(0, dtype=d, device="cuda")
    g = binding.SparseLinear(5, 40, z(torch.float32), z(torch.int32), z(torch.int32))
    q = q8.pack(torch.randn(3, 40, device="cuda"))
    bias = torch.arange(5.0, device="cuda")
    assert torch.equal(g.forward_q8(q, bias), bias.expand(3, 5))
    dw, db = g.backward_weight_q8(q, torch.ones(3, 5, device="cuda"), with_bias=True)
    assert dw.numel() == 0 and torch.equal(db, torch.full((5,), 3.0, device="cuda"))
    none = q8.pack(torch.empty(0, 40, device="cuda"))
    assert g.forward_q8(none).shape == (0, 5)
    g.close()


@pytest.mark.parametrize("large", ["on", "off"])
@pytest.mark.parametrize("group", [0, 32])
def test_scales_of_nan_zero_and_wide_range(torch, monkeypatch, large, group):
    """A NaN group reaches only the outputs of its columns; zero rows and rows of
    very different magnitude keep the tolerance."""
    monkeypatch.setenv("SNK_LARGE_BATCH", large)

    def spoil(x):
        x[3] = 0
        x[5, 70] = np.inf
        x[7] *= np.float32(1e-20)
        x[8] *= np.float32(1e4)
        x[9, :100] *= np.float32(1e-5)

    check(torch, synth.make_layer(150, 200, 90, 0.1, 261, 262), 130, "int8", group, 263, spoil)
    check(torch, synth.make_layer(150, 200, 90, 0.1, 261, 262), 130, "e4m3", group, 264, spoil)


@pytest.mark.parametrize("b", [4, 300])
def test_graph_capture(torch, b):
    lay = synth.make_layer(300, 200, 90, 0.1, 271, 272)
    g = make_gpu_layer(torch, lay)
    rng = np.random.default_rng(273)
    q, _ = q8_input(torch, rng, b, 200, "int8", 0)
    dy = dev(rng.standard_normal((b, 300)).astype(np.float32), torch)
    y0, dw0 = g.forward_q8(q), g.backward_weight_q8(q, dy)   # the first call builds the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dw = g.forward_q8(q), g.backward_weight_q8(q, dy)
    y.zero_()
    dw.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(dw, dw0)
    g.close()


def test_refusals(torch):
    from sparse_linear_layer_gb300 import q8
    lay = synth.make_layer(30, 20, 50, 0.1, 281, 282)
    g = make_gpu_layer(torch, lay)
    with pytest.raises(ValueError):
        g.forward_q8(q8.pack(torch.randn(3, 21, device="cuda")))
    q = q8.pack(torch.randn(3, 20, device="cuda"))
    with pytest.raises(ValueError):
        g.backward_weight_q8(q, torch.randn(4, 30, device="cuda"))
    with pytest.raises(ValueError):
        g.backward_weight_q8(q, torch.randn(3, 30, device="cuda").half())
    g.close()
