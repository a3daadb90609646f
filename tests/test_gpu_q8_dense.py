"""Dense products on 8-bit matrices, the packing they take, and the layer on them, against
64 bits: sizes of one row to several tiles, partial groups, blocks and tiles, strides,
streams, graphs and refusals.

Tolerances.  Codes and scales are defined bit for bit.  In a product each group of 128 is
exact up to the tensor cores' additions (five of them with the accumulator's, within 2^-23
of the group's magnitudes each), its scales' product and its addition round once more, and
the groups' sum rounds once per group: with A the sum of all terms' magnitudes the error is at
most (10 + groups) * 2^-23 * A, then half a unit of the result's type."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_linear_layer_gb300 import binding, dense, q8  # noqa: E402
from tests import dense_ref  # noqa: E402
from tests.gpu_util import need_gpu  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def bits(q):
    return q.codes.contiguous().view(torch.uint8)


def matrix(rows, cols, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    return (x * torch.logspace(-3, 1, cols, device="cuda")[torch.randperm(cols, device="cuda", generator=g)]).to(dtype)


def check_product(y, a, b, bias=None):
    """a, b in 64 bits."""
    want, mag = a @ b.T, a.abs() @ b.abs().T
    if bias is not None:
        want, mag = want + bias.double(), mag + bias.double().abs()
    tol = (10 + -(-a.shape[1] // 128)) * 2.0 ** -23 * mag + UNIT[y.dtype] * want.abs() + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), f"off by {(err / tol).max().item():.2f} of the tolerance"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (128, 128), (130, 257), (300, 260), (77, 1000), (1000, 33)])
def test_packing(rows, cols, dtype):
    x = matrix(rows, cols, dtype)
    a, at = q8.pack_both(x)
    for got, want in ((a, q8.pack(x, "e4m3", 128)), (at, q8.pack(x.T.contiguous(), "e4m3", 128))):
        assert torch.equal(bits(got), bits(want)) and torch.equal(got.scales, want.scales)
        assert torch.equal(got.dequantize(), want.dequantize())
    w, wt = q8.pack_blocks(x, transposed=True)
    codes, scales = dense_ref.pack_blocks(x)
    assert torch.equal(bits(w), codes.view(torch.uint8)) and torch.equal(w.scales, scales)
    assert torch.equal(bits(wt), codes.view(torch.uint8).T) and torch.equal(wt.scales, scales.T)
    assert torch.equal(bits(q8.pack_blocks(x)), bits(w))


def test_packing_of_what_has_no_scale():
    x = matrix(200, 300)
    x[5, 7], x[150, 290] = float("nan"), float("inf")
    x[64:, :128] = 1e-32
    a, at = q8.pack_both(x)
    for got, want in ((a, q8.pack(x, "e4m3", 128)), (at, q8.pack(x.T.contiguous(), "e4m3", 128))):
        assert torch.equal(bits(got), bits(want)) and torch.equal(got.scales.isnan(), want.scales.isnan())
        assert torch.equal(got.scales.nan_to_num(), want.scales.nan_to_num())
    w = q8.pack_blocks(x)
    codes, scales = dense_ref.pack_blocks(x)
    assert torch.equal(w.scales.isnan(), scales.isnan()) and int(scales.isnan().sum()) == 2
    assert torch.equal(bits(w), codes.view(torch.uint8))
    # a block that reads as NaN gives NaN to the outputs that it takes part in, and to no others
    y = q8.matmul(q8.pack(matrix(9, 300), "e4m3", 128), w)
    assert bool(y.isnan().all())
    x[5, 7] = 0
    y = q8.matmul(q8.pack(matrix(9, 300), "e4m3", 128), q8.pack_blocks(x))
    assert bool(y[:, 128:].isnan().all()) and bool(y[:, :128].isfinite().all())


SHAPES = [(1, 1, 1), (1, 2304, 768), (3, 100, 17), (8, 64, 1000), (16, 130, 2000), (17, 64, 128), (100, 200, 4096),
          (128, 1001, 130), (129, 300, 1000), (333, 1001, 1000), (600, 2000, 300), (2600, 2100, 260), (1000, 700, 20000), (500, 500, 6400)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("weight", ["blocks", "rows"])
@pytest.mark.parametrize("rows,out,cols", SHAPES)
def test_product(rows, out, cols, weight, dtype):
    a = q8.pack(matrix(rows, cols), "e4m3", 128)
    w = matrix(out, cols, seed=1) / cols ** 0.5
    b = q8.pack_blocks(w) if weight == "blocks" else q8.pack(w, "e4m3", 128)
    bias = torch.randn(out, device="cuda")
    va, vb = dense_ref.values(a.codes, a.scales), dense_ref.values(b.codes, b.scales, weight == "blocks")
    y = q8.matmul(a, b, bias=bias, dtype=dtype)
    assert y.dtype == dtype and y.shape == (rows, out)
    check_product(y, va, vb, bias)
    check_product(q8.matmul(a, b, dtype=dtype), va, vb)
    assert torch.equal(y, q8.matmul(a, b, bias=bias, dtype=dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("weight", ["blocks", "rows"])
@pytest.mark.parametrize("rows,out,cols,shift", [(512, 2048, 8192, 0), (512, 2048, 8192, 2), (520, 1030, 8000, 0), (2304, 768, 16384, 0)])
def test_product_in_ranges(rows, out, cols, shift, weight, dtype):
    """Few tiles and a long K: the sums of several ranges, joined by fours, or by ones where the output is not aligned."""
    g = torch.Generator(device="cuda").manual_seed(rows + out)
    a = q8.pack(torch.randn(rows, cols, device="cuda", generator=g), "e4m3", 128)
    w = torch.randn(out, cols, device="cuda", generator=g)
    b = q8.pack_blocks(w) if weight == "blocks" else q8.pack(w, "e4m3", 128)
    bias = torch.randn(out, device="cuda", generator=g)
    y = torch.empty(rows * out + 16, device="cuda", dtype=dtype)[shift:shift + rows * out].view(rows, out)
    q8.matmul(a, b, bias=bias, dtype=dtype, out=y)
    check_product(y, dense_ref.values(a.codes, a.scales), dense_ref.values(b.codes, b.scales, blocks=weight == "blocks"), bias)


@pytest.mark.parametrize("rows", [2, 40, 300])
def test_product_of_strided_and_shifted_codes(rows):
    """Rows further apart than they are long, with NaN codes between them, and codes that do not
    start on 16 bytes."""
    a, b = q8.pack(matrix(rows, 200), "e4m3", 128), q8.pack(matrix(70, 200, seed=1), "e4m3", 128)
    want = q8.matmul(a, b)
    for stride in (203, 208):
        far = torch.full((70, stride), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        far[:, :200] = b.codes
        got = q8.Q8Tensor(b.codes, b.scales, 128)
        got.codes = far[:, :200]
        assert torch.equal(q8.matmul(a, got), want)
    flat = torch.empty(rows * 200 + 5, dtype=torch.float8_e4m3fn, device="cuda")
    shifted = flat[5:].view(rows, 200)
    shifted.copy_(a.codes)
    assert torch.equal(q8.matmul(q8.Q8Tensor(shifted, a.scales, 128), b), want)
    codes, scales = dense_ref.pack_blocks(matrix(70, 200, seed=1))
    w = q8.Q8Blocks(codes, scales)
    assert w.codes.stride(0) % 16 == 0 and torch.equal(q8.matmul(a, w), q8.matmul(a, q8.pack_blocks(matrix(70, 200, seed=1))))


def test_product_leaves_its_neighbours():
    """Outputs in a larger buffer: what lies around them stays."""
    for rows, out in ((3, 37), (50, 133), (300, 515)):
        a, b = q8.pack(matrix(rows, 300), "e4m3", 128), q8.pack_blocks(matrix(out, 300, seed=1))
        for dtype in (torch.float32, torch.bfloat16):
            buf = torch.full((rows * out + 64,), 7.0, device="cuda", dtype=dtype)
            y = buf[32:32 + rows * out].view(rows, out)
            assert q8.matmul(a, b, dtype=dtype, out=y) is not None
            assert torch.equal(y, q8.matmul(a, b, dtype=dtype))
            assert bool((buf[:32] == 7).all()) and bool((buf[32 + rows * out:] == 7).all())


def test_nan_codes_reach_their_outputs_only():
    for rows in (5, 200):
        a, b = q8.pack(matrix(rows, 300), "e4m3", 128), q8.pack(matrix(90, 300, seed=1), "e4m3", 128)
        a.codes.view(torch.uint8)[2, 10] = 0x7f
        b.codes.view(torch.uint8)[50, 299] = 0xff
        y = q8.matmul(a, b)
        nan = y.isnan()
        assert bool(nan[2].all()) and bool(nan[:, 50].all()) and int(nan.sum()) == 90 + rows - 1


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements, written and checked at both ends; codes as many."""
    a, b = q8.pack(matrix(50_000, 128), "e4m3", 128), q8.pack_blocks(matrix(45_056, 128, seed=1))
    y = q8.matmul(a, b, dtype=torch.bfloat16)
    vb = dense_ref.values(b.codes, b.scales, True)
    for r in (slice(0, 3), slice(25_000, 25_003), slice(49_997, 50_000)):
        check_product(y[r], dense_ref.values(a.codes[r], a.scales[r]), vb)
    del y, vb
    x = torch.randn(1_100_000, 2048, device="cuda", dtype=torch.bfloat16)
    _, xt = q8.pack_both(x)
    part = slice(1_099_776, 1_100_000)   # (the last two groups of rows, the second one short)
    want = q8.pack(x[part].T.contiguous(), "e4m3", 128)
    assert torch.equal(xt.codes[:, part].contiguous().view(torch.uint8), bits(want))
    assert torch.equal(xt.scales[:, -2:], want.scales)
    w8 = q8.pack_blocks(x)
    y = q8.matmul(q8.pack(matrix(3, 2048), "e4m3", 128), w8)
    tail = dense_ref.values(w8.codes[part], w8.scales[-2:], True)
    check_product(y[:, part], dense_ref.values(*(lambda q: (q.codes, q.scales))(q8.pack(matrix(3, 2048), "e4m3", 128))), tail)


def test_more_dimensions_streams_and_empty():
    a, b = q8.pack(matrix(60, 256).view(3, 20, 256), "e4m3", 128), q8.pack_blocks(matrix(100, 256, seed=1))
    y = q8.matmul(a, b)
    assert y.shape == (3, 20, 100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = q8.matmul(a, b, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, z)
    empty = q8.pack(torch.empty(0, 256, device="cuda"), "e4m3", 128)
    assert q8.matmul(empty, b).shape == (0, 100)
    e, et = q8.pack_both(torch.empty(0, 256, device="cuda"))
    assert e.shape == (0, 256) and et.shape == (256, 0)


def test_captured_product():
    for rows in (4, 60, 300):
        a, b = q8.pack(matrix(rows, 1000), "e4m3", 128), q8.pack_blocks(matrix(200, 1000, seed=1))
        q8.matmul(a, b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = q8.matmul(a, b)
        other = q8.pack(matrix(rows, 1000, seed=9), "e4m3", 128)
        a.codes.copy_(other.codes)
        a.scales.copy_(other.scales)
        graph.replay()
        assert torch.equal(y, q8.matmul(other, b))


def rounded(x, along_rows=False, blocks=False):
    """The values of x's 8-bit form."""
    if blocks:
        q = q8.pack_blocks(x)
        return dense_ref.values(q.codes, q.scales, True)
    q = q8.pack(x.T.contiguous() if along_rows else x, "e4m3", 128)
    v = dense_ref.values(q.codes, q.scales)
    return v.T if along_rows else v


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("weight_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,out", [(1, 64, 32), (5, 100, 200), (130, 257, 65), (300, 1000, 520)])
def test_linear_and_its_gradients(rows, cols, out, weight_dtype, dtype):
    x = matrix(rows, cols, dtype).requires_grad_()
    w = (matrix(out, cols, seed=1) / cols ** 0.5).to(weight_dtype).requires_grad_()
    b = torch.randn(out, device="cuda").requires_grad_()
    dy = (0.01 * torch.randn(rows, out, device="cuda")).to(dtype)
    y = dense.linear_q8(x, w, b)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    xd, wd = x.detach(), w.detach()
    wv = rounded(wd, blocks=True)
    check_product(y, rounded(xd), wv, b.detach())
    check_product(dx, rounded(dy), wv.T)
    check_product(dw, rounded(dy, True).T, rounded(xd, True).T)
    assert (y.dtype, dx.dtype, dw.dtype, db.dtype) == (dtype, dtype, weight_dtype, torch.float32)
    # a column's sum: chains of 32 within a tile, then the tiles
    s = dy.double().abs().sum(0)
    assert bool(((db.double() - dy.double().sum(0)).abs() <= (66 + rows / 1024) * 2.0 ** -24 * s).all())


def test_linear_gradient_against_differences():
    """Of the function of the 8-bit values, whose derivative the layer passes through: differences
    of the exact product in 64 bits."""
    x, w = matrix(70, 200).requires_grad_(), (matrix(90, 200, seed=1) / 14).requires_grad_()
    dy = torch.randn(70, 90, device="cuda")
    dx, dw = torch.autograd.grad(dense.linear_q8(x, w), (x, w), dy)
    for got, fixed, vary in ((dx, rounded(w.detach(), blocks=True), "x"), (dw, rounded(x.detach(), True), "w")):
        v = torch.randn(got.shape, device="cuda", dtype=torch.float64)
        upstream = rounded(dy) if vary == "x" else rounded(dy, True)
        f = (lambda e: ((e * v) @ fixed.T * upstream).sum()) if vary == "x" else (lambda e: (fixed @ (e * v).T * upstream).sum())
        want = (f(0.5) - f(-0.5)) / 1.0
        scale = (got.double().abs() * v.abs()).sum()
        assert abs((want - (got.double() * v).sum()).item()) <= 20 * 2.0 ** -23 * scale.item() * 20


def test_linear_asks_only_for_what_is_needed():
    x, w, b = matrix(40, 100), matrix(50, 100, seed=1), torch.zeros(50, device="cuda")
    y = dense.linear_q8(x, w, b)
    assert not y.requires_grad
    leaves = [v.detach().requires_grad_() for v in (x, w, b)]
    grads = torch.autograd.grad(dense.linear_q8(*leaves).square().sum(), leaves)
    for i in range(3):
        one = [v.detach().requires_grad_(k == i) for k, v in enumerate((x, w, b))]
        got, = torch.autograd.grad(dense.linear_q8(*one).square().sum(), one[i])
        assert torch.equal(got, grads[i])
    assert torch.equal(dense.linear_q8(x[0], w, b), dense.linear_q8(x[:1], w, b)[0])
    assert torch.equal(dense.linear_q8(x.view(4, 10, 100), w, b), dense.linear_q8(x, w, b).view(4, 10, 50))
    wide = torch.zeros(40, 200, device="cuda")
    wide[:, ::2] = x
    wide.requires_grad_()
    dwide, = torch.autograd.grad(dense.linear_q8(wide[:, ::2], w, b).square().sum(), wide)
    assert torch.equal(dwide[:, ::2], grads[0]) and bool((dwide[:, 1::2] == 0).all())
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(dense.linear_q8(leaves[0], w, b).sum(), leaves[0], create_graph=True)
    xe = torch.empty(0, 100, device="cuda", requires_grad=True)
    ye = dense.linear_q8(xe, leaves[1], leaves[2])
    dx, dw, db = torch.autograd.grad(ye.sum(), (xe, leaves[1], leaves[2]))
    assert ye.shape == (0, 50) and dx.shape == (0, 100) and bool((dw == 0).all()) and bool((db == 0).all())


def test_captured_linear_step():
    layer = dense.Q8Linear(96, 200)
    x = matrix(150, 96).requires_grad_()
    dy = torch.randn(150, 200, device="cuda")

    def step():
        y = layer(x)
        return (y, *torch.autograd.grad(y, (x, layer.weight, layer.bias), dy))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    with torch.no_grad():
        x.copy_(matrix(150, 96, seed=4))
        layer.weight.mul_(1.5)
    graph.replay()
    got = [o.detach().clone() for o in outs]
    for a, b in zip(got, step()):
        assert torch.equal(a, b.detach())


def test_calls_from_threads():
    """Several threads at once, on streams of their own, each call the first CUDA work of its thread."""
    import threading
    x, w, wb = matrix(300, 512), matrix(400, 512, seed=1), matrix(400, 512, seed=1).bfloat16()
    xb, t = x.bfloat16(), torch.arange(300, device="cuda")
    x8, w8 = q8.pack(x, "e4m3", 128), q8.pack_blocks(w)
    calls = [lambda s: q8.matmul(x8, w8, stream=s), lambda s: q8.pack_both(x, stream=s)[1].codes.view(torch.uint8),
             lambda s: q8.pack_blocks(w, stream=s).codes.view(torch.uint8),
             lambda s: binding.ops().vocab_loss(xb, wb, t, -100, 0, s)[0]] * 2
    want = [f(None) for f in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [None] * len(calls)

    def work(i):
        got[i] = calls[i](streams[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    x = q8.pack(matrix(4, 256), "e4m3", 128)
    w = q8.pack_blocks(matrix(10, 256))
    for a, b in [(q8.pack(matrix(4, 256), "int8", 128), w), (q8.pack(matrix(4, 256), "e4m3", 64), w),
                 (q8.pack(matrix(4, 256), "e4m3", 0), w), (x, q8.pack(matrix(10, 256), "e4m3", 0)),
                 (x, q8.pack(matrix(10, 256), "int8", 128)), (x, q8.pack_blocks(matrix(10, 128)))]:
        with pytest.raises(ValueError):
            q8.matmul(a, b)
    for kw in [dict(bias=torch.zeros(9, device="cuda")), dict(bias=torch.zeros(10, device="cuda").half()),
               dict(bias=torch.zeros(10)), dict(dtype=torch.float64), dict(out=torch.empty(4, 9, device="cuda")),
               dict(out=torch.empty(4, 10, device="cuda").half()), dict(out=torch.empty(10, 4, device="cuda").T)]:
        with pytest.raises(ValueError):
            q8.matmul(x, w, **kw)
    with pytest.raises(ValueError):
        q8.Q8Blocks(w.codes, w.scales[:, :1])
    with pytest.raises(ValueError):
        q8.Q8Blocks(w.codes.float(), w.scales)
    with pytest.raises(ValueError):
        q8.pack_blocks(matrix(4, 256).double())
    with pytest.raises(ValueError):
        q8.pack_blocks(matrix(4, 256)[:, ::2])
    with pytest.raises(ValueError):
        dense.linear_q8(matrix(4, 256), matrix(10, 255))
    with pytest.raises(ValueError):
        dense.linear_q8(matrix(4, 256).double(), matrix(10, 256))
