"""The vocabulary loss and its gradients against the definition in 64 bits, at sizes of one
row to several row tiles, odd widths and vocabularies, ignored rows and what they hold,
streams, graphs and refusals.

Tolerances.  A logit is a sum of exact products accumulated by the tensor cores, whose
additions truncate: each of the cols / 16 steps loses at most 2^-23 of the running sum of
magnitudes, so |z - exact| <= cols / 16 * 2^-23 * A with A = sum |x w|.  The loss is a
difference of two such numbers through exp and log, whose own errors (2 units of ex2 and log
each, in sums of fp32) are below 16 * 2^-24 * (1 + |lse| + |z|).  A gradient's terms are dz w
with dz rounded to 16 bits (half a unit, u) and off by the relative error of p, 2 * |z - exact|
plus 8 * 2^-24 for exp; the sums truncate as above, over the rows or vocabulary, in splits; the
result is rounded to 16 bits (u once more)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_linear_layer_gb300 import binding, dense  # noqa: E402
from tests import dense_ref  # noqa: E402
from tests.gpu_util import need_gpu  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def case(rows, cols, vocab, dtype, ignored=0.3, seed=0, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    w = (torch.randn(vocab, cols, device="cuda", generator=g) * spread / cols ** 0.5).to(dtype)
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    t[torch.rand(rows, device="cuda", generator=g) < ignored] = -100
    return x, w, t


def logit_error(x, w):
    """The largest |z - exact| of each row."""
    return x.shape[1] / 16 * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T).amax(1) + 1e-30


def check_loss(loss, x, w, t):
    want, lse, _ = dense_ref.loss(x, w, t)
    e = logit_error(torch.where((t != -100)[:, None], x, 0), w)
    tol = 2 * e + 16 * 2.0 ** -24 * (1 + 2 * lse.abs() + want.abs())
    err = (loss.double() - want).abs()
    assert bool((err <= tol).all()), f"loss off by {(err / tol).max().item():.2f} of the tolerance"
    assert bool((loss[t == -100] == 0).all())


def check_gradients(dx, dw, x, w, t, g):
    want_x, want_w, ax, aw = dense_ref.loss_gradient(x, w, t, g)
    u = UNIT[x.dtype]
    kept = torch.where((t != -100)[:, None], x, 0)
    e = logit_error(kept, w)
    rel = 2 * e.max().item() + 8 * 2.0 ** -24 + u
    tiny = 2.0 ** -24 if x.dtype == torch.float16 else 0.0   # fp16's subnormal step: half of it
    for got, want, a, terms in ((dx, want_x, ax, w.shape[0]), (dw, want_w, aw, x.shape[0])):
        tol = (rel + (terms / 16 + 4) * 2.0 ** -23) * a + u * want.abs() + tiny
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), f"gradient off by {(err / tol).max().item():.2f} of the tolerance"


SHAPES = [(1, 8, 1), (1, 64, 300), (3, 100, 257), (128, 768, 1000), (129, 64, 512), (200, 1001, 700), (256, 65, 333),
          (257, 128, 4099), (700, 320, 2049)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols,vocab", SHAPES)
def test_loss_and_gradients(rows, cols, vocab, dtype):
    x, w, t = case(rows, cols, vocab, dtype)
    if bool((t == -100).all()):
        t[0] = vocab - 1
    check_loss(dense.linear_cross_entropy(x, w, t, reduction="none"), x, w, t)
    x.requires_grad_()
    w.requires_grad_()
    n = (t != -100).sum()
    loss = dense.linear_cross_entropy(x, w, t)
    want = dense_ref.loss(x.detach(), w.detach(), t)[0]
    assert abs(loss.item() - (want.sum() / n).item()) <= 2 * logit_error(x.detach(), w.detach()).max() + 1e-5
    dx, dw = torch.autograd.grad(loss, (x, w))
    assert dx.dtype == dtype and dw.dtype == dtype
    check_gradients(dx, dw, x.detach(), w.detach(), t, torch.full((rows,), 1.0 / n.item(), device="cuda"))
    assert bool((dx[t == -100] == 0).all())


# several row tiles and pairs of them, columns for one accumulator and for several
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols,vocab", [(2, 1, 3), (2000, 640, 30000), (1500, 1100, 20000), (1030, 2056, 9001)])
def test_larger_shapes(rows, cols, vocab, dtype):
    x, w, t = case(rows, cols, vocab, dtype, ignored=0.1)
    t[0] = 1
    x.requires_grad_()
    w.requires_grad_()
    each = dense.linear_cross_entropy(x, w, t, reduction="none")
    check_loss(each.detach(), x.detach(), w.detach(), t)
    g = torch.randn(rows, device="cuda")
    check_gradients(*torch.autograd.grad(each, (x, w), g), x.detach(), w.detach(), t, g)


def test_offsets_past_32_bits():
    """A weight and its gradient of more than 2^31 elements, and a batch whose logits have as many:
    sampled rows against 64 bits."""
    rows, cols, vocab = 3000, 4096, 800_000
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    w = torch.empty(vocab, cols, device="cuda", dtype=torch.bfloat16)
    for i in range(0, vocab, 100_000):
        w[i:i + 100_000] = torch.randn(100_000, cols, device="cuda", generator=g) / 64
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    t[rows - 1], t[0] = vocab - 1, 0
    x.requires_grad_()
    w.requires_grad_()
    each = dense.linear_cross_entropy(x, w, t, reduction="none")
    dx, dw = torch.autograd.grad(each.sum(), (x, w))
    pick = torch.tensor([0, 1, 1500, rows - 1], device="cuda")
    xs, z = x.detach()[pick].double(), torch.empty(4, vocab, device="cuda", dtype=torch.float64)
    for i in range(0, vocab, 100_000):
        z[:, i:i + 100_000] = xs @ w.detach()[i:i + 100_000].double().T
    lse = z.logsumexp(1)
    want = lse - z.gather(1, t[pick][:, None])[:, 0]
    assert (each.detach()[pick].double() - want).abs().max() < 1e-4
    p = (z - lse[:, None]).exp()
    p[torch.arange(4), t[pick]] -= 1
    want_dx = sum(p[:, i:i + 100_000] @ w.detach()[i:i + 100_000].double() for i in range(0, vocab, 100_000))
    assert ((dx[pick].double() - want_dx).norm(dim=1) <= 4 * UNIT[torch.bfloat16] * want_dx.norm(dim=1)).all()
    cols_at = torch.tensor([0, 5, vocab // 2, vocab - 1], device="cuda")
    zc = x.detach().double() @ w.detach()[cols_at].double().T
    # every row's lse from the loss itself, which is checked above on a sample
    at = (x.detach().double() * w.detach()[t].double()).sum(1)
    pc = (zc - (each.detach().double() + at)[:, None]).exp()
    for k, c in enumerate(cols_at.tolist()):
        pc[t == c, k] -= 1
    want_dw = pc.T @ x.detach().double()
    assert ((dw[cols_at].double() - want_dw).norm(dim=1) <= 4 * UNIT[torch.bfloat16] * want_dw.norm(dim=1)).all()


def test_another_ignored_value_and_strided_inputs():
    x, w, t = case(60, 48, 90, torch.bfloat16, ignored=0)
    t[:10] = 5
    want = dense_ref.loss(x, w, t, ignore=5)[0]
    got = dense.linear_cross_entropy(x, w, t, ignore=5, reduction="none")
    assert bool((got[:10] == 0).all()) and (got.double() - want).abs().max() < 1e-4
    # gradients reach the storage that strided inputs are views of
    base = torch.zeros(48, 120, device="cuda", dtype=torch.bfloat16)
    base[:, ::2] = x.T
    base.requires_grad_()
    wide = torch.zeros(90, 96, device="cuda", dtype=torch.bfloat16)
    wide[:, 48:] = w
    wide.requires_grad_()
    leaf_x, leaf_w = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(leaf_x, leaf_w, t), (leaf_x, leaf_w))
    db, dwide = torch.autograd.grad(dense.linear_cross_entropy(base[:, ::2].T, wide[:, 48:], t.repeat(2)[::1][:60]), (base, wide))
    assert torch.equal(db[:, ::2], dx.T) and bool((db[:, 1::2] == 0).all())
    assert torch.equal(dwide[:, 48:], dw) and bool((dwide[:, :48] == 0).all())


def test_no_second_derivative():
    x, w, t = case(10, 32, 40, torch.bfloat16)
    x.requires_grad_()
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(dense.linear_cross_entropy(x, w, t), x, create_graph=True)
    loss = dense.linear_cross_entropy(x, w.requires_grad_(), t)
    with torch.no_grad():
        w.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("rows", [5, 300])
def test_reductions_and_upstream_gradients(rows):
    x, w, t = case(rows, 96, 1000, torch.bfloat16)
    t[0] = 3
    x.requires_grad_()
    w.requires_grad_()
    g = torch.randn(rows, device="cuda") * torch.logspace(-6, 2, rows, device="cuda")
    each = dense.linear_cross_entropy(x, w, t, reduction="none")
    check_gradients(*torch.autograd.grad(each, (x, w), g), x.detach(), w.detach(), t, g)
    total = dense.linear_cross_entropy(x, w, t, reduction="sum")
    torch.testing.assert_close(total, each.sum(), rtol=1e-5, atol=1e-5)
    check_gradients(*torch.autograd.grad(total, (x, w), torch.tensor(-3.0, device="cuda")), x.detach(), w.detach(), t,
                    torch.full((rows,), -3.0, device="cuda"))


@pytest.mark.parametrize("g", [0.53014, 1.0, 700.0])
def test_upstream_gradient_costs_no_rounding(g):
    """Targets of probability about 1 / 5000 and an upstream gradient that puts 2^13 g (1 - p) halfway between
    two fp16 numbers just above a power of two.  Without g, p - 1 lies in [2^-1, 1) next to 1, where half a unit
    is 2^-12 of it: dw of a target is then within u of itself (its own rounding) plus 2^-12 of |g x_t| plus u of
    the other rows' terms; fp32 sums and logits add less than 2^-16 of the terms."""
    u = UNIT[torch.float16]
    x, w, _ = case(64, 128, 5000, torch.float16, ignored=0, seed=5, spread=0.05)
    t = torch.randperm(5000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))[:64]
    leaf = w.clone().requires_grad_()
    dw, = torch.autograd.grad(dense.linear_cross_entropy(x, leaf, t, reduction="sum"), leaf, torch.tensor(g, device="cuda"))
    xd = x.double()
    p = torch.softmax(xd @ w.double().T, 1)[:, t]           # [row, target]
    own = torch.diag(torch.diag(p) - 1)
    others = p - torch.diag(torch.diag(p))
    want = g * (own + others).T @ xd
    sizes = g * others.T @ xd.abs()
    first = g * xd.abs()
    tol = u * want.abs() + 2.0 ** -12 * first + u * sizes + 2.0 ** -16 * (first + sizes) + 2.0 ** -25
    err = (dw[t].double() - want).abs()
    assert bool((err <= tol).all()), f"off by {(err / tol).max().item():.2f} of the tolerance"


def test_gradient_against_differences():
    """Central differences of the loss along random directions.  With a step of h |direction| the
    fp64 loss of the rounded points is exact; the gradient is the kernel's."""
    x, w, t = case(40, 64, 200, torch.bfloat16, seed=3)
    x.requires_grad_()
    w.requires_grad_()
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), (x, w))
    g = torch.Generator(device="cuda").manual_seed(5)
    for _ in range(4):
        vx = torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64)
        vw = torch.randn(w.shape, device="cuda", generator=g, dtype=torch.float64)
        h = 1e-5
        up = dense_ref.loss(x.detach().double() + h * vx, w.detach().double() + h * vw, t)[0].sum()
        down = dense_ref.loss(x.detach().double() - h * vx, w.detach().double() - h * vw, t)[0].sum()
        along = (dx.double() * vx).sum() + (dw.double() * vw).sum()
        # the directions are independent of the roundings, each 2 u of a term: their sum is within
        # 8 standard deviations of 2 u times the root of the gradients' squares
        tol = 8 * 2 * UNIT[torch.bfloat16] * (dx.double().pow(2).sum() + dw.double().pow(2).sum()).sqrt() + 1e-4
        assert abs(((up - down) / (2 * h) - along).item()) <= tol.item()


def test_all_rows_ignored():
    for rows in (4, 300):
        x, w, t = case(rows, 64, 100, torch.bfloat16)
        t.fill_(-100)
        x.requires_grad_()
        w.requires_grad_()
        assert bool((dense.linear_cross_entropy(x, w, t, reduction="none") == 0).all())
        assert dense.linear_cross_entropy(x, w, t, reduction="sum").item() == 0
        loss = dense.linear_cross_entropy(x, w, t)
        assert torch.isnan(loss)
        dx, dw = torch.autograd.grad(loss, (x, w))
        assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("rows", [100, 300])
def test_all_rows_ignored_many_tiles(rows):
    """Several tiles of dW per pair of processors, each a sum over no rows."""
    x, w, t = case(rows, 768, 50257, torch.float16)
    t.fill_(-100)
    x.requires_grad_()
    w.requires_grad_()
    for _ in range(3):
        dx, dw = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), (x, w))
        assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("rows", [60, 400])
def test_what_ignored_rows_hold_reaches_nothing(rows):
    x, w, t = case(rows, 80, 500, torch.float16)
    t[1] = 7
    clean = x.clone()
    bad = t == -100
    x[bad] = torch.tensor([float("nan"), float("inf"), -float("inf"), 65504.0], device="cuda",
                          dtype=torch.float16)[torch.arange(int(bad.sum()), device="cuda") % 4][:, None]
    g = torch.ones(rows, device="cuda")
    g[bad] = float("nan")
    outs = []
    for v in (clean, x):
        v = v.detach().requires_grad_()
        wl = w.detach().requires_grad_()
        loss = dense.linear_cross_entropy(v, wl, t, reduction="none")
        outs.append((loss, *torch.autograd.grad(loss, (v, wl), g)))
    for a, b in zip(*outs):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


@pytest.mark.parametrize("rows,cols,vocab", [(200, 256, 9000), (500, 768, 20001), (513, 128, 20001), (250, 2048, 5000)])
def test_what_ignored_rows_hold_reaches_no_loss(rows, cols, vocab):
    """One row tile of any kind, which reads x as it is, and one row more."""
    x, w, t = case(rows, cols, vocab, torch.bfloat16, seed=rows)
    want = dense.linear_cross_entropy(x, w, t, reduction="none")
    mean = dense.linear_cross_entropy(x, w, t)
    check_loss(want, x, w, t)
    x[t == -100] = float("nan")
    assert torch.equal(dense.linear_cross_entropy(x, w, t, reduction="none"), want)
    assert torch.equal(dense.linear_cross_entropy(x, w, t), mean)


def test_other_targets_and_infinite_logits():
    x, w, t = case(150, 64, 300, torch.bfloat16, ignored=0)
    t[3], t[140] = 300, -1                       # out of range: NaN, and only there
    loss = dense.linear_cross_entropy(x, w, t, reduction="none")
    assert torch.isnan(loss[[3, 140]]).all() and int(torch.isnan(loss).sum()) == 2
    x.requires_grad_()
    dx, = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), x)
    assert torch.isnan(dx[[3, 140]]).all() and int(torch.isnan(dx).any(1).sum()) == 2
    x, w, t = case(4, 64, 600, torch.bfloat16, ignored=0, spread=1.0)
    x[:, 0] = 1.0
    w[5:, 0] = -float("inf")                     # logits of -inf, whole tiles of them: no weight, no NaN
    t[:] = torch.arange(4, device="cuda")
    want = torch.logsumexp(x.double() @ w[:5].double().T, 1) - (x.double() @ w[:5].double().T)[torch.arange(4), t]
    got = dense.linear_cross_entropy(x, w, t, reduction="none")
    assert (got.double() - want).abs().max() < 1e-4
    x[2, 1] = float("nan")
    got = dense.linear_cross_entropy(x, w, t, reduction="none")
    assert torch.isnan(got[2]) and bool(torch.isfinite(got[[0, 1, 3]]).all())


@pytest.mark.parametrize("shift", [0.0, 200.0, -200.0])
def test_large_logits(shift):
    """Logits of several hundred, all positive or all negative (behind the last column of a
    partial tile lie zeros)."""
    x, w, t = case(200, 64, 777, torch.bfloat16, ignored=0.1)
    x[:, 0] = 16.0
    w[:, 0] = shift / 16
    check_loss(dense.linear_cross_entropy(x, w, t, reduction="none"), x, w, t)
    x.requires_grad_()
    w.requires_grad_()
    g = torch.ones(200, device="cuda")
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), (x, w))
    check_gradients(dx, dw, x.detach(), w.detach(), t, g)


def test_several_pieces():
    """A vocabulary whose dz does not fit one piece: the call's scratch stays bounded, pieces add up."""
    rows, cols, vocab = 8192, 64, 40000
    assert binding.snk_vocab_loss_scratch(rows, cols, vocab, True) < 2 * rows * vocab
    x, w, t = case(rows, cols, vocab, torch.bfloat16)
    x.requires_grad_()
    w.requires_grad_()
    loss = dense.linear_cross_entropy(x, w, t, reduction="sum")
    dx, dw = torch.autograd.grad(loss, (x, w))
    xd, wd = x.detach(), w.detach()
    check_gradients(dx, dw, xd, wd, t, torch.ones(rows, device="cuda"))


@pytest.mark.parametrize("cols", [9, 1])
def test_several_pieces_of_odd_rows(cols):
    x, w, t = case(2000, cols, 140001, torch.float16, ignored=0.1, seed=11)
    x.requires_grad_()
    w.requires_grad_()
    g = torch.randn(2000, device="cuda")
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="none"), (x, w), g)
    check_gradients(dx, dw, x.detach(), w.detach(), t, g)


@pytest.mark.parametrize("rows,cols,vocab", [(1, 1001, 50257), (300, 7, 4001), (40, 15, 9), (5, 3, 1), (64, 2047, 3000)])
def test_odd_rows(rows, cols, vocab):
    """Gradients whose rows begin anywhere in a word."""
    x, w, t = case(rows, cols, vocab, torch.bfloat16, ignored=0, seed=rows)
    x.requires_grad_()
    w.requires_grad_()
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), (x, w))
    check_gradients(dx, dw, x.detach(), w.detach(), t, torch.ones(rows, device="cuda"))


def test_repeats_views_and_streams():
    x, w, t = case(300, 72, 900, torch.bfloat16)
    a = dense.linear_cross_entropy(x, w, t, reduction="none")
    assert torch.equal(a, dense.linear_cross_entropy(x, w, t, reduction="none"))
    # operands that start off 16 bytes, are not contiguous, or have more dimensions
    off = torch.empty(w.numel() + 1, dtype=w.dtype, device="cuda")[1:].view_as(w).copy_(w)
    assert off.data_ptr() % 16 and torch.equal(a, dense.linear_cross_entropy(x, off, t, reduction="none"))
    wide = torch.zeros(300, 144, dtype=x.dtype, device="cuda")
    wide[:, ::2] = x
    assert torch.equal(a, dense.linear_cross_entropy(wide[:, ::2], w, t, reduction="none"))
    b = dense.linear_cross_entropy(x.view(3, 100, 72), w, t.view(3, 100), reduction="none")
    assert b.shape == (3, 100) and torch.equal(a, b.reshape(-1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = dense.linear_cross_entropy(x, w, t, reduction="none")
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)


def test_captured_step():
    """Loss and gradients in a graph, replayed on other inputs: the bits of a direct call."""
    for rows in (40, 400):
        x, w, t = case(rows, 64, 1000, torch.bfloat16, seed=1)
        x.requires_grad_()
        w.requires_grad_()

        def step():
            loss = dense.linear_cross_entropy(x, w, t)
            return (loss, *torch.autograd.grad(loss, (x, w)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for seed in (2, 3):
            with torch.no_grad():
                for a, b in zip((x, w, t), case(rows, 64, 1000, torch.bfloat16, seed=seed, ignored=0.2 * seed)):
                    a.copy_(b)
            graph.replay()
            got = [o.detach().clone() for o in outs]
            for a, b in zip(got, step()):
                assert torch.equal(a, b.detach())


def test_empty_batch():
    w = torch.randn(50, 16, device="cuda").bfloat16().requires_grad_()
    x = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    t = torch.empty(0, device="cuda", dtype=torch.int64)
    assert dense.linear_cross_entropy(x, w, t, reduction="none").shape == (0,)
    assert torch.isnan(dense.linear_cross_entropy(x, w, t))
    loss = dense.linear_cross_entropy(x, w, t, reduction="sum")
    assert loss.item() == 0
    dx, dw = torch.autograd.grad(loss, (x, w))
    assert dx.shape == x.shape and bool((dw == 0).all())


def test_one_gradient_only():
    x, w, t = case(150, 64, 500, torch.bfloat16)
    both = [v.detach().requires_grad_() for v in (x, w)]
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(*both, t), both)
    a = x.detach().requires_grad_()
    assert torch.equal(dx, torch.autograd.grad(dense.linear_cross_entropy(a, w, t), a)[0])
    a = w.detach().requires_grad_()
    assert torch.equal(dw, torch.autograd.grad(dense.linear_cross_entropy(x, a, t), a)[0])


def test_one_gradient_only_of_odd_rows():
    x, w, t = case(150, 77, 500, torch.bfloat16)
    both = [v.detach().requires_grad_() for v in (x, w)]
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(*both, t), both)
    check_gradients(dx, dw, x, w, t, torch.full((150,), 1.0 / (t != -100).sum().item(), device="cuda"))
    a = x.detach().requires_grad_()
    assert torch.equal(dx, torch.autograd.grad(dense.linear_cross_entropy(a, w, t), a)[0])
    a = w.detach().requires_grad_()
    assert torch.equal(dw, torch.autograd.grad(dense.linear_cross_entropy(x, a, t), a)[0])


@pytest.mark.parametrize("rows,cols,vocab", [(1, 768, 20000), (300, 256, 4000), (40, 129, 3000)])
def test_inputs_written_right_before_the_call(rows, cols, vocab):
    """Nothing of a call may be read before the kernels in front of it have written it."""
    sets = [case(rows, cols, vocab, torch.bfloat16, ignored=0, seed=s) for s in range(4)]
    want = [dense.linear_cross_entropy(*s, reduction="none") for s in sets]
    x, w, t = (v.clone() for v in sets[0])
    got = []
    for i in range(24):
        for to, v in zip((x, w, t), sets[i % 4]):
            to.copy_(v)
        got.append(dense.linear_cross_entropy(x, w, t, reduction="none"))
    for i, l in enumerate(got):
        assert torch.equal(l, want[i % 4])


def test_refusals():
    x, w, t = case(4, 16, 50, torch.bfloat16)
    for bad in [(x.float(), w.float(), t), (x, w.half(), t), (x, w[:, :8], t), (x, w, t.int()), (x, w, t[:3]), (x.cpu(), w, t),
                (x, w.cpu(), t), (x, w, t.cpu()), (x, w[:0], t), (x, w.view(5, 10, 16), t)]:
        with pytest.raises(ValueError):
            dense.linear_cross_entropy(*bad)
    with pytest.raises(ValueError):
        dense.linear_cross_entropy(x, w, t, reduction="max")
