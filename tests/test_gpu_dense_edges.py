"""The dense operators at the edges of what their calls take: very long rows and sums, upstream
gradients at the ends of fp32, layers converted to 16 bits, few rows of large weights, and the
entry points by the names of the C calls."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_linear_layer_gb300 import binding, dense, q8  # noqa: E402
from tests import dense_ref  # noqa: E402
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


def reference(x, w, t, g):
    """(dx, dw, |dz| |w|, |dz|^T |x|) in 64 bits."""
    x, w = x.double(), w.double()
    p = torch.softmax(x @ w.T, 1)
    p[torch.arange(len(t)), t.clamp_min(0)] -= 1
    dz = torch.where((t >= 0)[:, None], p * g.double()[:, None], 0)
    return dz @ w, dz.T @ x, dz.abs() @ w.abs(), dz.abs().T @ x.abs()


def within(got, want, magnitudes, dtype, least):
    """Two roundings to 16 bits (dz and the result) and fp32 sums of a few hundred terms, the latter within
    2^-14 of the terms' magnitudes; least: what the type's (or dz's) smallest steps add."""
    tol = 1.01 * UNIT[dtype] * (magnitudes + want.abs()) + 2.0 ** -14 * magnitudes + least
    return bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("size", [2.0 ** -149, 1e-42, 1e-38, 3e-37, 1.4e-36, 2.4e-35, 1e-30, 1.0, 1e30, 1.7e38, 3.4e38])
def test_upstream_gradients_at_the_ends_of_fp32(dtype, size):
    """Losses row by row, upstream gradients up to `size`, one of them zero, one row left out.  Whether a result
    is a number of the type or an infinity is the reference's, rounded."""
    torch.manual_seed(1)
    x, w = torch.randn(6, 40, device="cuda").to(dtype), (0.5 * torch.randn(30, 40, device="cuda")).to(dtype)
    t = torch.tensor([3, 0, -100, 29, 7, 7], device="cuda")
    g = torch.tensor([1.0, 0.0, 3e38, -1.0, 0.5, 0.25], device="cuda") * torch.tensor([size] * 2 + [1.0] + [size] * 3, device="cuda")
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(a, b, t, reduction="none"), (a, b), g)
    assert bool((dx[1] == 0).all()) and bool((dx[2] == 0).all())
    want_x, want_w, mx, mw = reference(x, w, t, g)
    top = torch.finfo(dtype).max
    # steps of the type below its normal numbers; dz in fp16 has steps of 2^-24 / 8192 of G, the sum's fp32 of 2^-149
    least = torch.finfo(dtype).tiny * torch.finfo(dtype).eps + 2.0 ** -149 + (2 * size * 2.0 ** -37 * 30 * 4 if dtype == torch.float16 else 0)
    for got, want, m in ((dx, want_x, mx), (dw, want_w, mw)):
        assert not bool(got.isnan().any())
        fits = (want.abs() + 4 * UNIT[dtype] * m) < top
        assert within(got[fits], want[fits], m[fits], dtype, least), (got, want)
        over = (want.abs() - 4 * UNIT[dtype] * m) > 1.01 * top
        assert bool(got[over].isinf().all())


@pytest.mark.parametrize("rows,cols", [(6, 40), (6, 41), (400, 64), (3, 2048)])
@pytest.mark.parametrize("upstream", [math.inf, -math.inf, math.nan])
def test_upstream_gradients_that_are_no_numbers_reach_no_ignored_row(rows, cols, upstream):
    """A sum's or mean's upstream gradient multiplies every row that counts (an overflowed loss scale), and those only."""
    torch.manual_seed(2)
    x, w = torch.randn(rows, cols, device="cuda").bfloat16(), (0.5 * torch.randn(5000, cols, device="cuda")).bfloat16()
    t = torch.arange(rows, device="cuda")
    t[1::3] = -100
    for reduction in ("sum", "mean"):
        a = x.clone().requires_grad_()
        dx, = torch.autograd.grad(dense.linear_cross_entropy(a, w, t, reduction=reduction), a, torch.tensor(upstream, device="cuda"))
        assert bool((dx[t == -100] == 0).all()) and not bool(dx[t != -100].isfinite().any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_projection_converted_to_16_bits(dtype):
    """A converted layer gives what one with the same numbers in fp32 gives, and gradients rounded once."""
    torch.manual_seed(3)
    layer = dense.Q8Linear(200, 136).to(dtype)
    with torch.no_grad():
        layer.bias.normal_()
    same = dense.Q8Linear(200, 136)
    same.load_state_dict({k: v.float() for k, v in layer.state_dict().items()})
    x = torch.randn(3, 50, 200, device="cuda").to(dtype)
    dy = torch.randn(3, 50, 136, device="cuda").to(dtype)
    outs = []
    for m in (layer, same):
        a = x.clone().requires_grad_()
        y = m(a)
        y.backward(dy)
        outs.append((y, a.grad, m.weight.grad, m.bias.grad))
    assert outs[0][2].dtype == dtype and outs[0][3].dtype == dtype
    for got, want in zip(*outs):
        assert torch.equal(got, want.to(dtype))
    with torch.no_grad():
        assert torch.equal(layer(x), outs[0][0])
    with pytest.raises(ValueError):
        dense.linear_q8(x, layer.weight, torch.zeros(136, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        dense.linear_q8(x, layer.weight, torch.zeros(135, device="cuda", dtype=dtype))


def slope(got, want):
    """By how much `got` is longer than `want`, along it."""
    return ((got.double() * want).sum() / (want * want).sum() - 1).item()


def test_weight_gradient_of_many_rows_keeps_its_length():
    """The tensor cores' additions truncate, toward zero: a sum of terms of one sign loses up to two units of
    2^-23 of itself a step (a step's 16 products are added in two parts), which for an accumulator of 1024 steps is
    2^-12 of it, and adds up to nothing where accumulators are added with rounding.  The roundings to 16 bits of dz and of the result have no
    sign: over thousands of elements they leave less than 2^-13 of the length."""
    rows, cols, vocab = 262144, 32, 400
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (1 + 0.3 * torch.randn(rows, cols, device="cuda", generator=g)).half()
    w = (0.5 * torch.randn(vocab, cols, device="cuda", generator=g)).half().requires_grad_()
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    dw, = torch.autograd.grad(dense.linear_cross_entropy(x, w, t), w)
    want = torch.zeros(vocab, cols, device="cuda", dtype=torch.float64)
    for i in range(0, rows, 65536):
        p = torch.softmax(x[i:i + 65536].double() @ w.detach().double().T, 1)
        p[torch.arange(len(p)), t[i:i + 65536]] -= 1
        want += p.T @ x[i:i + 65536].double() / rows
    assert abs(slope(dw, want)) < 2.0 ** -12 + 2.0 ** -13


def test_input_gradient_over_a_long_vocabulary():
    """Weights around 1 and targets in the last columns: each element's sum over the vocabulary grows to 1 before the
    target takes about 1 off it.  Truncation of 1024 steps at most (as above) takes less than 2^-12 off the
    first, always of the same sign; the mean over a row's elements of what dz's roundings leave is far below."""
    rows, cols, vocab = 4096, 1024, 65536
    g = torch.Generator(device="cuda").manual_seed(5)
    x = (0.05 * torch.randn(rows, cols, device="cuda", generator=g)).half().requires_grad_()
    w = (1 + 0.05 * torch.randn(vocab, cols, device="cuda", generator=g)).half()
    t = torch.randint(vocab - 100, vocab, (rows,), device="cuda", generator=g)
    dx, = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), x)
    off = []
    for i in range(0, rows, 1024):
        p = torch.softmax(x.detach()[i:i + 1024].double() @ w.double().T, 1)
        p[torch.arange(len(p)), t[i:i + 1024]] -= 1
        off.append(dx[i:i + 1024].double() - p @ w.double())
    assert abs(torch.cat(off).mean().item()) < 2.0 ** -12


def test_gradients_of_wide_fp16_rows_over_several_pieces():
    """fp16, rows of ordinary width, a vocabulary in two pieces of 25 000 columns: within what one rounding of the exact
    result is off and a fifth, norm against norm (dz's rounding alone: a twelfth at most)."""
    rows, cols, vocab = 8192, 512, 50001
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(rows, cols, device="cuda", generator=g).half().requires_grad_()
    w = (2 / cols ** 0.5 * torch.randn(vocab, cols, device="cuda", generator=g)).half().requires_grad_()
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    dx, dw = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), (x, w))
    want_x, want_w = torch.empty_like(x, dtype=torch.float64), torch.zeros_like(w, dtype=torch.float64)
    for i in range(0, rows, 2048):
        xd = x.detach()[i:i + 2048].double()
        p = torch.softmax(xd @ w.detach().double().T, 1)
        p[torch.arange(len(p)), t[i:i + 2048]] -= 1
        want_x[i:i + 2048] = p @ w.detach().double()
        want_w += p.T @ xd
    for got, want in ((dx, want_x), (dw, want_w)):
        assert (got.double() - want).norm() <= 1.2 * (want.half().double() - want).norm()


def test_gradients_of_very_wide_rows():
    """Logits of more columns than one accumulator adds: p from the same kind of sums as the loss."""
    rows, cols, vocab = 200, 40000, 600
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16().requires_grad_()
    w = (2 / cols ** 0.5 * torch.randn(vocab, cols, device="cuda", generator=g)).bfloat16().requires_grad_()
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    t[5] = -100
    outs = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), (x, w))
    want = reference(x.detach(), w.detach(), t, torch.ones(rows, device="cuda"))
    for got, exact, magnitudes in zip(outs, want[:2], want[2:]):
        assert within(got, exact, magnitudes, torch.bfloat16, 0)


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 16, 17])
@pytest.mark.parametrize("cols,out", [(10000, 10000), (768, 50257), (4096, 6001)])
@pytest.mark.parametrize("blocks", [True, False])
def test_few_rows_of_large_weights(rows, cols, out, blocks):
    """Products of few rows by whichever kernel the weight's size and the scales call for: each group of 128 is exact up to the tensor
    cores' additions (within 10 * 2^-23 of its terms' magnitudes), the groups are added with rounding (or by eight warps and
    then added)."""
    g = torch.Generator(device="cuda").manual_seed(8)
    a = q8.pack(torch.randn(rows, cols, device="cuda", generator=g), "e4m3", 128)
    w = torch.randn(out, cols, device="cuda", generator=g)
    b = q8.pack_blocks(w) if blocks else q8.pack(w, "e4m3", 128)
    y = q8.matmul(a, b)
    assert torch.equal(y, q8.matmul(a, b))
    va, vb = dense_ref.values(a.codes, a.scales), dense_ref.values(b.codes, b.scales, blocks)
    tol = (10 + -(-cols // 128)) * 2.0 ** -23 * (va.abs() @ vb.abs().T)
    assert bool(((y.double() - va @ vb.T).abs() <= tol).all())


def test_entry_points_by_the_c_calls_names():
    """binding's functions of the dense calls give the bits of the calls on tensors."""
    rows, cols, vocab = 150, 200, 1000
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    w = (0.1 * torch.randn(vocab, cols, device="cuda", generator=g)).bfloat16()
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    t[3] = -100

    def scratch(n):
        return torch.empty(n, device="cuda", dtype=torch.uint8) if n else None
    for reduction, name in enumerate(("none", "sum", "mean")):
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        want = dense.linear_cross_entropy(a, b, t, reduction=name)
        up = torch.randn(want.shape, device="cuda", generator=g)
        wants = torch.autograd.grad(want, (a, b), up)
        loss, lse = torch.empty_like(want), torch.empty(rows, device="cuda")
        binding.snk_vocab_loss(x, w, binding.SNK_BF16, t, -100, rows, cols, vocab, reduction, loss, lse,
                               scratch(binding.snk_vocab_loss_scratch(rows, cols, vocab, False)))
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        binding.snk_vocab_loss_backward(x, w, binding.SNK_BF16, t, -100, lse, up, rows, cols, vocab, reduction, dx, dw,
                                        scratch(binding.snk_vocab_loss_scratch(rows, cols, vocab, True)))
        assert torch.equal(loss, want) and torch.equal(dx, wants[0]) and torch.equal(dw, wants[1])
    q, qt = q8.pack_both(x)
    codes, codes_t = torch.empty(rows, 256, device="cuda", dtype=torch.uint8)[:, :cols], torch.empty(cols, rows, device="cuda", dtype=torch.uint8)
    scales, scales_t, sums = torch.empty_like(q.scales), torch.empty_like(qt.scales), torch.empty(cols, device="cuda")
    binding.snk_q8_pack_both(x, binding.SNK_BF16, rows, cols, codes, scales, codes_t, scales_t, sums,
                             scratch(binding.snk_q8_pack_both_scratch(rows, cols)))
    assert torch.equal(codes, q.codes.view(torch.uint8)) and torch.equal(codes_t, qt.codes.view(torch.uint8))
    assert torch.equal(scales, q.scales) and torch.equal(scales_t, qt.scales)
    assert bool(((sums.double() - x.double().sum(0)).abs() <= rows * 2.0 ** -24 * x.double().abs().sum(0)).all())
    b8, b8t = q8.pack_blocks(w, transposed=True)
    bc, bt = torch.empty(vocab, cols, device="cuda", dtype=torch.uint8), torch.empty(cols, vocab, device="cuda", dtype=torch.uint8)
    bs, bst = torch.empty_like(b8.scales), torch.empty_like(b8t.scales)
    binding.snk_q8_pack_blocks(w, binding.SNK_BF16, vocab, cols, bc, bs, bt, bst)
    assert torch.equal(bc, b8.codes.contiguous().view(torch.uint8)) and torch.equal(bt, b8t.codes.contiguous().view(torch.uint8))
    assert torch.equal(bs, b8.scales) and torch.equal(bst, b8t.scales)
    for m in (rows, 5):
        y = torch.empty(m, vocab, device="cuda", dtype=torch.bfloat16)
        a = codes[:m]   # rows 256 bytes apart, the weight's 200, which is no multiple of 16
        binding.snk_q8_matmul(a, scales, bc, bs, True, m, vocab, cols, None, y, binding.SNK_BF16,
                              scratch(binding.snk_q8_matmul_scratch(m, vocab, cols, 256, 200, True)))
        assert torch.equal(y, q8.matmul(q8.Q8Tensor(q.codes[:m], q.scales[:m], 128), b8, dtype=torch.bfloat16))


@pytest.mark.parametrize("cols", [16, 9])
def test_few_rows_of_a_vocabulary_of_more_than_a_million(cols):
    """More columns than dx's ranges of K hold at a time: pieces of the vocabulary, for few rows too."""
    rows, vocab = 3, 1_300_001
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16().requires_grad_()
    w = torch.randn(vocab, cols, device="cuda", generator=g).bfloat16().requires_grad_()
    t = torch.tensor([vocab - 1, 0, 1_048_576], device="cuda")
    outs = torch.autograd.grad(dense.linear_cross_entropy(x, w, t, reduction="sum"), (x, w))
    want = reference(x.detach(), w.detach(), t, torch.ones(rows, device="cuda"))
    for got, exact, magnitudes in zip(outs, want[:2], want[2:]):
        assert within(got, exact, magnitudes, torch.bfloat16, 0)
