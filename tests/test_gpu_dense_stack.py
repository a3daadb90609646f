"""The dense operators as a model uses them: token rows through a dense projection on 8 bits,
a truly sparse MLP block on 8-bit activations, and the vocabulary head; trained by a step with
all gradients, and served from 8-bit weights."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_linear_layer_gb300 import dense, q8  # noqa: E402
from sparse_linear_layer_gb300.mlp import SparseMLP  # noqa: E402
from sparse_linear_layer_gb300.module import SET  # noqa: E402
from tests import dense_ref  # noqa: E402
from tests.gpu_util import need_gpu  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


class Model(torch.nn.Module):
    def __init__(self, features=128, hidden=512, vocab=1000):
        super().__init__()
        torch.manual_seed(0)
        self.embed = torch.nn.Parameter(torch.randn(vocab, features, device="cuda"))
        self.mix = dense.Q8Linear(features, features)
        self.mlp = SparseMLP(features, hidden, 0.9, format="e4m3", group=128)
        self.head = dense.VocabularyHead(features, vocab)

    def hidden(self, tokens):
        x = self.embed[tokens]
        y, total = self.mlp(self.mix(x), x)
        return y + total

    def forward(self, tokens, target):
        return self.head(self.hidden(tokens), target)


def batch(seed, rows=6, length=50, vocab=1000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, vocab, (rows, length), device="cuda", generator=g)
    target = (tokens * 7 + 3) % vocab
    target[torch.rand(rows, length, device="cuda", generator=g) < 0.2] = -100
    return tokens, target


def test_training_step_and_its_gradients():
    model = Model()
    tokens, target = batch(1)
    loss = model(tokens, target)
    loss.backward()
    for name, p in model.named_parameters():
        assert p.grad is not None and p.grad.shape == p.shape and bool(torch.isfinite(p.grad).all()), name
        assert float(p.grad.float().abs().max()) > 0, name
    # the head's part against 64 bits, on the hidden states that it was given
    with torch.no_grad():
        h = model.hidden(tokens).reshape(-1, 128).to(torch.bfloat16)
    t = target.reshape(-1)
    n = int((t != -100).sum())
    row, _, _ = dense_ref.loss(h, model.head.weight.detach(), t)
    # logits of 128 columns: 8 steps of 2^-23 of a sum of magnitudes below 64
    assert abs(loss.item() - row.sum().item() / n) < 2 * 8 * 2.0 ** -23 * 64 + 1e-5
    _, dw, _, mag = dense_ref.loss_gradient(h, model.head.weight.detach(), t, torch.full((t.numel(),), 1.0 / n, device="cuda"))
    err = (model.head.weight.grad.double() - dw).abs()
    # dz and the result rounded to 16 bits, p off by twice a logit's error (below 2^-13 here)
    assert bool((err <= (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * dw.abs()).all())


def test_steps_with_an_optimizer_and_a_restructure():
    model = Model()
    opt = torch.optim.SGD(model.parameters(), lr=1e-2)
    schedule = SET(model.mlp.sparse_layers(), every=2)
    before = [p.detach().clone() for p in model.parameters()]
    for i in range(4):
        loss = model(*batch(i))
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        schedule.step()
        assert torch.isfinite(loss)
    assert schedule.restructures == 2
    assert all(not torch.equal(a, p) for a, p in zip(before, model.parameters()))


def test_captured_training_step():
    """Loss and gradients of a projection and the head in one graph, replayed on new tokens."""
    mix, head = dense.Q8Linear(96, 128), dense.VocabularyHead(128, 700)
    x = torch.randn(200, 96, device="cuda")
    target = torch.randint(0, 700, (200,), device="cuda")
    leaves = [*mix.parameters(), *head.parameters()]

    def step():
        loss = head(mix(x), target)
        return (loss, *torch.autograd.grad(loss, leaves))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    x.copy_(torch.randn(200, 96, device="cuda"))
    target.copy_(torch.randint(0, 700, (200,), device="cuda"))
    graph.replay()
    got = [o.detach().clone() for o in outs]
    for a, b in zip(got, step()):
        assert torch.equal(a, b.detach())


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
def test_serving_from_the_norm(rows):
    """The last norm writes 8 bits, the head multiplies them with the weight packed once."""
    head = dense.VocabularyHead(256, 1111)
    gain = 1 + 0.1 * torch.randn(256, device="cuda")
    x = torch.randn(rows, 256, device="cuda").bfloat16()
    n, _, _ = q8.rmsnorm(x, gain, format="e4m3", group=128)
    w8 = head.pack()
    logits = head.logits(n, w8)
    a, b = dense_ref.values(n.codes, n.scales), dense_ref.values(w8.codes, w8.scales, True)
    want, mag = a @ b.T, a.abs() @ b.abs().T
    assert bool(((logits.double() - want).abs() <= 12 * 2.0 ** -23 * mag + 2.0 ** -24 * want.abs()).all())
    assert torch.equal(logits, head.logits(n)) and torch.equal(logits, head.logits(n.dequantize(), w8))
    assert head.logits(n, w8, dtype=torch.bfloat16).dtype == torch.bfloat16
    # after the weight changes, a new pack is a new answer; the old one still answers for the old weight
    with torch.no_grad():
        head.weight.mul_(2)
    assert torch.equal(head.logits(n, w8), logits) and torch.equal(head.logits(n), 2 * logits)
