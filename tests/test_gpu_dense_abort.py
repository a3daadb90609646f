"""Kernels of the dense operators whose bounded waits run out leave NaN, never a wrong number.

A build with a short limit (SNK_TC_WAIT_CYCLES, and SNK_TC_WAIT_POLL so that it is kept) makes
some waits give up, as in a real stall: what has been issued is waited for (with the separate
drain limit), and what a role could not compute is NaN.  Each call runs in that build, in
a child process, several times on the same inputs, and each of its outputs has to be NaN or the
bits that the library gives; what the outputs held before is in none of them.  A plain operation
afterwards shows that the context still works.  Every wait is bounded and every copy that was
issued is waited for before a CTA exits, so nothing here faults a GPU."""
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.gpu_util import need_gpu  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def packing(run):
    """Codes count where their scale is a number."""
    from sparse_linear_layer_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(1)
    for dtype, d in ((torch.bfloat16, binding.SNK_BF16), (torch.float32, binding.SNK_F32)):
        rows, cols = 4000, 3200   # five tiles and more of a block of threads
        x = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
        codes, codes_t = (torch.full(s, 99, device="cuda", dtype=torch.uint8) for s in ((rows, cols), (cols, rows)))
        scales, scales_t = torch.full((rows, 25), 777.0, device="cuda"), torch.full((cols, 32), 777.0, device="cuda")
        sums = torch.full((cols,), 777.0, device="cuda")
        scratch = torch.full((binding.snk_q8_pack_both_scratch(rows, cols),), 99, device="cuda", dtype=torch.uint8)
        binding.snk_q8_pack_both(x, d, rows, cols, codes, scales, codes_t, scales_t, sums, scratch)
        run(f"both {dtype}", scales=scales, scales_t=scales_t, sums=sums,
            codes=torch.where(scales.repeat_interleave(128, 1).isnan(), float("nan"), codes.float()),
            codes_t=torch.where(scales_t.repeat_interleave(128, 1)[:, :rows].isnan(), float("nan"), codes_t.float()))
        codes.fill_(99), codes_t.fill_(99)
        scales, scales_t = torch.full((32, 25), 777.0, device="cuda"), torch.full((25, 32), 777.0, device="cuda")
        binding.snk_q8_pack_blocks(x, d, rows, cols, codes, scales, codes_t, scales_t)
        wide = scales.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)
        run(f"blocks {dtype}", scales=scales, scales_t=scales_t, codes=torch.where(wide.isnan(), float("nan"), codes.float()),
            codes_t=torch.where(wide.T.isnan(), float("nan"), codes_t.float()))


def loss(run):
    """Tiles of every kind: one row, one tile of rows, pairs, dual tiles, accumulators that take turns."""
    from sparse_linear_layer_gb300 import binding
    for rows, cols, vocab in ((1, 768, 20000), (100, 320, 30000), (200, 1100, 20000), (1500, 256, 20000), (2000, 2048, 9000)):
        x, w, t = vocabulary(rows, cols, vocab)
        out, lse = torch.full((rows,), 777.0, device="cuda"), torch.full((rows,), 777.0, device="cuda")
        scratch = torch.full((binding.snk_vocab_loss_scratch(rows, cols, vocab, False),), 99, device="cuda", dtype=torch.uint8)
        for reduction in (0, 2):
            binding.snk_vocab_loss(x, w, binding.SNK_BF16, t, -100, rows, cols, vocab, reduction, out, lse, scratch)
            run(f"loss {rows} {reduction}", loss=out[:rows if reduction == 0 else 1].clone(), lse=lse.clone())


def gradients(run):
    from sparse_linear_layer_gb300 import binding
    for rows, cols, vocab in ((100, 320, 30000), (200, 1101, 9000), (1500, 256, 20000), (3000, 768, 9000)):
        x, w, t = vocabulary(rows, cols, vocab)
        t[::7] = -100
        lse = torch.logsumexp(x.float() @ w.float().T, 1)
        dx, dw = torch.full_like(x, 777.0), torch.full_like(w, 777.0)
        scratch = torch.full((binding.snk_vocab_loss_scratch(rows, cols, vocab, True),), 99, device="cuda", dtype=torch.uint8)
        binding.snk_vocab_loss_backward(x, w, binding.SNK_BF16, t, -100, lse, torch.ones(1, device="cuda"), rows, cols, vocab, 2,
                                        dx, dw, scratch)
        run(f"gradients {rows}", dx=dx, dw=dw)
        dx.fill_(777.0)
        binding.snk_vocab_loss_backward(x, w, binding.SNK_BF16, t, -100, lse, torch.ones(rows, device="cuda"), rows, cols, vocab, 0,
                                        dx, None, scratch)
        run(f"gradient {rows}", dx=dx)


def products(run):
    """Pairs and single CTAs, scales of blocks and of rows, ranges of K, outputs by TMA and by plain stores."""
    from sparse_linear_layer_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(3)
    for m, n, k in ((40, 9000, 1000), (300, 1001, 1000), (2000, 4096, 1536), (512, 512, 8192), (100, 777, 700)):
        for blocks in (True, False):
            a, b = (torch.randn(r, k, device="cuda", generator=g).to(torch.float8_e4m3fn) for r in (m, n))
            gk = -(-k // 128)
            sa = torch.rand(m, gk, device="cuda", generator=g)
            sb = torch.rand(-(-n // 128) if blocks else n, gk, device="cuda", generator=g)
            for dtype, d in ((torch.float32, binding.SNK_F32), (torch.bfloat16, binding.SNK_BF16)):
                y = torch.full((m, n), 777.0, device="cuda", dtype=dtype)
                need = binding.snk_q8_matmul_scratch(m, n, k, k, k, blocks)
                scratch = torch.full((need,), 99, device="cuda", dtype=torch.uint8) if need else None
                binding.snk_q8_matmul(a, sa, b, sb, blocks, m, n, k, None, y, d, scratch)
                run(f"product {m} {blocks} {dtype}", y=y)


def vocabulary(rows, cols, vocab):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    w = (2 / cols ** 0.5 * torch.randn(vocab, cols, device="cuda", generator=g)).bfloat16()
    return x, w, torch.randint(0, vocab, (rows,), device="cuda", generator=g)


CALLS = {"packing": packing, "loss": loss, "gradients": gradients, "products": products}


def child(name, variant, path):
    from sparse_linear_layer_gb300 import binding
    binding.LIB_PATH = variant
    want, result = torch.load(path), {"nan": 0, "numbers": 0, "wrong": {}}

    def check(what, **outputs):
        for k, got in outputs.items():
            nan = got.isnan()
            wrong = int((~nan & (got != want[f"{what} {k}"].cuda())).sum())
            result["nan"] += int(nan.sum())
            result["numbers"] += int((~nan).sum())
            if wrong:
                result["wrong"][f"{what} {k}"] = wrong
    for _ in range(3):
        CALLS[name](check)
    torch.cuda.synchronize()
    result["fine"] = int(torch.arange(1000, device="cuda").sum())
    print("RESULT " + json.dumps(result))


@pytest.fixture(scope="module", params=[0, 5000])
def variant(request):
    """The library with a short limit of its waits, in cycles."""
    need_gpu()
    from sparse_linear_layer_gb300 import build
    out = os.path.join(build.PKG, "_build", f"waitlimit{request.param}", "libsnk.so")
    build.build(extra_flags=[f"-DSNK_TC_WAIT_CYCLES={request.param}", "-DSNK_TC_WAIT_POLL"], out=out)
    return request.param, out


@pytest.mark.parametrize("name", sorted(CALLS))
def test_nan_or_right(name, variant, tmp_path):
    limit, lib = variant
    want = {}

    def keep(what, **outputs):
        for k, v in outputs.items():
            assert not bool(v.isnan().any()), (what, k)
            want[f"{what} {k}"] = v.cpu()
    CALLS[name](keep)
    path = str(tmp_path / "want.pt")
    torch.save(want, path)
    code = f"import sys; sys.path.insert(0, {ROOT!r}); from tests.test_gpu_dense_abort import child; child({name!r}, {lib!r}, {path!r})"
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600, cwd=ROOT)
    lines = [ln for ln in p.stdout.splitlines() if ln.startswith("RESULT ")]
    assert p.returncode == 0 and lines, p.stdout[-2000:] + p.stderr[-4000:]
    res = json.loads(lines[-1][len("RESULT "):])
    assert not res["wrong"] and res["fine"] == 499500, res
    # (no copy is there at once; with the other limit about half of the outputs are numbers, by the GPU's clock)
    assert limit > 0 or res["nan"] > 0, res
