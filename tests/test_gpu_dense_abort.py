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


CALLS = {"packing": packing}


def child(name, variant, path):
    from sparse_linear_layer_gb300 import binding
    binding.LIB_PATH = variant
    want, result = torch.load(path), {"nan": 0, "wrong": {}}

    def check(what, **outputs):
        for k, got in outputs.items():
            nan = got.isnan()
            wrong = int((~nan & (got != want[f"{what} {k}"].cuda())).sum())
            result["nan"] += int(nan.sum())
            if wrong:
                result["wrong"][f"{what} {k}"] = wrong
    for _ in range(5):
        CALLS[name](check)
    torch.cuda.synchronize()
    result["fine"] = int(torch.arange(1000, device="cuda").sum())
    print("RESULT " + json.dumps(result))


@pytest.fixture(scope="module", params=[0, 1000])
def variant(request):
    """The library with a short limit of its waits, in cycles."""
    need_gpu()
    from sparse_linear_layer_gb300 import build
    out = os.path.join(build.PKG, "_build", f"waitlimit{request.param}", "libsnk.so")
    build.build(extra_flags=[f"-DSNK_TC_WAIT_CYCLES={request.param}", "-DSNK_TC_WAIT_POLL"], out=out)
    return out


@pytest.mark.parametrize("name", sorted(CALLS))
def test_nan_or_right(name, variant, tmp_path):
    want = {}

    def keep(what, **outputs):
        for k, v in outputs.items():
            assert not bool(v.isnan().any()), (what, k)
            want[f"{what} {k}"] = v.cpu()
    CALLS[name](keep)
    path = str(tmp_path / "want.pt")
    torch.save(want, path)
    code = f"import sys; sys.path.insert(0, {ROOT!r}); from tests.test_gpu_dense_abort import child; child({name!r}, {variant!r}, {path!r})"
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600, cwd=ROOT)
    lines = [ln for ln in p.stdout.splitlines() if ln.startswith("RESULT ")]
    assert p.returncode == 0 and lines, p.stdout[-2000:] + p.stderr[-4000:]
    res = json.loads(lines[-1][len("RESULT "):])
    print(name, res)
    assert not res["wrong"] and res["fine"] == 499500, res
    assert res["nan"] > 0, res
