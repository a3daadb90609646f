"""The norm and its gradient: outputs on the buffers that include/snk.h lets them
share, and row counts on both sides of every choice of kernel.  Tolerances as in
test_gpu_q8.py: a row's sum has at most 3 * 8 products per lane, 5 additions over
the lanes and 32 over the warps, under the 32 + 5 + 32 stated there; dgain adds a
row at a time at worst, (rows + 64) u."""
import numpy as np
import pytest

from tests import q8_ref as ref
from tests.gpu_util import dev, host, need_gpu
from tests.test_gpu_q8 import HALF_UNIT, U, check_rounded, data, on_gpu

pytestmark = pytest.mark.gpu

TYPES = {"float32": 0, "float16": 1, "bfloat16": 2}   # SNK_F32, SNK_F16, SNK_BF16


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


def backward(torch, dy, total, rstd, gain, dtotal, dx):
    from sparse_linear_layer_gb300 import binding
    rows, cols = dy.shape
    dgain = torch.empty(cols, device="cuda")
    n = binding.snk_rmsnorm_backward_scratch(rows, cols)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    binding.snk_rmsnorm_backward(dy, total, TYPES[str(total.dtype)[6:]], rstd, gain, dtotal, rows, cols, dx, dgain,
                                 scratch)
    return dgain


# few rows in one launch (up to 256 rows and 2^20 elements), then one warp per row and
# several, with and without rows in flight, and rows read again for each step
@pytest.mark.parametrize("rows,cols", [(1, 768), (7, 500), (64, 768), (200, 1152), (256, 4096), (256, 4104), (257, 200),
                                       (300, 77), (333, 5000), (2500, 256), (2433, 264), (5, 20000)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gradient_over_its_own_inputs(torch, dtype, rows, cols):
    """dx may be total or dtotal: the bits of a dx of its own, every time."""
    rng = np.random.default_rng(21)
    total, tv = on_gpu(torch, data(rng, rows, cols), dtype)
    dtotal, _ = on_gpu(torch, data(rng, rows, cols, 1e-2), dtype)
    dy = dev(data(rng, rows, cols, 1e-2), torch)
    gain = dev((1 + 0.1 * rng.standard_normal(cols)).astype(np.float32), torch)
    rstd = dev((1 / np.sqrt((tv.astype(np.float64) ** 2).mean(1) + 1e-5)).astype(np.float32), torch)
    for d in (dtotal, None):
        dx = torch.empty_like(total)
        dgain = backward(torch, dy, total, rstd, gain, d, dx)
        for _ in range(10):
            over = total.clone()
            assert torch.equal(backward(torch, dy, over, rstd, gain, d, over), dgain), "dgain, dx over total"
            assert torch.equal(over, dx), "dx over total"
        if d is not None:
            over = dtotal.clone()
            assert torch.equal(backward(torch, dy, total, rstd, gain, over, over), dgain), "dgain, dx over dtotal"
            assert torch.equal(over, dx), "dx over dtotal"


@pytest.mark.parametrize("rows,cols", [(1, 768), (7, 500), (300, 264), (2500, 768), (700, 9000), (3, 20000)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("group", [0, 64])
def test_norm_over_its_own_inputs(torch, dtype, rows, cols, group):
    """total may be x or residual."""
    from sparse_linear_layer_gb300 import binding, q8
    rng = np.random.default_rng(22)
    x, _ = on_gpu(torch, data(rng, rows, cols), dtype)
    residual, _ = on_gpu(torch, data(rng, rows, cols, 3.0), dtype)
    gain = dev((1 + 0.1 * rng.standard_normal(cols)).astype(np.float32), torch)
    want, total, rstd = q8.rmsnorm(x, gain, residual=residual, group=group)
    for over_x in (True, False):
        a, r = x.clone(), residual.clone()
        over = a if over_x else r
        codes, scales, rs = torch.empty_like(want.codes), torch.empty_like(want.scales), torch.empty_like(rstd)
        binding.snk_rmsnorm_q8(a, r, TYPES[dtype], gain, rows, cols, 1e-5, binding.SNK_Q8_INT8, group, codes, scales,
                               over, rs)
        assert torch.equal(over, total) and torch.equal(rs, rstd)
        assert torch.equal(codes, want.codes) and torch.equal(scales, want.scales)


# One warp per row with rows in flight starts at 2 * 152 * 8 = 2432 rows (norm: up to
# 768 columns, gradient: up to 256), several warps at 304; two tiles per warp from
# 8200 columns; none of these row counts is a multiple of the slots times the grid.
MANY_ROWS = [(2500, 768), (5001, 520), (2441, 200), (2433, 256), (300, 200), (700, 77), (257, 768), (310, 10000),
             (257, 9001), (3001, 301)]


@pytest.mark.parametrize("rows,cols", MANY_ROWS)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_norm_of_many_rows(torch, dtype, rows, cols):
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(23)
    x, _ = on_gpu(torch, data(rng, rows, cols), dtype)
    residual, _ = on_gpu(torch, data(rng, rows, cols, 3.0), dtype)
    gain = (1 + 0.1 * rng.standard_normal(cols)).astype(np.float32)
    for res in (residual, None):
        want = x + res if res is not None else x
        y, rs = ref.rmsnorm(want.double().cpu().numpy(), gain.astype(np.float64), 1e-5)
        for fmt, group in (("int8", 0), ("e4m3", 128)):
            q, total, rstd = q8.rmsnorm(x, dev(gain, torch), residual=res, eps=1e-5, format=fmt, group=group)
            assert torch.equal(total, want), "total"
            np.testing.assert_allclose(host(rstd), rs, rtol=(32 + 5 + 32 + 4) * U)
            check_rounded(q, y, (32 + 5 + 32 + 8) * U * np.abs(y), fmt, group, f"norm {rows}x{cols}")


@pytest.mark.parametrize("rows,cols", MANY_ROWS)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_gradient_of_many_rows(torch, dtype, rows, cols):
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(24)
    total, tv = on_gpu(torch, data(rng, rows, cols), dtype)
    dt, dtv = on_gpu(torch, data(rng, rows, cols, 1e-2), dtype)
    dy = data(rng, rows, cols, 1e-2)
    gain = (1 + 0.1 * rng.standard_normal(cols)).astype(np.float32)
    rstd = (1 / np.sqrt((tv.astype(np.float64) ** 2).mean(1) + 1e-5)).astype(np.float32)
    f8 = lambda a: np.asarray(a, np.float64)
    for d, dv in ((dt, dtv), (None, 0.0 * dtv)):
        dx, dgain = q8.rmsnorm_backward(dev(dy, torch), total, dev(rstd, torch), dev(gain, torch), dtotal=d)
        wx, wg, ax, ag = ref.rmsnorm_backward(f8(dy), f8(tv), f8(rstd), f8(gain), f8(dv))
        bad = np.abs(dx.float().cpu().numpy() - wx) > \
            96 * U * ax + HALF_UNIT[dtype] * np.abs(wx) + 2.0 ** -25 * (dtype == "float16")
        assert not bad.any(), f"dx {rows}x{cols}: {int(bad.sum())} off"
        assert (np.abs(host(dgain) - wg) <= (rows + 64) * U * ag + 1e-40).all(), f"dgain {rows}x{cols}"
