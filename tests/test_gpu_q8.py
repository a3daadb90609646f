"""8-bit activations on the GPU: pack / unpack, GELU and its gradient, the norm
and its gradient, against the references of q8_ref.py.

Tolerances (u = 2^-24, the fp32 rounding unit), fixed from the arithmetic:
- pack: codes and scales are defined step by step in fp32: equal bits.
- unpack: one fp32 product, then one rounding to the output type: equal bits.
- GELU, norm -> 8 bits: half a code step around the 64-bit value, plus the
  error of the fp32 value before rounding: GELU 16 u max(|h|, 1); norm
  (n_sum + 8) u |y| with n_sum <= 32 + 5 + 32 additions in a row's sum.  A
  scale may move by the same relative error.
- GELU gradient: 32 u |da| (1 + |h|) and half a unit of the output type.
- norm gradient: dx 96 u times the sum of its terms' magnitudes and half a unit
  of the output type; dgain (rows + 64) u times that of its terms.
"""
import numpy as np
import pytest

from tests import q8_ref as ref
from tests.gpu_util import dev, host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_UNIT = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


def data(rng, rows, cols, scale=1.0):
    x = rng.standard_normal((rows, cols)) * scale
    x *= 1 + 9 * (rng.random(cols) < 0.05)
    return x.astype(np.float32)


def on_gpu(torch, x, dtype):
    """x rounded to dtype on the GPU, and as fp32 values."""
    t = dev(x, torch).to(getattr(torch, dtype))
    return t, t.float().cpu().numpy()


def code_values(q):
    return q.codes.float().cpu().numpy().astype(np.float64)


def same_bits(a, b, what):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    ok = (a == b) | (np.isnan(a) & np.isnan(b))
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} differ, first at {tuple(np.argwhere(~ok)[0])}"


SHAPES = [(1, 1), (1, 768), (3, 7), (5, 64), (2, 257), (9, 500), (4, 1000), (1, 3072), (33, 768), (3, 5001),
          (2, 10000), (300, 1032), (2, 16392), (2, 40004)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
def test_pack_and_unpack_bits(torch, dtype, fmt, group):
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(11)
    for rows, cols in SHAPES:
        t, x = on_gpu(torch, data(rng, rows, cols), dtype)
        q = q8.pack(t, fmt, group)
        codes, scales = ref.pack(x, fmt, group)
        same_bits(host(q.scales), scales, f"scales {rows}x{cols}")
        same_bits(code_values(q), codes, f"codes {rows}x{cols}")
        v = ref.values(codes, scales, group)
        for out in ("float32", "float16", "bfloat16"):
            got = q8.unpack(q, getattr(torch, out)).float().cpu().numpy()
            want = torch.from_numpy(v.astype(np.float32)).to(getattr(torch, out)).float().numpy()
            same_bits(got, want, f"values {rows}x{cols} {out}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 256])
def test_pack_of_extreme_values(torch, fmt, group):
    """Zero rows, tiny and huge magnitudes, infinities and NaN stay in their
    own group; the type's largest value; -0."""
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(12)
    x = data(rng, 8, 520)
    x[0] = 0
    x[1] = -0.0
    x[2] *= np.float32(1e-35)
    x[3] *= np.float32(1e-42)
    x[4, 7] = np.inf
    x[5, 300] = np.nan
    x[6, 519] = -np.inf
    x[7] = np.float32(3.4028235e38) * np.sign(x[7])
    q = q8.pack(dev(x, torch), fmt, group)
    codes, scales = ref.pack(x, fmt, group)
    same_bits(host(q.scales), scales, "scales")
    same_bits(code_values(q), codes, "codes")
    v = host(q8.unpack(q))
    same_bits(v, ref.values(codes, scales, group), "values")
    if group:
        assert np.isfinite(v[4, group:]).all() and np.isnan(v[4, :group]).all()
    else:
        assert np.isnan(v[4]).all() and np.isfinite(v[0]).all()


@pytest.mark.parametrize("off", [1, 3])
def test_unaligned_and_sliced_buffers(torch, off):
    """Tensors that start at an odd element: no wide access may be used."""
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(13)
    rows, cols = 6, 512
    for dtype in ("float32", "bfloat16"):
        flat, x = on_gpu(torch, data(rng, 1, rows * cols + off), dtype)
        t, x = flat[0, off:].view(rows, cols), x[0, off:].reshape(rows, cols)
        for group in (0, 64):
            q = q8.pack(t, "int8", group)
            codes, scales = ref.pack(x, "int8", group)
            same_bits(code_values(q), codes, "codes")
            # codes at an odd byte
            room = torch.empty(rows * cols + off, dtype=torch.int8, device="cuda")
            odd = room[off:].view(rows, cols)
            odd.copy_(q.codes)
            got = q8.unpack(q8.Q8Tensor(odd, q.scales, group))
            same_bits(host(got), ref.values(codes, scales, group), "values")
            gain = torch.ones(cols + off, device="cuda")[off:]
            n, _, rstd = q8.rmsnorm(t, gain, residual=t, group=group)
            n0, _, rstd0 = q8.rmsnorm(t.clone(), gain.clone(), residual=t.clone(), group=group)
            # both layouts add the same squares, in another order
            np.testing.assert_allclose(host(rstd), host(rstd0), rtol=80 * U)
            assert (n.codes.int() - n0.codes.int()).abs().max() <= 1
    with pytest.raises(ValueError):
        q8.pack(torch.zeros(8, 64, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        q8.pack(torch.zeros(64, 8, device="cuda").T)


def check_rounded(q, y, err, fmt, group, what):
    """The 8-bit matrix is y (64 bits, fp32 error err) to half a code step."""
    codes, scales = code_values(q), host(q.scales)
    v = ref.values(codes, scales, group)
    width = group or y.shape[1]
    m = np.stack([np.abs(y[:, i:i + width]).max(1) for i in range(0, y.shape[1], width)], 1)
    em = np.stack([err[:, i:i + width].max(1) for i in range(0, y.shape[1], width)], 1)
    top = float(ref.TOP[fmt])
    assert (np.abs(scales - m / top) <= (em + 2 * U * m) / top).all(), what + " scales"
    step = ref.half_step(codes, scales, fmt, group)
    bad = np.abs(v - y) > step * (1 + 1e-5) + err + 8 * U * np.abs(y)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}"


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_gelu_and_its_gradient(torch, dtype, fmt, group):
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(14)
    for rows, cols in [(1, 1), (2, 77), (5, 768), (64, 3072), (3, 10001), (2, 33000)]:
        t, x = on_gpu(torch, data(rng, rows, cols), dtype)
        a, kept = q8.gelu(t, fmt, group, keep=True)
        codes, scales = ref.pack(x, fmt, group)
        same_bits(host(kept.scales), scales, "kept scales")
        same_bits(code_values(kept), codes, "kept codes")
        h = x.astype(np.float64)
        check_rounded(a, ref.gelu(h), 16 * U * np.maximum(np.abs(h), 1), fmt, group, f"gelu {rows}x{cols}")
        alone = q8.gelu(t, fmt, group)
        assert torch.equal(alone.codes.view(torch.uint8), a.codes.view(torch.uint8))
        g, gv = on_gpu(torch, data(rng, rows, cols, 1e-3), dtype)
        dh = q8.gelu_backward(g, kept).float().cpu().numpy()
        hk = ref.values(codes, scales, group)
        want = gv * ref.gelu_slope(hk)
        bound = 32 * U * np.abs(gv) * (1 + np.abs(hk)) + HALF_UNIT[dtype] * np.abs(want) + 1e-40
        assert (np.abs(dh - want) <= bound).all(), f"dh {rows}x{cols}"
        same = g.clone()
        assert torch.equal(q8.gelu_backward(same, kept, out=same), q8.gelu_backward(g, kept))


def test_gelu_gradient_is_that_of_gelu():
    """The reference slope against differences of the reference GELU."""
    h = np.linspace(-6, 6, 241)
    d = 1e-5
    np.testing.assert_allclose(ref.gelu_slope(h), (ref.gelu(h + d) - ref.gelu(h - d)) / (2 * d), rtol=0, atol=1e-9)


NORM_SHAPES = [(1, 1), (1, 768), (2, 5), (7, 500), (3, 1000), (33, 768), (5, 3072), (2, 10000), (2, 33000),
               (611, 264), (2, 17001)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("fmt,group", [("int8", 0), ("e4m3", 0), ("int8", 32), ("e4m3", 128), ("int8", 256)])
def test_rmsnorm(torch, dtype, fmt, group):
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(15)
    for rows, cols in NORM_SHAPES:
        t, x = on_gpu(torch, data(rng, rows, cols), dtype)
        r, rv = on_gpu(torch, data(rng, rows, cols, 3.0), dtype)
        gain = (1 + 0.1 * rng.standard_normal(cols)).astype(np.float32)
        for res in (r, None):
            q, total, rstd = q8.rmsnorm(t, dev(gain, torch), residual=res, eps=1e-5, format=fmt, group=group)
            want = t + res if res is not None else t
            assert torch.equal(total, want), "total"
            rr = want.double().cpu().numpy()
            y, rs = ref.rmsnorm(rr, gain.astype(np.float64), 1e-5)
            n_sum = 32 + 5 + 32
            np.testing.assert_allclose(host(rstd), rs, rtol=(n_sum + 4) * U)
            check_rounded(q, y, (n_sum + 8) * U * np.abs(y), fmt, group, f"norm {rows}x{cols}")


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_rmsnorm_backward(torch, dtype):
    from sparse_linear_layer_gb300 import q8
    rng = np.random.default_rng(16)
    for rows, cols in NORM_SHAPES:
        r, rv = on_gpu(torch, data(rng, rows, cols), dtype)
        dt, dtv = on_gpu(torch, data(rng, rows, cols, 1e-2), dtype)
        dy = data(rng, rows, cols, 1e-2)
        gain = (1 + 0.1 * rng.standard_normal(cols)).astype(np.float32)
        rstd = (1 / np.sqrt((rv.astype(np.float64) ** 2).mean(1) + 1e-5)).astype(np.float32)
        for d, dv in ((dt, dtv), (None, 0.0 * dtv)):
            dx, dgain = q8.rmsnorm_backward(dev(dy, torch), r, dev(rstd, torch), dev(gain, torch), dtotal=d)
            f8 = lambda a: np.asarray(a, np.float64)
            wx, wg, ax, ag = ref.rmsnorm_backward(f8(dy), f8(rv), f8(rstd), f8(gain), f8(dv))
            got = dx.float().cpu().numpy()
            bad = np.abs(got - wx) > 96 * U * ax + HALF_UNIT[dtype] * np.abs(wx) + 2.0 ** -25 * (dtype == "float16")
            assert not bad.any(), f"dx {rows}x{cols}: {int(bad.sum())} off"
            assert (np.abs(host(dgain) - wg) <= (rows + 64) * U * ag + 1e-40).all(), f"dgain {rows}x{cols}"


def test_rmsnorm_gradient_is_that_of_the_norm():
    """The reference gradient against differences of the reference norm, both
    paths of total included."""
    rng = np.random.default_rng(17)
    rows, cols, eps = 3, 11, 1e-3
    r, dy, dt = (rng.standard_normal((rows, cols)) for _ in range(3))
    gain = 1 + 0.1 * rng.standard_normal(cols)

    def loss(r, gain):
        return (dy * ref.rmsnorm(r, gain, eps)[0]).sum() + (dt * r).sum()

    _, rstd = ref.rmsnorm(r, gain, eps)
    dx, dgain, _, _ = ref.rmsnorm_backward(dy, r, rstd, gain, dt)
    d = 1e-6
    for i in range(rows):
        for c in range(cols):
            e = np.zeros_like(r)
            e[i, c] = d
            assert abs((loss(r + e, gain) - loss(r - e, gain)) / (2 * d) - dx[i, c]) < 1e-7
    for c in range(cols):
        e = np.zeros_like(gain)
        e[c] = d
        assert abs((loss(r, gain + e) - loss(r, gain - e)) / (2 * d) - dgain[c]) < 1e-7


def test_zero_and_non_finite_rows_of_the_norm(torch):
    from sparse_linear_layer_gb300 import q8
    x = torch.ones(4, 256, device="cuda")
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    q, _, rstd = q8.rmsnorm(x, torch.ones(256, device="cuda"), eps=1e-6, group=64)
    v = host(q8.unpack(q))
    assert (v[0] == 0).all() and np.isclose(host(rstd)[0], 1e3)
    assert np.isnan(v[1]).all()                        # the row's norm is NaN
    assert np.isnan(v[2, 192:]).all() and (v[2, :192] == 0).all()   # x / inf = 0, inf / inf = NaN
    assert np.allclose(v[3], 1, atol=1e-2)


def test_no_rows(torch):
    from sparse_linear_layer_gb300 import q8
    x = torch.empty(0, 96, device="cuda")
    gain = torch.ones(96, device="cuda")
    a, kept = q8.gelu(x, keep=True, group=32)
    q, total, rstd = q8.rmsnorm(x, gain, residual=x)
    dx, dgain = q8.rmsnorm_backward(x, total, rstd, gain)
    assert a.codes.shape == (0, 96) and a.scales.shape == (0, 3) and q8.unpack(q).shape == (0, 96)
    assert dx.shape == (0, 96) and (host(dgain) == 0).all() and q8.gelu_backward(x, kept).shape == (0, 96)


def test_leading_dimensions_are_rows(torch):
    from sparse_linear_layer_gb300 import q8
    x = torch.randn(2, 3, 40, device="cuda")
    gain = torch.ones(40, device="cuda")
    q, total, rstd = q8.rmsnorm(x, gain, residual=x, group=32)
    assert q.codes.shape == x.shape and q.scales.shape == (2, 3, 2) and rstd.shape == (2, 3)
    flat, _, _ = q8.rmsnorm(x.view(6, 40), gain, residual=x.view(6, 40), group=32)
    assert torch.equal(flat.codes.view(2, 3, 40), q.codes)


def test_offsets_past_32_bits(torch):
    """More than 2^31 elements: the last rows are those of a small matrix."""
    from sparse_linear_layer_gb300 import q8
    cols, rows = 16384, 131080
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB free")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(8, cols, device="cuda").bfloat16()
    x[-8:] = tail
    for group in (0, 128):
        q = q8.pack(x, "int8", group)
        t = q8.pack(tail, "int8", group)
        assert torch.equal(q.codes[-8:], t.codes) and torch.equal(q.scales[-8:], t.scales)
        assert not q.codes[:8].any()
        assert torch.equal(q8.unpack(q, torch.bfloat16)[-8:], q8.unpack(t, torch.bfloat16))
        del q, t
    gain = torch.ones(cols, device="cuda")
    n, _, rstd = q8.rmsnorm(x, gain)
    m, _, rm = q8.rmsnorm(tail, gain)
    assert (n.codes[-8:].int() - m.codes.int()).abs().max() <= 1
    torch.testing.assert_close(rstd[-8:], rm, rtol=80 * U, atol=0)


def test_results_repeat_and_streams(torch):
    from sparse_linear_layer_gb300 import q8
    rows, cols = 777, 768
    x = torch.randn(rows, cols, device="cuda")
    gain = torch.ones(cols, device="cuda")
    dy = torch.randn(rows, cols, device="cuda")
    q, total, rstd = q8.rmsnorm(x, gain, residual=x)
    first = q8.rmsnorm_backward(dy, total, rstd, gain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q2, total2, rstd2 = q8.rmsnorm(x, gain, residual=x)
        again = q8.rmsnorm_backward(dy, total2, rstd2, gain)
    side.synchronize()
    assert torch.equal(q.codes, q2.codes) and torch.equal(rstd, rstd2)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_stream_argument_owns_what_the_call_allocates(torch):
    """Memory that the current stream still writes is not taken for another stream's
    outputs or scratch."""
    from sparse_linear_layer_gb300 import q8
    rows, cols = 2048, 768
    x = torch.randn(rows, cols, device="cuda")
    gain = torch.ones(cols, device="cuda")
    want, _, rstd = q8.rmsnorm(x, gain)
    grads = q8.rmsnorm_backward(x, x, rstd, gain)
    nbytes = sorted({rows * cols, rows * 4, rows * cols * 4, cols * 4, 1 << 21})
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        pending = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in nbytes for _ in range(3)]
        torch.cuda._sleep(50_000_000)   # some 25 ms
        for t in pending:
            t.fill_(77)
        del pending, t                  # free for the current stream, still to be written
        q, _, r = q8.rmsnorm(x, gain, stream=stream)
        dx, dgain = q8.rmsnorm_backward(x, x, r, gain, stream=stream)
        back = q8.unpack(q, stream=stream)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales) and torch.equal(r, rstd)
        assert torch.equal(dx, grads[0]) and torch.equal(dgain, grads[1])
        assert torch.equal(back, q8.unpack(want))


def test_graph_capture(torch):
    from sparse_linear_layer_gb300 import q8
    x = torch.randn(64, 3072, device="cuda")
    kept0 = q8.gelu(x, keep=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, kept = q8.gelu(x, keep=True)
        dh = q8.gelu_backward(x, kept)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.codes, kept0[0].codes) and torch.equal(dh, q8.gelu_backward(x, kept0[1]))


def test_refusals(torch):
    from sparse_linear_layer_gb300 import binding, q8
    x = torch.randn(4, 64, device="cuda")
    gain = torch.ones(64, device="cuda")
    for bad in (dict(format="fp4"), dict(group=48), dict(group=-1)):
        with pytest.raises(ValueError):
            q8.pack(x, **bad)
    for t in (x.double(), x.cpu(), x.int()):
        with pytest.raises(ValueError):
            q8.pack(t)
    with pytest.raises(ValueError):
        q8.rmsnorm(x, gain[:32])
    with pytest.raises(ValueError):
        q8.rmsnorm(x, gain.half())
    with pytest.raises(ValueError):
        q8.rmsnorm(x, gain, residual=x.half())
    with pytest.raises(binding.SnkError) as e:
        q8.rmsnorm(x, gain, eps=0.0)
    assert e.value.status == binding.SNK_ERR_ARG
    q = q8.pack(x)
    with pytest.raises(ValueError):
        q8.Q8Tensor(q.codes, q.scales, 32)       # too few scales for groups of 32
    with pytest.raises(ValueError):
        q8.Q8Tensor(q.codes.float(), q.scales, 0)
    with pytest.raises(ValueError):
        q8.gelu_backward(x[:2], q)
    with pytest.raises(ValueError):
        q8.rmsnorm_backward(x.half(), x, gain[:4], gain)
