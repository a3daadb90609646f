"""The 8-bit activation calls refuse bad arguments on the host, before any work
is queued, and the wrappers refuse tensors that are not CUDA tensors."""
import ctypes

import pytest

from sparse_linear_layer_gb300 import binding, build

ARG, LIMIT, OK = binding.SNK_ERR_ARG, binding.SNK_ERR_LIMIT, binding.SNK_OK
P = 0x1000   # never read: every call below is refused first
F32, BF16 = binding.SNK_F32, binding.SNK_BF16
I8 = binding.SNK_Q8_INT8


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def f(x):
    return ctypes.c_float(x)


def test_pack_and_unpack(L):
    for args in [(None, F32, 1, 8, I8, 0, P, P), (P, 3, 1, 8, I8, 0, P, P), (P, F32, -1, 8, I8, 0, P, P),
                 (P, F32, 1, 0, I8, 0, P, P), (P, F32, 1, 8, 2, 0, P, P), (P, F32, 1, 8, I8, 16, P, P),
                 (P, F32, 1, 8, I8, 512, P, P), (P, F32, 1, 8, I8, 0, None, P), (P, F32, 1, 8, I8, 0, P, None),
                 (P + 2, F32, 1, 8, I8, 0, P, P), (P + 1, BF16, 1, 8, I8, 0, P, P), (P, F32, 1, 8, I8, 0, P, P + 1)]:
        assert L.snk_q8_pack(*args, None) == ARG, args
        x, dtype, rows, cols, fmt, group, codes, scales = args
        assert L.snk_q8_unpack(codes, scales, rows, cols, fmt, group, x, dtype, None) == ARG, args
        assert L.snk_gelu_q8(*args, None, None, None) == ARG, args
        assert L.snk_gelu_backward_q8(x, dtype, codes, scales, rows, cols, fmt, group, P, None) == ARG, args
    assert L.snk_gelu_q8(P, F32, 1, 8, I8, 0, P, P, P, None, None) == ARG      # kept: both or neither
    assert L.snk_gelu_backward_q8(P, F32, P, P, 1, 8, I8, 0, None, None) == ARG
    assert L.snk_q8_pack(P, F32, 2**31, 8, I8, 0, P, P, None) == LIMIT
    assert L.snk_q8_pack(None, F32, 0, 8, I8, 0, None, None, None) == OK


def test_rmsnorm(L):
    def norm(x=P, res=P, dtype=F32, gain=P, rows=1, cols=8, eps=1e-5, fmt=I8, group=0, codes=P, scales=P, total=P,
             rstd=P):
        return L.snk_rmsnorm_q8(x, res, dtype, gain, rows, cols, f(eps), fmt, group, codes, scales, total, rstd, None)

    for bad in [dict(x=None), dict(gain=None), dict(codes=None), dict(scales=None), dict(rstd=None),
                dict(total=None), dict(res=None), dict(dtype=7), dict(rows=-2), dict(cols=0), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(fmt=5), dict(group=1), dict(gain=P + 2),
                dict(res=P + 1), dict(total=P + 3), dict(rstd=P + 2)]:
        assert norm(**bad) == ARG, bad
    assert norm(rows=2**31) == LIMIT
    assert norm(rows=0, x=None) == OK


def test_rmsnorm_backward(L):
    def grad(dy=P, total=P, dtype=F32, rstd=P, gain=P, dtotal=P, rows=1000, cols=8, dx=P, dgain=P, scratch=P):
        return L.snk_rmsnorm_backward(dy, total, dtype, rstd, gain, dtotal, rows, cols, dx, dgain, scratch, None)

    for bad in [dict(dy=None), dict(total=None), dict(rstd=None), dict(gain=None), dict(dx=None),
                dict(scratch=None), dict(scratch=P + 16), dict(dtype=-1), dict(cols=0), dict(dgain=P + 2),
                dict(dtotal=P + 2)]:
        assert grad(**bad) == ARG, bad
    assert L.snk_rmsnorm_backward_scratch(0, 8) == 0
    assert L.snk_rmsnorm_backward_scratch(5, 7) == 0                     # a few rows need none
    assert L.snk_rmsnorm_backward_scratch(300, 7) == 300 * 8 * 4
    assert L.snk_rmsnorm_backward_scratch(5, 20000) == 5 * 20000 * 4     # but long ones do


def test_products(L):
    assert L.snk_forward_q8(None, P, P, I8, 0, 1, None, P, None) == ARG
    assert L.snk_backward_weight_q8(None, P, P, I8, 0, P, 1, P, None, None) == ARG


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    from sparse_linear_layer_gb300 import q8
    with pytest.raises(ValueError):
        q8.pack(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        q8.Q8Tensor(torch.zeros(2, 8, dtype=torch.int8), torch.zeros(2, 1), 0)
