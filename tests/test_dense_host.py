"""The dense operators' calls refuse bad arguments on the host, before any work is queued,
and the wrappers refuse tensors that are not CUDA tensors."""
import pytest

from sparse_linear_layer_gb300 import binding, build

ARG, LIMIT, OK = binding.SNK_ERR_ARG, binding.SNK_ERR_LIMIT, binding.SNK_OK
P = 0x1000   # never read: every call below is refused first
F32, F16, BF16 = binding.SNK_F32, binding.SNK_F16, binding.SNK_BF16


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def test_vocab_loss(L):
    def loss(x=P, w=P, dtype=BF16, target=P, rows=4, cols=8, vocab=10, reduction=2, loss=P, lse=P, scratch=P):
        return L.snk_vocab_loss(x, w, dtype, target, -100, rows, cols, vocab, reduction, loss, lse, scratch, None)

    for bad in [dict(x=None), dict(w=None), dict(target=None), dict(loss=None), dict(scratch=None), dict(dtype=F32),
                dict(dtype=5), dict(rows=-1), dict(cols=0), dict(vocab=0), dict(reduction=3), dict(reduction=-1),
                dict(x=P + 8), dict(w=P + 2), dict(target=P + 4), dict(loss=P + 2), dict(lse=P + 1), dict(scratch=P + 128)]:
        assert loss(**bad) == ARG, bad
    for big in [dict(rows=2**31), dict(cols=2**31), dict(vocab=2**31), dict(rows=2**30, vocab=2**30)]:
        assert loss(**big) == LIMIT, big
    assert loss(rows=0, x=None, target=None, loss=None, scratch=None, reduction=0) == OK


def test_vocab_loss_backward(L):
    def grad(x=P, w=P, dtype=F16, target=P, lse=P, dloss=P, rows=4, cols=8, vocab=10, reduction=2, dx=P, dw=P, scratch=P):
        return L.snk_vocab_loss_backward(x, w, dtype, target, -100, lse, dloss, rows, cols, vocab, reduction, dx, dw, scratch, None)

    for bad in [dict(x=None), dict(w=None), dict(target=None), dict(lse=None), dict(dloss=None), dict(scratch=None),
                dict(dtype=F32), dict(rows=-1), dict(cols=0), dict(vocab=-3), dict(reduction=4), dict(x=P + 2), dict(w=P + 4),
                dict(lse=P + 2), dict(dloss=P + 1), dict(dx=P + 8), dict(dw=P + 2), dict(scratch=P + 16)]:
        assert grad(**bad) == ARG, bad
    assert grad(vocab=2**31) == LIMIT
    assert grad(dx=None, dw=None) == OK
    assert grad(rows=0, x=None, dw=None) == OK


def test_matmul(L):
    def product(a=P, lda=32, sa=P, b=P, ldb=32, sb=P, blocks=1, m=4, n=5, k=20, bias=None, y=P, dtype=F32, scratch=P):
        return L.snk_q8_matmul(a, lda, sa, b, ldb, sb, blocks, m, n, k, bias, y, dtype, scratch, None)

    for bad in [dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(y=None), dict(lda=19), dict(ldb=0), dict(m=-1),
                dict(n=0), dict(k=0), dict(dtype=3), dict(dtype=-1), dict(a=P + 8), dict(b=P + 1), dict(sa=P + 2), dict(sb=P + 1),
                dict(bias=P + 2), dict(y=P + 2), dict(y=P + 1, dtype=BF16), dict(scratch=P + 64)]:
        assert product(**bad) == ARG, bad
    for big in [dict(m=2**31), dict(n=2**31), dict(k=2**31, lda=2**31, ldb=2**31), dict(m=2**30, n=2**30)]:
        assert product(**big) == LIMIT, big
    assert product(m=0, a=None, sa=None, y=None) == OK


def test_packing(L):
    def both(x=P, dtype=F32, rows=4, cols=20, codes=P, ld=20, scales=P, codes_t=P, ld_t=4, scales_t=P, sums=P, scratch=P):
        return L.snk_q8_pack_both(x, dtype, rows, cols, codes, ld, scales, codes_t, ld_t, scales_t, sums, scratch, None)

    for bad in [dict(x=None), dict(dtype=3), dict(rows=-1), dict(cols=0), dict(scales=None), dict(scales_t=None),
                dict(codes=None), dict(codes_t=None), dict(ld=19), dict(ld_t=3), dict(x=P + 2), dict(scales=P + 2),
                dict(scales_t=P + 1), dict(sums=P + 2), dict(scratch=None), dict(scratch=P + 2)]:
        assert both(**bad) == ARG, bad
    assert both(rows=2**31) == LIMIT
    assert both(codes=None, scales=None, codes_t=None, scales_t=None, sums=None, scratch=None) == OK
    assert both(rows=0, x=None, sums=None) == OK

    def blocks(w=P, dtype=F32, rows=4, cols=20, codes=P, ld=20, scales=P, codes_t=P, ld_t=4, scales_t=P):
        return L.snk_q8_pack_blocks(w, dtype, rows, cols, codes, ld, scales, codes_t, ld_t, scales_t, None)

    for bad in [dict(w=None), dict(dtype=-1), dict(cols=-1), dict(scales=None), dict(codes_t=None), dict(ld=3), dict(ld_t=0),
                dict(w=P + 1)]:
        assert blocks(**bad) == ARG, bad
    assert blocks(cols=2**31) == LIMIT
    assert L.snk_q8_pack_both_scratch(300, 10) == 3 * 10 * 4
    assert L.snk_q8_pack_both_scratch(0, 10) == 0


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    from sparse_linear_layer_gb300 import dense, q8
    with pytest.raises(ValueError):
        q8.pack_both(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        q8.pack_blocks(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        q8.Q8Blocks(torch.zeros(2, 8).to(torch.float8_e4m3fn), torch.zeros(1, 1))
    with pytest.raises(ValueError):
        dense.linear_q8(torch.zeros(2, 8), torch.zeros(3, 8))
    with pytest.raises(ValueError):
        dense.linear_cross_entropy(torch.zeros(2, 8).bfloat16(), torch.zeros(3, 8).bfloat16(), torch.zeros(2).long())
    with pytest.raises(ValueError):
        dense.VocabularyHead(8, 10, dtype=torch.float32, device="cpu")
