"""Thin ctypes binding over libsnk: the C-ABI entry points under the same names.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are passed by device pointer, streams by handle.  PyTorch
serves as the device-memory allocator and stream provider.  If the library
has not been built, loading fails loudly; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
# the in-tree library that build.py writes; nothing selects another one
LIB_PATH = os.path.join(_PKG, "libsnk.so")
OPS_PATH = os.path.join(_PKG, "_q8ops.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "snk.h")

SNK_OK, SNK_ERR_ARG, SNK_ERR_DUP, SNK_ERR_RANGE = 0, 1, 2, 3
SNK_ERR_CUDA, SNK_ERR_OOM, SNK_ERR_NOSPACE, SNK_ERR_LIMIT = 4, 5, 6, 7
SNK_F32, SNK_F16, SNK_BF16 = 0, 1, 2
SNK_Q8_INT8, SNK_Q8_E4M3 = 0, 1

_lock = threading.Lock()
_lib = None
_raw_stream = None
_ops = None


class SnkError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call} failed: {snk_status_string(status)} (status {status})")
        self.status = status


def lib():
    """Load libsnk.so (built by ``sparse_linear_layer_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libsnk.so is not built ({LIB_PATH}); run "
                               "sparse_linear_layer_gb300.build.build() first")
        L = ctypes.CDLL(LIB_PATH)
        i64, u64, f32, P, I = (ctypes.c_int64, ctypes.c_uint64, ctypes.c_float,
                               ctypes.c_void_p, ctypes.c_int)
        L.snk_create.argtypes = [ctypes.POINTER(P), i64, i64, i64, P, P, P, P]
        L.snk_forward.argtypes = [P, P, i64, P, P, P]
        L.snk_backward_input.argtypes = [P, P, i64, P, P]
        L.snk_backward_weight.argtypes = [P, P, P, i64, P, P, P]
        L.snk_prune_regrow.argtypes = [P, f32, u64, P]
        L.snk_prune_regrow_gradient.argtypes = [P, f32, P, P, i64, P]
        L.snk_destroy.argtypes = [P]
        L.snk_status_string.argtypes = [I]
        L.snk_status_string.restype = ctypes.c_char_p
        L.snk_get_shape.argtypes = [P, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                    ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.snk_copy_topology.argtypes = [P, P, P, P, P, P]
        L.snk_check.argtypes = [P, P]
        L.snk_forward_csr_noalloc.argtypes = [i64, i64, i64, P, P, P, P, i64, P, P, P]
        L.snk_pcsr_build.argtypes = [P, I, P]
        L.snk_pcsr_info.argtypes = [P, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                    ctypes.POINTER(i64), P]
        L.snk_pcsr_copy.argtypes = [P, P, P, P, P, P, P]
        L.snk_pcsr_insert.argtypes = [P, i64, P, P, P, P]
        L.snk_pcsr_delete.argtypes = [P, i64, P, P, P]
        L.snk_pcsr_compact.argtypes = [P, P]
        L.snk_pcsr_export.argtypes = [P, P, P, P, i64, ctypes.POINTER(i64), P]
        L.snk_q8_pack.argtypes = [P, I, i64, i64, I, I, P, P, P]
        L.snk_q8_unpack.argtypes = [P, P, i64, i64, I, I, P, I, P]
        L.snk_gelu_q8.argtypes = [P, I, i64, i64, I, I, P, P, P, P, P]
        L.snk_gelu_backward_q8.argtypes = [P, I, P, P, i64, i64, I, I, P, P]
        L.snk_rmsnorm_q8.argtypes = [P, P, I, P, i64, i64, f32, I, I, P, P, P, P, P]
        L.snk_rmsnorm_backward_scratch.argtypes = [i64, i64]
        L.snk_rmsnorm_backward_scratch.restype = i64
        L.snk_rmsnorm_backward.argtypes = [P, P, I, P, P, P, i64, i64, P, P, P, P]
        L.snk_forward_q8.argtypes = [P, P, P, I, I, i64, P, P, P]
        L.snk_backward_weight_q8.argtypes = [P, P, P, I, I, P, i64, P, P, P]
        L.snk_q8_pack_both_scratch.argtypes = [i64, i64]
        L.snk_q8_pack_both_scratch.restype = i64
        L.snk_q8_pack_both.argtypes = [P, I, i64, i64, P, i64, P, P, i64, P, P, P, P]
        L.snk_q8_pack_blocks.argtypes = [P, I, i64, i64, P, i64, P, P, i64, P, P]
        L.snk_q8_matmul_scratch.argtypes = [i64, i64, i64, i64, i64, I]
        L.snk_q8_matmul_scratch.restype = i64
        L.snk_q8_matmul.argtypes = [P, i64, P, P, i64, P, I, i64, i64, i64, P, P, I, P, P]
        L.snk_vocab_loss_scratch.argtypes = [i64, i64, i64, I]
        L.snk_vocab_loss_scratch.restype = i64
        L.snk_vocab_loss.argtypes = [P, P, I, P, i64, i64, i64, i64, I, P, P, P, P]
        L.snk_vocab_loss_backward.argtypes = [P, P, I, P, i64, P, P, i64, i64, i64, I, P, P, P, P]
        for name in ("snk_create", "snk_forward", "snk_backward_input", "snk_backward_weight",
                     "snk_prune_regrow", "snk_prune_regrow_gradient", "snk_destroy",
                     "snk_get_shape", "snk_copy_topology", "snk_check", "snk_forward_csr_noalloc",
                     "snk_pcsr_build", "snk_pcsr_info", "snk_pcsr_copy", "snk_pcsr_insert",
                     "snk_pcsr_delete", "snk_pcsr_compact", "snk_pcsr_export", "snk_q8_pack",
                     "snk_q8_unpack", "snk_gelu_q8", "snk_gelu_backward_q8", "snk_rmsnorm_q8",
                     "snk_rmsnorm_backward", "snk_forward_q8", "snk_backward_weight_q8",
                     "snk_q8_pack_both", "snk_q8_pack_blocks", "snk_q8_matmul", "snk_vocab_loss", "snk_vocab_loss_backward"):
            getattr(L, name).restype = I
        _lib = L
        return L


def ops():
    """The native module that makes the calls on 8-bit matrices and the vocabulary loss on torch tensors
    (csrc/q8_ops.cpp), bound to the same library."""
    global _ops
    if _ops is None:
        lib()
        if not os.path.exists(OPS_PATH):
            raise RuntimeError(f"_q8ops.so is not built ({OPS_PATH}); run "
                               "sparse_linear_layer_gb300.build.build() first")
        import torch  # noqa: F401  (the module has no run path: torch's libraries have to be there already)
        from . import _q8ops
        _q8ops.load(LIB_PATH, SnkError)
        _ops = _q8ops
    return _ops


def declared_symbols():
    """Function names declared in include/snk.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(snk_\w+)\s*\(", text, re.M)))


def _check(status: int, call: str):
    if status != SNK_OK:
        raise SnkError(status, call)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return current_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def current_stream(device: int) -> int:
    """The handle of torch's current stream on the device."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        # without building a Stream object, where torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def snk_status_string(status: int) -> str:
    return lib().snk_status_string(status).decode()


def snk_create(out_features: int, in_features: int, values, rows, cols, stream=None) -> int:
    """Bind a layer to (values, rows, cols); sorts them in place.  Returns the handle."""
    h = ctypes.c_void_p()
    nnz = values.numel() if hasattr(values, "numel") else int(values)
    _check(lib().snk_create(ctypes.byref(h), out_features, in_features, nnz, _ptr(values),
                            _ptr(rows), _ptr(cols), _stream(stream)), "snk_create")
    return h.value


def snk_forward(handle: int, X, bias, Y, stream=None, batch: int | None = None):
    b = X.shape[0] if batch is None else batch
    _check(lib().snk_forward(handle, _ptr(X), b, _ptr(bias), _ptr(Y), _stream(stream)),
           "snk_forward")


def snk_backward_input(handle: int, dY, dX, stream=None, batch: int | None = None):
    b = dY.shape[0] if batch is None else batch
    _check(lib().snk_backward_input(handle, _ptr(dY), b, _ptr(dX), _stream(stream)),
           "snk_backward_input")


def snk_backward_weight(handle: int, X, dY, dW, db=None, stream=None, batch: int | None = None):
    b = X.shape[0] if batch is None else batch
    _check(lib().snk_backward_weight(handle, _ptr(X), _ptr(dY), b, _ptr(dW), _ptr(db),
                                     _stream(stream)), "snk_backward_weight")


def snk_prune_regrow(handle: int, zeta: float, seed: int, stream=None):
    _check(lib().snk_prune_regrow(handle, float(zeta), seed & (2**64 - 1), _stream(stream)),
           "snk_prune_regrow")


def snk_prune_regrow_gradient(handle: int, zeta: float, X, dY, stream=None,
                              batch: int | None = None):
    b = X.shape[0] if batch is None else batch
    _check(lib().snk_prune_regrow_gradient(handle, float(zeta), _ptr(X), _ptr(dY), b,
                                           _stream(stream)), "snk_prune_regrow_gradient")


def snk_destroy(handle: int):
    _check(lib().snk_destroy(handle), "snk_destroy")


def snk_check(handle: int, stream=None):
    """Synchronise the stream and raise SnkError(SNK_ERR_LIMIT) if a
    tensor-core kernel of this handle stopped on a wait limit since the last
    check (its outputs were written as NaN)."""
    _check(lib().snk_check(handle, _stream(stream)), "snk_check")


def snk_get_shape(handle: int):
    o, i, n, v = (ctypes.c_int64() for _ in range(4))
    _check(lib().snk_get_shape(handle, ctypes.byref(o), ctypes.byref(i), ctypes.byref(n),
                               ctypes.byref(v)), "snk_get_shape")
    return o.value, i.value, n.value, v.value


def snk_copy_topology(handle: int, row_ptr=None, col_ptr=None, rows_c=None, perm=None,
                      stream=None):
    _check(lib().snk_copy_topology(handle, _ptr(row_ptr), _ptr(col_ptr), _ptr(rows_c),
                                   _ptr(perm), _stream(stream)), "snk_copy_topology")


def snk_forward_csr_noalloc(out_features: int, in_features: int, row_ptr, cols, values, X, bias,
                            Y, stream=None, batch: int | None = None):
    """Forward product on a caller's CSR without any device allocation (the
    library's fixed scratch array is used instead)."""
    b = X.shape[0] if batch is None else batch
    nnz = values.numel() if hasattr(values, "numel") else 0
    _check(lib().snk_forward_csr_noalloc(out_features, in_features, nnz, _ptr(row_ptr), _ptr(cols),
                                         _ptr(values), _ptr(X), b, _ptr(bias), _ptr(Y),
                                         _stream(stream)), "snk_forward_csr_noalloc")


def snk_pcsr_build(handle: int, padding_pct: int = 20, stream=None):
    _check(lib().snk_pcsr_build(handle, int(padding_pct), _stream(stream)), "snk_pcsr_build")


def snk_pcsr_info(handle: int, stream=None):
    """(used_slots, n_live, version)"""
    u, n, v = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().snk_pcsr_info(handle, ctypes.byref(u), ctypes.byref(n), ctypes.byref(v),
                               _stream(stream)), "snk_pcsr_info")
    return u.value, n.value, v.value


def snk_pcsr_copy(handle: int, slot_values=None, slot_cols=None, row_start=None, row_nnz=None,
                  row_capacity=None, stream=None):
    _check(lib().snk_pcsr_copy(handle, _ptr(slot_values), _ptr(slot_cols), _ptr(row_start),
                               _ptr(row_nnz), _ptr(row_capacity), _stream(stream)),
           "snk_pcsr_copy")


def snk_pcsr_insert(handle: int, rows, cols, values, stream=None):
    _check(lib().snk_pcsr_insert(handle, rows.numel(), _ptr(rows), _ptr(cols), _ptr(values),
                                 _stream(stream)), "snk_pcsr_insert")


def snk_pcsr_delete(handle: int, rows, cols, stream=None):
    _check(lib().snk_pcsr_delete(handle, rows.numel(), _ptr(rows), _ptr(cols), _stream(stream)),
           "snk_pcsr_delete")


def snk_pcsr_compact(handle: int, stream=None):
    _check(lib().snk_pcsr_compact(handle, _stream(stream)), "snk_pcsr_compact")


def snk_pcsr_export(handle: int, values, rows, cols, stream=None) -> int:
    """Canonical live triple into the given tensors; returns nnz."""
    n = ctypes.c_int64()
    _check(lib().snk_pcsr_export(handle, _ptr(values), _ptr(rows), _ptr(cols), values.numel(),
                                 ctypes.byref(n), _stream(stream)), "snk_pcsr_export")
    return n.value


def snk_q8_pack(x, dtype: int, rows: int, cols: int, format: int, group: int, codes, scales,
                stream=None):
    _check(lib().snk_q8_pack(_ptr(x), dtype, rows, cols, format, group, _ptr(codes), _ptr(scales),
                             _stream(stream)), "snk_q8_pack")


def snk_q8_unpack(codes, scales, rows: int, cols: int, format: int, group: int, x, dtype: int,
                  stream=None):
    _check(lib().snk_q8_unpack(_ptr(codes), _ptr(scales), rows, cols, format, group, _ptr(x), dtype,
                               _stream(stream)), "snk_q8_unpack")


def snk_gelu_q8(x, dtype: int, rows: int, cols: int, format: int, group: int, codes, scales,
                kept_codes=None, kept_scales=None, stream=None):
    _check(lib().snk_gelu_q8(_ptr(x), dtype, rows, cols, format, group, _ptr(codes), _ptr(scales),
                             _ptr(kept_codes), _ptr(kept_scales), _stream(stream)), "snk_gelu_q8")


def snk_gelu_backward_q8(da, dtype: int, codes, scales, rows: int, cols: int, format: int,
                         group: int, dh, stream=None):
    _check(lib().snk_gelu_backward_q8(_ptr(da), dtype, _ptr(codes), _ptr(scales), rows, cols, format,
                                      group, _ptr(dh), _stream(stream)), "snk_gelu_backward_q8")


def snk_rmsnorm_q8(x, residual, dtype: int, gain, rows: int, cols: int, eps: float, format: int,
                   group: int, codes, scales, total, rstd, stream=None):
    _check(lib().snk_rmsnorm_q8(_ptr(x), _ptr(residual), dtype, _ptr(gain), rows, cols, eps, format,
                                group, _ptr(codes), _ptr(scales), _ptr(total), _ptr(rstd),
                                _stream(stream)), "snk_rmsnorm_q8")


def snk_rmsnorm_backward_scratch(rows: int, cols: int) -> int:
    """Bytes of scratch that snk_rmsnorm_backward needs."""
    return lib().snk_rmsnorm_backward_scratch(rows, cols)


def snk_rmsnorm_backward(dy, total, dtype: int, rstd, gain, dtotal, rows: int, cols: int, dx, dgain,
                         scratch, stream=None):
    _check(lib().snk_rmsnorm_backward(_ptr(dy), _ptr(total), dtype, _ptr(rstd), _ptr(gain),
                                      _ptr(dtotal), rows, cols, _ptr(dx), _ptr(dgain), _ptr(scratch),
                                      _stream(stream)), "snk_rmsnorm_backward")


def snk_forward_q8(handle: int, codes, scales, format: int, group: int, batch: int, bias, Y,
                   stream=None):
    _check(lib().snk_forward_q8(handle, _ptr(codes), _ptr(scales), format, group, batch, _ptr(bias),
                                _ptr(Y), _stream(stream)), "snk_forward_q8")


def snk_backward_weight_q8(handle: int, codes, scales, format: int, group: int, dY, batch: int, dW,
                           db=None, stream=None):
    _check(lib().snk_backward_weight_q8(handle, _ptr(codes), _ptr(scales), format, group, _ptr(dY),
                                        batch, _ptr(dW), _ptr(db), _stream(stream)),
           "snk_backward_weight_q8")


def _rows_ptr(t):
    """(pointer, row stride) of a matrix whose rows are contiguous."""
    if t is None:
        return None, 0
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("a matrix with contiguous rows is needed")
    return t.data_ptr(), t.stride(0)


def snk_q8_pack_both_scratch(rows: int, cols: int) -> int:
    """Bytes of scratch that snk_q8_pack_both needs for sums."""
    return lib().snk_q8_pack_both_scratch(rows, cols)


def snk_q8_pack_both(x, dtype: int, rows: int, cols: int, codes=None, scales=None, codes_t=None, scales_t=None,
                     sums=None, scratch=None, stream=None):
    _check(lib().snk_q8_pack_both(_ptr(x), dtype, rows, cols, *_rows_ptr(codes), _ptr(scales), *_rows_ptr(codes_t),
                                  _ptr(scales_t), _ptr(sums), _ptr(scratch), _stream(stream)), "snk_q8_pack_both")


def snk_q8_pack_blocks(w, dtype: int, rows: int, cols: int, codes=None, scales=None, codes_t=None, scales_t=None,
                       stream=None):
    _check(lib().snk_q8_pack_blocks(_ptr(w), dtype, rows, cols, *_rows_ptr(codes), _ptr(scales), *_rows_ptr(codes_t),
                                    _ptr(scales_t), _stream(stream)), "snk_q8_pack_blocks")


def snk_q8_matmul_scratch(m: int, n: int, k: int, lda: int, ldb: int, b_blocks: bool) -> int:
    """Bytes of scratch that snk_q8_matmul needs."""
    return lib().snk_q8_matmul_scratch(m, n, k, lda, ldb, int(b_blocks))


def snk_q8_matmul(a, a_scales, b, b_scales, b_blocks: bool, m: int, n: int, k: int, bias, y, dtype: int, scratch=None,
                  stream=None):
    _check(lib().snk_q8_matmul(*_rows_ptr(a), _ptr(a_scales), *_rows_ptr(b), _ptr(b_scales), int(b_blocks), m, n, k,
                               _ptr(bias), _ptr(y), dtype, _ptr(scratch), _stream(stream)), "snk_q8_matmul")


def snk_vocab_loss_scratch(rows: int, cols: int, vocab: int, backward: bool) -> int:
    """Bytes of scratch that snk_vocab_loss (snk_vocab_loss_backward) needs."""
    return lib().snk_vocab_loss_scratch(rows, cols, vocab, int(backward))


def snk_vocab_loss(x, weight, dtype: int, target, ignore: int, rows: int, cols: int, vocab: int, reduction: int,
                   loss, lse, scratch, stream=None):
    _check(lib().snk_vocab_loss(_ptr(x), _ptr(weight), dtype, _ptr(target), ignore, rows, cols, vocab, reduction,
                                _ptr(loss), _ptr(lse), _ptr(scratch), _stream(stream)), "snk_vocab_loss")


def snk_vocab_loss_backward(x, weight, dtype: int, target, ignore: int, lse, dloss, rows: int, cols: int, vocab: int,
                            reduction: int, dx, dweight, scratch, stream=None):
    _check(lib().snk_vocab_loss_backward(_ptr(x), _ptr(weight), dtype, _ptr(target), ignore, _ptr(lse), _ptr(dloss),
                                         rows, cols, vocab, reduction, _ptr(dx), _ptr(dweight), _ptr(scratch),
                                         _stream(stream)), "snk_vocab_loss_backward")


class SparseLinear:
    """Convenience owner of one layer: keeps the caller-side tensors alive for
    the handle's lifetime and allocates outputs with torch."""

    def __init__(self, out_features: int, in_features: int, values, rows, cols, stream=None):
        self.out_features, self.in_features = out_features, in_features
        self.values, self.rows, self.cols = values, rows, cols
        self.handle = snk_create(out_features, in_features, values, rows, cols, stream)

    @property
    def nnz(self) -> int:
        return self.values.numel()

    @property
    def topology_version(self) -> int:
        return snk_get_shape(self.handle)[3]

    def forward(self, X, bias=None, out=None, stream=None):
        import torch
        Y = out if out is not None else torch.empty((X.shape[0], self.out_features),
                                                    dtype=torch.float32, device=X.device)
        snk_forward(self.handle, X, bias, Y, stream)
        return Y

    def backward_input(self, dY, out=None, stream=None):
        import torch
        dX = out if out is not None else torch.empty((dY.shape[0], self.in_features),
                                                     dtype=torch.float32, device=dY.device)
        snk_backward_input(self.handle, dY, dX, stream)
        return dX

    def backward_weight(self, X, dY, with_bias: bool = False, out=None, stream=None):
        import torch
        dW = out if out is not None else torch.empty_like(self.values)
        db = torch.empty(self.out_features, dtype=torch.float32, device=dY.device) if with_bias else None
        snk_backward_weight(self.handle, X, dY, dW, db, stream)
        return (dW, db) if with_bias else dW

    def forward_q8(self, X, bias=None, out=None, stream=None):
        """forward() with X an 8-bit matrix (q8.Q8Tensor, [batch, in])."""
        return ops().forward(self.handle, self.out_features, self.in_features, X.codes, X.scales, X.group, bias, out,
                             stream)

    def backward_weight_q8(self, X, dY, with_bias: bool = False, out=None, stream=None):
        """backward_weight() with X an 8-bit matrix (q8.Q8Tensor, [batch, in])."""
        dW, db = ops().backward_weight(self.handle, self.out_features, self.in_features, self.nnz, X.codes, X.scales,
                                       X.group, dY, with_bias, out, stream)
        return (dW, db) if with_bias else dW

    def prune_regrow(self, zeta: float, seed: int, stream=None):
        snk_prune_regrow(self.handle, zeta, seed, stream)

    def prune_regrow_gradient(self, zeta: float, X, dY, stream=None):
        snk_prune_regrow_gradient(self.handle, zeta, X, dY, stream)

    def pcsr(self):
        """The Padded-CSR view as host-readable torch tensors (slot arrays cut
        to the used slots)."""
        import torch
        dev = self.values.device
        used, live, version = snk_pcsr_info(self.handle)
        out = dict(slot_values=torch.empty(used, dtype=torch.float32, device=dev),
                   slot_cols=torch.empty(used, dtype=torch.int32, device=dev),
                   row_start=torch.empty(self.out_features, dtype=torch.int32, device=dev),
                   row_nnz=torch.empty(self.out_features, dtype=torch.int32, device=dev),
                   row_capacity=torch.empty(self.out_features, dtype=torch.int32, device=dev))
        snk_pcsr_copy(self.handle, out["slot_values"], out["slot_cols"], out["row_start"],
                      out["row_nnz"], out["row_capacity"])
        out["n_live"], out["version"] = live, version
        return out

    def topology(self):
        import torch
        dev = self.values.device
        out = dict(row_ptr=torch.empty(self.out_features + 1, dtype=torch.int32, device=dev),
                   col_ptr=torch.empty(self.in_features + 1, dtype=torch.int32, device=dev),
                   rows_c=torch.empty(self.nnz, dtype=torch.int32, device=dev),
                   perm=torch.empty(self.nnz, dtype=torch.int32, device=dev))
        snk_copy_topology(self.handle, out["row_ptr"], out["col_ptr"], out["rows_c"], out["perm"])
        return out

    def close(self):
        if getattr(self, "handle", None):
            snk_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
