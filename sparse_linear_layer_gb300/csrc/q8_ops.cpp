// Python entry points of the 8-bit matrices' calls and of the vocabulary loss on torch
// tensors: argument checks, outputs, the current stream, and the call into libsnk, in one native
// step.  (Through ctypes and torch's Python API a call took 16 to 24 us of host
// time, most of a decoding step; here 4 to 9.)  The module is built against torch's
// headers beside libsnk.so, which load() opens; q8.py, dense.py and
// binding.py are its only users.  Wrong tensors raise ValueError, a status from libsnk raises
// binding.SnkError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "snk.h"

namespace {

PyObject* g_error = nullptr;   // binding.SnkError

struct Calls {
    decltype(&snk_q8_pack) pack = nullptr;
    decltype(&snk_q8_unpack) unpack = nullptr;
    decltype(&snk_gelu_q8) gelu = nullptr;
    decltype(&snk_gelu_backward_q8) gelu_backward = nullptr;
    decltype(&snk_rmsnorm_q8) rmsnorm = nullptr;
    decltype(&snk_rmsnorm_backward) rmsnorm_backward = nullptr;
    decltype(&snk_rmsnorm_backward_scratch) scratch = nullptr;
    decltype(&snk_forward_q8) forward = nullptr;
    decltype(&snk_backward_weight_q8) backward_weight = nullptr;
    decltype(&snk_q8_pack_both_scratch) both_scratch = nullptr;
    decltype(&snk_q8_pack_both) pack_both = nullptr;
    decltype(&snk_q8_pack_blocks) pack_blocks = nullptr;
    decltype(&snk_q8_matmul_scratch) matmul_scratch = nullptr;
    decltype(&snk_q8_matmul) matmul = nullptr;
    decltype(&snk_vocab_loss_scratch) vocab_scratch = nullptr;
    decltype(&snk_vocab_loss) vocab_loss = nullptr;
    decltype(&snk_vocab_loss_backward) vocab_loss_backward = nullptr;
    decltype(&snk_status_string) status_string = nullptr;
} g;

struct Wrong : std::runtime_error {   // becomes ValueError
    using std::runtime_error::runtime_error;
};
struct NoTangent : std::runtime_error {   // becomes NotImplementedError
    using std::runtime_error::runtime_error;
};
struct Status {
    int status;
    const char* call;
};

std::string what(const at::Tensor& t) {
    std::ostringstream s;
    s << "got " << t.scalar_type() << " " << t.sizes() << " on " << t.device() << ", strides " << t.strides();
    return s.str();
}
void require(bool ok, const char* need, const at::Tensor& t) {
    if (!ok) throw Wrong(std::string(need) + ": " + what(t));
}
const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Wrong(std::string(name) + " is a tensor");
    return THPVariable_Unpack(o);
}
// as at::Tensor, undefined for None
at::Tensor optional(PyObject* o, const char* name) { return o == Py_None ? at::Tensor() : tensor(o, name); }
int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Wrong("an integer is needed");
    return v;
}

int dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return SNK_F32;
        case at::kHalf: return SNK_F16;
        case at::kBFloat16: return SNK_BF16;
        default: throw Wrong("float32, float16 or bfloat16 is needed: " + what(t));
    }
}
int format_of(const at::Tensor& codes) {
    switch (codes.scalar_type()) {
        case at::kChar: return SNK_Q8_INT8;
        case at::kFloat8_e4m3fn: return SNK_Q8_E4M3;
        default: throw Wrong("codes are int8 or float8_e4m3fn: " + what(codes));
    }
}
int64_t groups(int64_t cols, int group) { return group ? (cols + group - 1) / group : 1; }
int group_of(PyObject* o) {
    const int64_t v = integer(o);
    if (v != 0 && v != 32 && v != 64 && v != 128 && v != 256)
        throw Wrong("group is 0, 32, 64, 128 or 256: got " + std::to_string(v));
    return (int)v;
}

// A contiguous CUDA tensor [..., cols] with cols >= 1, as a matrix.
struct Matrix {
    int64_t rows, cols;
    explicit Matrix(const at::Tensor& t) {
        require(t.is_cuda() && t.is_contiguous() && t.dim() >= 1 && t.size(-1) >= 1,
                "a contiguous CUDA tensor [..., cols] with cols >= 1 is needed", t);
        cols = t.size(-1);
        rows = t.numel() / cols;
    }
};
void require_like(const at::Tensor& t, const at::Tensor& like, const char* name) {
    if (t.sizes() != like.sizes() || t.scalar_type() != like.scalar_type() || t.device() != like.device() ||
        !t.is_contiguous())
        throw Wrong(std::string(name) + " has the shape, type and device of its matrix (" + what(like) +
                    "), contiguous: " + what(t));
}
void require_f32(const at::Tensor& t, int64_t n, const at::Device& device, const char* name) {
    if (t.scalar_type() != at::kFloat || t.numel() != n || t.device() != device || !t.is_contiguous())
        throw Wrong(std::string(name) + " is contiguous float32 with " + std::to_string(n) + " elements: " + what(t));
}
void require_codes(const Matrix& m, const at::Tensor& codes, const at::Tensor& scales, int group) {
    require_f32(scales, m.rows * groups(m.cols, group), codes.device(), "scales");
}

// The call's device and stream, both current while it lives: outputs and scratch then
// come from the allocator's blocks of that stream, which no work of another stream
// still uses or takes over.
class OnStream {
public:
    OnStream(PyObject* o, const at::Device& device) : device_(device) {
        if (o == Py_None) {
            handle_ = c10::cuda::getCurrentCUDAStream(device.index()).stream();
            return;
        }
        if (PyLong_Check(o)) {
            handle_ = (cudaStream_t)PyLong_AsVoidPtr(o);
        } else {
            PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
            if (!h) throw Wrong("stream is None, a stream or a stream handle");
            handle_ = (cudaStream_t)PyLong_AsVoidPtr(h);
            Py_DECREF(h);
        }
        if (PyErr_Occurred()) throw Wrong("stream is None, a stream or a stream handle");
        // (cudaStreamLegacy is the default stream's other name)
        stream_.reset_stream(handle_ == nullptr || handle_ == cudaStreamLegacy
                                 ? c10::cuda::getDefaultCUDAStream(device.index())
                                 : c10::cuda::getStreamFromExternal(handle_, device.index()));
    }
    void* get() const { return handle_; }

private:
    c10::cuda::CUDAGuard device_;
    c10::cuda::OptionalCUDAStreamGuard stream_;
    cudaStream_t handle_ = nullptr;
};
void check(int status, const char* call) {
    if (status != SNK_OK) throw Status{status, call};
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

struct Packed {
    at::Tensor codes, scales;
};
Packed new_packed(const at::Tensor& x, const Matrix& m, int format, int group) {
    if (format != SNK_Q8_INT8 && format != SNK_Q8_E4M3) throw Wrong("no such format");
    const auto options = x.options().requires_grad(false);
    c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
    Packed p;
    p.codes = at::empty(shape, options.dtype(format == SNK_Q8_INT8 ? at::kChar : at::kFloat8_e4m3fn));
    shape.back() = groups(m.cols, group);
    p.scales = at::empty(shape, options.dtype(at::kFloat));
    return p;
}

// New tuple of tensors (None for an undefined one).
template <typename... T>
PyObject* tuple(T&&... t) {
    PyObject* r = PyTuple_New(sizeof...(T));
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    bool ok = true;
    auto put = [&](at::Tensor&& v) {
        PyObject* o = v.defined() ? THPVariable_Wrap(std::move(v)) : Py_NewRef(Py_None);
        ok = ok && o;
        PyTuple_SET_ITEM(r, i++, o);
    };
    (put(std::forward<T>(t)), ...);
    if (!ok) Py_CLEAR(r);
    return r;
}

// C++ errors end here.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    try {
        if (!g.pack) throw Wrong("the library is not loaded");
        if (n != want) throw Wrong("wrong number of arguments");
        return f();
    } catch (const Status& s) {
        PyObject* args = Py_BuildValue("is", s.status, s.call);
        if (args) PyErr_SetObject(g_error, args);
        Py_XDECREF(args);
    } catch (const Wrong& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const NoTangent& e) {
        PyErr_SetString(PyExc_NotImplementedError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// pack(x, format, group, stream) -> (codes, scales)
PyObject* op_pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        const at::Tensor& x = tensor(a[0], "x");
        const int d = dtype_of(x), format = (int)integer(a[1]), group = group_of(a[2]);
        const Matrix m(x);
        const OnStream on(a[3], x.device());
        Packed p = new_packed(x, m, format, group);
        check(g.pack(x.data_ptr(), d, m.rows, m.cols, format, group, p.codes.data_ptr(), (float*)p.scales.data_ptr(),
                     on.get()),
              "snk_q8_pack");
        return tuple(std::move(p.codes), std::move(p.scales));
    });
}

// unpack(codes, scales, group, like, stream) -> x, of the type of the tensor `like`
// or float32 / float16 / bfloat16 by SNK_* number
PyObject* op_unpack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const at::Tensor& codes = tensor(a[0], "codes");
        const at::Tensor& scales = tensor(a[1], "scales");
        const int format = format_of(codes), group = group_of(a[2]), d = (int)integer(a[3]);
        if (d < SNK_F32 || d > SNK_BF16) throw Wrong("float32, float16 or bfloat16 is needed");
        const Matrix m(codes);
        require_codes(m, codes, scales, group);
        const OnStream on(a[4], codes.device());
        at::Tensor x = at::empty(codes.sizes(), codes.options().dtype(d == SNK_F32   ? at::kFloat
                                                                      : d == SNK_F16 ? at::kHalf
                                                                                     : at::kBFloat16));
        check(g.unpack(codes.data_ptr(), (const float*)scales.data_ptr(), m.rows, m.cols, format, group, x.data_ptr(), d,
                       on.get()),
              "snk_q8_unpack");
        return THPVariable_Wrap(std::move(x));
    });
}

// gelu(x, format, group, keep, stream) -> (codes, scales, kept codes, kept scales)
PyObject* op_gelu(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const at::Tensor& x = tensor(a[0], "x");
        const int d = dtype_of(x), format = (int)integer(a[1]), group = group_of(a[2]);
        const Matrix m(x);
        const OnStream on(a[4], x.device());
        Packed p = new_packed(x, m, format, group), kept;
        if (PyObject_IsTrue(a[3])) kept = new_packed(x, m, format, group);
        check(g.gelu(x.data_ptr(), d, m.rows, m.cols, format, group, p.codes.data_ptr(), (float*)p.scales.data_ptr(),
                     ptr(kept.codes), (float*)ptr(kept.scales), on.get()),
              "snk_gelu_q8");
        return tuple(std::move(p.codes), std::move(p.scales), std::move(kept.codes), std::move(kept.scales));
    });
}

// gelu_backward(da, codes, scales, group, out or None, stream) -> dh
PyObject* op_gelu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& da = tensor(a[0], "da");
        const at::Tensor& codes = tensor(a[1], "codes");
        const at::Tensor& scales = tensor(a[2], "scales");
        const int d = dtype_of(da), format = format_of(codes), group = group_of(a[3]);
        const Matrix m(da);
        if (da.sizes() != codes.sizes() || da.device() != codes.device() || !codes.is_contiguous())
            throw Wrong("da has the shape and device of the kept input (" + what(codes) + "): " + what(da));
        require_codes(m, codes, scales, group);
        const OnStream on(a[5], da.device());
        at::Tensor out = optional(a[4], "out");
        if (out.defined()) require_like(out, da, "out");
        else out = at::empty(da.sizes(), da.options().requires_grad(false));
        check(g.gelu_backward(da.data_ptr(), d, codes.data_ptr(), (const float*)scales.data_ptr(), m.rows, m.cols, format,
                              group, out.data_ptr(), on.get()),
              "snk_gelu_backward_q8");
        return THPVariable_Wrap(std::move(out));
    });
}

// rmsnorm(x, gain, residual or None, eps, format, group, stream)
//   -> (codes, scales, total or None, rstd)
PyObject* op_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const at::Tensor& x = tensor(a[0], "x");
        const at::Tensor& gain = tensor(a[1], "gain");
        const at::Tensor residual = optional(a[2], "residual");
        const double eps = PyFloat_AsDouble(a[3]);
        if (eps == -1.0 && PyErr_Occurred()) throw Wrong("eps is a number");
        const int d = dtype_of(x), format = (int)integer(a[4]), group = group_of(a[5]);
        const Matrix m(x);
        require_f32(gain, m.cols, x.device(), "gain");
        const OnStream on(a[6], x.device());
        const auto options = x.options().requires_grad(false);
        at::Tensor total;
        if (residual.defined()) {
            require_like(residual, x, "residual");
            total = at::empty(x.sizes(), options);
        }
        Packed p = new_packed(x, m, format, group);
        at::Tensor rstd = at::empty(x.sizes().slice(0, x.dim() - 1), options.dtype(at::kFloat));
        check(g.rmsnorm(x.data_ptr(), ptr(residual), d, (const float*)gain.data_ptr(), m.rows, m.cols, (float)eps, format,
                        group, p.codes.data_ptr(), (float*)p.scales.data_ptr(), ptr(total), (float*)rstd.data_ptr(),
                        on.get()),
              "snk_rmsnorm_q8");
        return tuple(std::move(p.codes), std::move(p.scales), std::move(total), std::move(rstd));
    });
}

// rmsnorm_backward(dy, total, rstd, gain, dtotal or None, stream) -> (dx, dgain)
PyObject* op_rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& dy = tensor(a[0], "dy");
        const at::Tensor& total = tensor(a[1], "total");
        const at::Tensor& rstd = tensor(a[2], "rstd");
        const at::Tensor& gain = tensor(a[3], "gain");
        const at::Tensor dtotal = optional(a[4], "dtotal");
        const int d = dtype_of(total);
        const Matrix m(total);
        require_f32(dy, m.rows * m.cols, total.device(), "dy");
        require_f32(rstd, m.rows, total.device(), "rstd");
        require_f32(gain, m.cols, total.device(), "gain");
        if (dtotal.defined()) require_like(dtotal, total, "dtotal");
        const OnStream on(a[5], total.device());
        const auto options = total.options().requires_grad(false);
        at::Tensor dx = at::empty(total.sizes(), options);
        at::Tensor dgain = at::empty(gain.sizes(), options.dtype(at::kFloat)), scratch;
        const int64_t bytes = g.scratch(m.rows, m.cols);
        if (bytes > 0) scratch = at::empty({bytes}, options.dtype(at::kByte));
        check(g.rmsnorm_backward((const float*)dy.data_ptr(), total.data_ptr(), d, (const float*)rstd.data_ptr(),
                                 (const float*)gain.data_ptr(), ptr(dtotal), m.rows, m.cols, dx.data_ptr(),
                                 (float*)dgain.data_ptr(), ptr(scratch), on.get()),
              "snk_rmsnorm_backward");
        return tuple(std::move(dx), std::move(dgain));
    });
}

// A layer's X: shape and columns checked against in_features.
struct LayerInput {
    const at::Tensor &codes, &scales;
    int format, group;
    Matrix m;
    LayerInput(PyObject* c, PyObject* s, PyObject* gr, int64_t in_f)
        : codes(tensor(c, "codes")), scales(tensor(s, "scales")), format(format_of(codes)), group(group_of(gr)), m(codes) {
        if (m.cols != in_f) throw Wrong("X has " + std::to_string(in_f) + " columns: " + what(codes));
        require_codes(m, codes, scales, group);
    }
};

// forward(handle, out_f, in_f, codes, scales, group, bias or None, out or None, stream) -> Y
PyObject* op_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const int64_t out_f = integer(a[1]);
        const LayerInput x(a[3], a[4], a[5], integer(a[2]));
        const at::Tensor bias = optional(a[6], "bias");
        if (bias.defined()) require_f32(bias, out_f, x.codes.device(), "bias");
        const OnStream on(a[8], x.codes.device());
        at::Tensor y = optional(a[7], "out");
        if (y.defined()) require_f32(y, x.m.rows * out_f, x.codes.device(), "out");
        else y = at::empty({x.m.rows, out_f}, x.codes.options().dtype(at::kFloat));
        check(g.forward((snk_handle)PyLong_AsVoidPtr(a[0]), x.codes.data_ptr(), (const float*)x.scales.data_ptr(), x.format,
                        x.group, x.m.rows, (const float*)ptr(bias), (float*)y.data_ptr(),
                        on.get()),
              "snk_forward_q8");
        return THPVariable_Wrap(std::move(y));
    });
}

// backward_weight(handle, out_f, in_f, nnz, codes, scales, group, dY, with_bias, out or None, stream)
//   -> (dW, db or None)
PyObject* op_backward_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const int64_t out_f = integer(a[1]), nnz = integer(a[3]);
        const LayerInput x(a[4], a[5], a[6], integer(a[2]));
        const at::Tensor& dy = tensor(a[7], "dY");
        require_f32(dy, x.m.rows * out_f, x.codes.device(), "dY");
        const OnStream on(a[10], x.codes.device());
        const auto options = x.codes.options().dtype(at::kFloat);
        at::Tensor dw = optional(a[9], "out"), db;
        if (dw.defined()) require_f32(dw, nnz, x.codes.device(), "out");
        else dw = at::empty({nnz}, options);
        if (PyObject_IsTrue(a[8])) db = at::empty({out_f}, options);
        check(g.backward_weight((snk_handle)PyLong_AsVoidPtr(a[0]), x.codes.data_ptr(), (const float*)x.scales.data_ptr(),
                                x.format, x.group, (const float*)dy.data_ptr(), x.m.rows, (float*)dw.data_ptr(),
                                (float*)ptr(db), on.get()),
              "snk_backward_weight_q8");
        return tuple(std::move(dw), std::move(db));
    });
}

// The tensor, or a copy of it where it does not start on 16 bytes.
at::Tensor aligned(const at::Tensor& t) { return ((uintptr_t)t.data_ptr() & 15) ? t.clone() : t; }

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
// Row stride of codes that only products read: whole 128-byte lines.
int64_t padded(int64_t n) { return up(n, 128); }
// New E4M3 codes [rows, cols] (pad: rows at that stride, else contiguous).
at::Tensor new_codes(int64_t rows, int64_t cols, bool pad, const at::TensorOptions& options) {
    const int64_t ld = pad ? padded(cols) : cols;
    at::Tensor t = at::empty({rows, ld}, options.dtype(at::kFloat8_e4m3fn));
    return ld == cols ? t : t.narrow(1, 0, cols);
}

// pack_both(x, want rows, want transposed, want sums, padded, stream)
//   -> (codes, scales, codes of x^T, scales of x^T, sums), None for what is not wanted
PyObject* op_pack_both(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& x = tensor(a[0], "x");
        const int d = dtype_of(x);
        const Matrix m(x);
        const bool pad = PyObject_IsTrue(a[4]);
        const OnStream on(a[5], x.device());
        const auto options = x.options().requires_grad(false);
        at::Tensor codes, scales, codes_t, scales_t, sums, scratch;
        if (PyObject_IsTrue(a[1])) {
            codes = new_codes(m.rows, m.cols, pad, options);
            scales = at::empty({m.rows, groups(m.cols, 128)}, options.dtype(at::kFloat));
        }
        if (PyObject_IsTrue(a[2])) {
            codes_t = new_codes(m.cols, m.rows, pad, options);
            scales_t = at::empty({m.cols, groups(m.rows, 128)}, options.dtype(at::kFloat));
        }
        if (PyObject_IsTrue(a[3])) {
            sums = at::empty({m.cols}, options.dtype(at::kFloat));
            scratch = at::empty({g.both_scratch(m.rows, m.cols)}, options.dtype(at::kByte));
        }
        // (no codes of an empty matrix: nothing to write)
        const bool some = m.rows > 0;
        check(g.pack_both(x.data_ptr(), d, m.rows, m.cols, some ? ptr(codes) : nullptr, codes.defined() ? codes.stride(0) : 0,
                          some ? (float*)ptr(scales) : nullptr, some ? ptr(codes_t) : nullptr,
                          codes_t.defined() ? codes_t.stride(0) : 0, some ? (float*)ptr(scales_t) : nullptr,
                          (float*)ptr(sums), ptr(scratch), on.get()),
              "snk_q8_pack_both");
        return tuple(std::move(codes), std::move(scales), std::move(codes_t), std::move(scales_t), std::move(sums));
    });
}

// pack_blocks(w, want rows, want transposed, stream) -> (codes, scales, codes of w^T, scales of w^T)
PyObject* op_pack_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        const at::Tensor& w = tensor(a[0], "w");
        const int d = dtype_of(w);
        const Matrix m(w);
        if (w.dim() != 2 || m.rows < 1) throw Wrong("w is [rows, cols] with rows >= 1: " + what(w));
        const OnStream on(a[3], w.device());
        const auto options = w.options().requires_grad(false);
        const int64_t gr = groups(m.rows, 128), gc = groups(m.cols, 128);
        at::Tensor codes, scales, codes_t, scales_t;
        if (PyObject_IsTrue(a[1])) {
            codes = new_codes(m.rows, m.cols, true, options);
            scales = at::empty({gr, gc}, options.dtype(at::kFloat));
        }
        if (PyObject_IsTrue(a[2])) {
            codes_t = new_codes(m.cols, m.rows, true, options);
            scales_t = at::empty({gc, gr}, options.dtype(at::kFloat));
        }
        check(g.pack_blocks(w.data_ptr(), d, m.rows, m.cols, ptr(codes), codes.defined() ? codes.stride(0) : 0,
                            (float*)ptr(scales), ptr(codes_t), codes_t.defined() ? codes_t.stride(0) : 0,
                            (float*)ptr(scales_t), on.get()),
              "snk_q8_pack_blocks");
        return tuple(std::move(codes), std::move(scales), std::move(codes_t), std::move(scales_t));
    });
}

// Codes of a product's operand: E4M3, rows of contiguous columns, any stride between rows.
struct Operand {
    at::Tensor codes;
    const at::Tensor& scales;
    int64_t rows, cols;
    Operand(PyObject* c, PyObject* s, const char* name) : codes(tensor(c, name)), scales(tensor(s, "scales")) {
        const bool matrix = codes.dim() == 2 && codes.stride(1) == 1 && codes.stride(0) >= codes.size(1);
        if (!codes.is_cuda() || codes.scalar_type() != at::kFloat8_e4m3fn || codes.dim() < 1 || codes.size(-1) < 1 ||
            !(matrix || codes.is_contiguous()))
            throw Wrong(std::string(name) + " has float8_e4m3fn codes [..., cols] with cols >= 1 on a CUDA device: " + what(codes));
        cols = codes.size(-1);
        rows = codes.numel() / cols;
    }
};

// matmul(a codes, a scales, b codes, b scales, b in blocks, bias or None, dtype, out or None, stream) -> y
PyObject* op_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        Operand x(a[0], a[1], "a"), w(a[2], a[3], "b");
        const bool blocks = PyObject_IsTrue(a[4]);
        const int d = (int)integer(a[6]);
        if (d < SNK_F32 || d > SNK_BF16) throw Wrong("float32, float16 or bfloat16 is needed");
        const auto device = x.codes.device();
        if (w.codes.dim() != 2 || w.rows < 1 || w.cols != x.cols || w.codes.device() != device)
            throw Wrong("b is [n, " + std::to_string(x.cols) + "] with n >= 1 on a's device: " + what(w.codes));
        const int64_t gk = groups(x.cols, 128);
        require_f32(x.scales, x.rows * gk, device, "a's scales");
        require_f32(w.scales, (blocks ? groups(w.rows, 128) : w.rows) * gk, device, "b's scales");
        const at::Tensor bias = optional(a[5], "bias");
        if (bias.defined()) require_f32(bias, w.rows, device, "bias");
        const OnStream on(a[8], device);
        const auto options = x.codes.options().requires_grad(false);
        const auto type = d == SNK_F32 ? at::kFloat : d == SNK_F16 ? at::kHalf : at::kBFloat16;
        c10::SmallVector<int64_t, 5> shape(x.codes.sizes().begin(), x.codes.sizes().end());
        shape.back() = w.rows;
        at::Tensor y = optional(a[7], "out");
        if (!y.defined()) y = at::empty(shape, options.dtype(type));
        else if (y.sizes() != at::IntArrayRef(shape) || y.scalar_type() != type || y.device() != device || !y.is_contiguous())
            throw Wrong("out is contiguous, of the product's shape, type and device: " + what(y));
        x.codes = aligned(x.codes);
        w.codes = aligned(w.codes);
        const int64_t lda = x.codes.is_contiguous() ? x.cols : x.codes.stride(0);
        const int64_t ldb = w.codes.is_contiguous() ? w.cols : w.codes.stride(0);
        at::Tensor scratch;
        const int64_t bytes = g.matmul_scratch(x.rows, w.rows, x.cols, lda, ldb, blocks);
        if (bytes > 0) scratch = at::empty({bytes}, options.dtype(at::kByte));
        check(g.matmul(x.codes.data_ptr(), lda, (const float*)x.scales.data_ptr(), w.codes.data_ptr(), ldb,
                       (const float*)w.scales.data_ptr(), blocks, x.rows, w.rows, x.cols, (const float*)ptr(bias), y.data_ptr(),
                       d, ptr(scratch), on.get()),
              "snk_q8_matmul");
        return THPVariable_Wrap(std::move(y));
    });
}

// ---- the vocabulary loss, with autograd

// Its operands.
struct Head {
    at::Tensor x, weight;
    const at::Tensor target;
    int dtype, reduction;
    int64_t ignore, rows, cols, vocab;
    Head(const at::Tensor& x_, const at::Tensor& w_, const at::Tensor& t_, int64_t ignore_, int64_t reduction_)
        : x(x_), weight(w_), target(t_), ignore(ignore_) {
        const Matrix m(x), w(weight);
        if ((x.scalar_type() != at::kHalf && x.scalar_type() != at::kBFloat16) || x.scalar_type() != weight.scalar_type())
            throw Wrong("x and weight are both float16 or both bfloat16: " + what(x) + "; " + what(weight));
        if (weight.dim() != 2 || w.cols != m.cols || weight.device() != x.device() || w.rows < 1)
            throw Wrong("weight is [vocab, " + std::to_string(m.cols) + "] with vocab >= 1 on x's device: " + what(weight));
        if (target.scalar_type() != at::kLong || target.sizes() != x.sizes().slice(0, x.dim() - 1) ||
            target.device() != x.device() || !target.is_contiguous())
            throw Wrong("target is contiguous int64 with the leading dimensions of x (" + what(x) + "): " + what(target));
        dtype = dtype_of(x);
        rows = m.rows;
        cols = m.cols;
        vocab = w.rows;
        if (reduction_ < 0 || reduction_ > 2) throw Wrong("reduction is 0 (none), 1 (sum) or 2 (mean)");
        reduction = (int)reduction_;
    }
    // on the call's stream: copies where an operand is not aligned, and scratch
    at::Tensor scratch(bool backward) {
        x = aligned(x);
        weight = aligned(weight);
        return at::empty({g.vocab_scratch(rows, cols, vocab, backward)}, x.options().requires_grad(false).dtype(at::kByte));
    }
    // (loss, lse) on the current stream
    std::pair<at::Tensor, at::Tensor> forward(void* stream) {
        const auto options = x.options().requires_grad(false).dtype(at::kFloat);
        at::Tensor lse = at::empty(target.sizes(), options);
        at::Tensor loss = reduction == 0 ? at::empty(target.sizes(), options) : at::empty({}, options);
        const at::Tensor s = scratch(false);
        check(g.vocab_loss(x.data_ptr(), weight.data_ptr(), dtype, (const int64_t*)target.data_ptr(), ignore, rows, cols, vocab,
                           reduction, (float*)loss.data_ptr(), (float*)lse.data_ptr(), ptr(s), stream),
              "snk_vocab_loss");
        return {loss, lse};
    }
    // (dx, dweight), undefined for what is not wanted
    std::pair<at::Tensor, at::Tensor> backward(const at::Tensor& lse, const at::Tensor& dloss, bool want_x, bool want_w, void* stream) {
        require_f32(lse, rows, x.device(), "lse");
        require_f32(dloss, reduction == 0 ? rows : 1, x.device(), "dloss");
        const auto options = x.options().requires_grad(false);
        at::Tensor dx, dw;
        if (want_x) dx = at::empty(x.sizes(), options);
        if (want_w) dw = at::empty(weight.sizes(), options);
        const at::Tensor s = scratch(true);
        check(g.vocab_loss_backward(x.data_ptr(), weight.data_ptr(), dtype, (const int64_t*)target.data_ptr(), ignore,
                                    (const float*)lse.data_ptr(), (const float*)dloss.data_ptr(), rows, cols, vocab, reduction,
                                    ptr(dx), ptr(dw), ptr(s), stream),
              "snk_vocab_loss_backward");
        return {dx, dw};
    }
};

// vocab_loss(x, weight, target, ignore, reduction, stream) -> (loss, lse)
PyObject* op_vocab_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        Head h(tensor(a[0], "x"), tensor(a[1], "weight"), tensor(a[2], "target"), integer(a[3]), integer(a[4]));
        const OnStream on(a[5], h.x.device());
        auto [loss, lse] = h.forward(on.get());
        return tuple(std::move(loss), std::move(lse));
    });
}

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// A backward pass: f's errors as exceptions that the engine passes on, and no second derivative
// (gradients are on in a backward pass only where one is asked for: create_graph).
template <typename F>
variable_list backward_pass(F f) {
    if (at::GradMode::is_enabled()) throw std::runtime_error("this operation has no second derivative (create_graph)");
    try {
        return f();
    } catch (const Status& s) {
        throw std::runtime_error(std::string(s.call) + " failed: " + g.status_string(s.status) + " (status " +
                                 std::to_string(s.status) + ")");
    }
}
bool wants_gradient(const at::Tensor& t) { return at::GradMode::is_enabled() && t.defined() && t.requires_grad(); }
// A tensor of forward-mode differentiation needs no gradient: without this its result would have no tangent, which
// counts as a derivative of zero.
void refuse_tangents(std::initializer_list<const at::Tensor*> inputs) {
    if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
    for (const at::Tensor* t : inputs)
        if (t->defined() && t->_fw_grad(0).defined())
            throw NoTangent("this operation has no forward-mode derivative (its gradients are those of the backward pass)");
}
void* current_stream(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

struct HeadFunction : torch::autograd::Function<HeadFunction> {
    static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, const at::Tensor& weight, const at::Tensor& target,
                              int64_t ignore, int64_t reduction) {
        Head h(x, weight, target, ignore, reduction);
        const c10::cuda::CUDAGuard on(x.device());
        auto [loss, lse] = h.forward(current_stream(x));
        ctx->save_for_backward({x, weight, target, lse});
        ctx->saved_data["ignore"] = ignore;
        ctx->saved_data["reduction"] = reduction;
        return loss;
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
        return backward_pass([&]() -> variable_list {
            if (!grads[0].defined()) return {{}, {}, {}, {}, {}};
            const auto saved = ctx->get_saved_variables();
            Head h(saved[0], saved[1], saved[2], ctx->saved_data["ignore"].toInt(), ctx->saved_data["reduction"].toInt());
            const c10::cuda::CUDAGuard on(h.x.device());
            auto [dx, dw] = h.backward(saved[3], grads[0].contiguous(), ctx->needs_input_grad(0), ctx->needs_input_grad(1),
                                       current_stream(h.x));
            return {dx, dw, {}, {}, {}};
        });
    }
};

// linear_cross_entropy(x, weight, target, ignore, reduction) -> loss, on the current stream, differentiable
PyObject* op_linear_cross_entropy(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&] {
        const at::Tensor x = tensor(a[0], "x").contiguous(), w = tensor(a[1], "weight").contiguous();
        const at::Tensor target = tensor(a[2], "target").contiguous();
        const int64_t ignore = integer(a[3]), reduction = integer(a[4]);
        refuse_tangents({&x, &w});
        if (wants_gradient(x) || wants_gradient(w))
            return THPVariable_Wrap(HeadFunction::apply(x, w, target, ignore, reduction));
        Head h(x, w, target, ignore, reduction);
        const c10::cuda::CUDAGuard on(x.device());
        return THPVariable_Wrap(h.forward(current_stream(x)).first);
    });
}

// ---- a dense layer on 8-bit matrices, with autograd

// Pieces of one allocation, 256-byte aligned.
struct Pieces {
    at::Tensor memory;
    char* at = nullptr;
    explicit Pieces(std::initializer_list<int64_t> bytes, const at::TensorOptions& options) {
        int64_t n = 0;
        for (int64_t b : bytes) n += up(b, 256);
        memory = at::empty({n}, options.dtype(at::kByte));
        at = (char*)memory.data_ptr();
    }
    template <typename T = void>
    T* take(int64_t bytes) {
        T* p = (T*)at;
        at += up(bytes, 256);
        return p;
    }
};
void product(const void* a, int64_t lda, const float* sa, const void* b, int64_t ldb, const float* sb, bool blocks, int64_t m, int64_t n,
             int64_t k, const float* bias, const at::Tensor& y, const at::TensorOptions& options, void* stream) {
    const int64_t bytes = g.matmul_scratch(m, n, k, lda, ldb, blocks);
    at::Tensor scratch;
    if (bytes > 0) scratch = at::empty({bytes}, options.dtype(at::kByte));
    check(g.matmul(a, lda, sa, b, ldb, sb, blocks, m, n, k, bias, y.data_ptr(), dtype_of(y), ptr(scratch), stream), "snk_q8_matmul");
}

// x [rows, cols] and weight [out, cols], checked.
void require_layer(const at::Tensor& x, const at::Tensor& w, const at::Tensor& bias) {
    const Matrix mx(x), mw(w);
    dtype_of(x);
    dtype_of(w);
    if (w.dim() != 2 || mw.cols != mx.cols || mw.rows < 1 || w.device() != x.device())
        throw Wrong("weight is [out, " + std::to_string(mx.cols) + "] with out >= 1 on x's device: " + what(w));
    if (bias.defined()) require_f32(bias, mw.rows, x.device(), "bias");
}
struct LayerOut {
    at::Tensor y, xt, xt_scales, wt, wt_scales;   // transposed forms: what the gradients take
};
LayerOut layer_forward(const at::Tensor& x, const at::Tensor& w, const at::Tensor& bias, bool keep_x, bool keep_w, void* stream) {
    const int64_t rows = x.size(0), cols = x.size(1), out = w.size(0), gk = groups(cols, 128);
    const auto options = x.options().requires_grad(false);
    LayerOut o;
    o.y = at::empty({rows, out}, options);
    if (keep_x) {
        o.xt = at::empty({cols, padded(rows)}, options.dtype(at::kFloat8_e4m3fn));
        o.xt_scales = at::empty({cols, groups(rows, 128)}, options.dtype(at::kFloat));
    }
    if (keep_w) {
        o.wt = at::empty({cols, padded(out)}, options.dtype(at::kFloat8_e4m3fn));
        o.wt_scales = at::empty({gk, groups(out, 128)}, options.dtype(at::kFloat));
    }
    const int64_t ld = padded(cols), nx = rows * ld, nw = out * ld, nsx = 4 * rows * gk, nsw = 4 * groups(out, 128) * gk;
    Pieces p({nx, nw, nsx, nsw}, options);
    void *cx = p.take(nx), *cw = p.take(nw);
    float *sx = p.take<float>(nsx), *sw = p.take<float>(nsw);
    if (rows == 0) return o;
    check(g.pack_both(x.data_ptr(), dtype_of(x), rows, cols, cx, ld, sx, ptr(o.xt), padded(rows), (float*)ptr(o.xt_scales), nullptr,
                      nullptr, stream),
          "snk_q8_pack_both");
    check(g.pack_blocks(w.data_ptr(), dtype_of(w), out, cols, cw, ld, sw, ptr(o.wt), padded(out), (float*)ptr(o.wt_scales), stream),
          "snk_q8_pack_blocks");
    product(cx, ld, sx, cw, ld, sw, true, rows, out, cols, (const float*)ptr(bias), o.y, options, stream);
    return o;
}

struct LayerFunction : torch::autograd::Function<LayerFunction> {
    static at::Tensor forward(AutogradContext* ctx, const at::Tensor& x, const at::Tensor& w, const std::optional<at::Tensor>& bias,
                              bool keep_x, bool keep_w) {
        const c10::cuda::CUDAGuard on(x.device());
        LayerOut o = layer_forward(x, w, bias ? *bias : at::Tensor(), keep_x, keep_w, current_stream(x));
        ctx->saved_data["bias"] = bias.has_value();
        ctx->save_for_backward({o.xt, o.xt_scales, o.wt, o.wt_scales});
        ctx->saved_data["rows"] = x.size(0);
        ctx->saved_data["cols"] = x.size(1);
        ctx->saved_data["out"] = w.size(0);
        ctx->saved_data["weight"] = (int64_t)w.scalar_type();
        return o.y;
    }
    static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
        return backward_pass([&]() -> variable_list {
            if (!grads[0].defined()) return {{}, {}, {}, {}, {}};
            const int64_t rows = ctx->saved_data["rows"].toInt(), cols = ctx->saved_data["cols"].toInt();
            const int64_t out = ctx->saved_data["out"].toInt();
            const auto weight = (at::ScalarType)ctx->saved_data["weight"].toInt();
            const auto saved = ctx->get_saved_variables();
            const at::Tensor &xt = saved[0], &xt_scales = saved[1], &wt = saved[2], &wt_scales = saved[3];
            const at::Tensor dy = grads[0].contiguous();
            const bool want_x = ctx->needs_input_grad(0), want_w = ctx->needs_input_grad(1);
            const bool want_b = ctx->saved_data["bias"].toBool() && ctx->needs_input_grad(2);
            const c10::cuda::CUDAGuard on(dy.device());
            void* stream = current_stream(dy);
            const auto options = dy.options().requires_grad(false);
            at::Tensor dx, dw, db;
            if (want_x) dx = at::empty({rows, cols}, options);
            if (want_w) dw = rows ? at::empty({out, cols}, options.dtype(weight)) : at::zeros({out, cols}, options.dtype(weight));
            if (want_b) db = at::empty({out}, options.dtype(at::kFloat));
            const int64_t ld = padded(out), ldt = padded(rows), gn = groups(out, 128), gm = groups(rows, 128);
            const int64_t nr = want_x ? rows * ld : 0, nt = want_w ? out * ldt : 0, nb = want_b ? g.both_scratch(rows, out) : 0;
            Pieces p({nr, nt, want_x ? 4 * rows * gn : 0, want_w ? 4 * out * gm : 0, nb}, options);
            void *c = p.take(nr), *ct = p.take(nt);
            float *s = p.take<float>(want_x ? 4 * rows * gn : 0), *st = p.take<float>(want_w ? 4 * out * gm : 0);
            void* parts = p.take(nb);
            const bool rx = want_x && rows, rw = want_w && rows;
            check(g.pack_both(dy.data_ptr(), dtype_of(dy), rows, out, rx ? c : nullptr, ld, rx ? s : nullptr, rw ? ct : nullptr, ldt,
                              rw ? st : nullptr, (float*)ptr(db), parts, stream),
                  "snk_q8_pack_both");
            if (rx)
                product(c, ld, s, wt.data_ptr(), padded(out), (const float*)wt_scales.data_ptr(), true, rows, cols, out, nullptr, dx,
                        options, stream);
            if (rw)
                product(ct, ldt, st, xt.data_ptr(), ldt, (const float*)xt_scales.data_ptr(), false, out, cols, rows, nullptr, dw,
                        options, stream);
            return {dx, dw, db, {}, {}};
        });
    }
};

// linear_q8(x, weight, bias or None) -> y, on the current stream, differentiable
PyObject* op_linear_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&] {
        const at::Tensor& x = tensor(a[0], "x");
        const at::Tensor w = tensor(a[1], "weight").contiguous();
        at::Tensor bias = optional(a[2], "bias");
        refuse_tangents({&x, &w, &bias});
        // a bias in 16 bits (a model converted as a whole) is added as the fp32 numbers that it holds; autograd rounds
        // its gradient, a sum in fp32, to its type
        if (bias.defined() && (bias.scalar_type() == at::kHalf || bias.scalar_type() == at::kBFloat16)) bias = bias.to(at::kFloat);
        if (x.dim() < 1 || x.size(-1) < 1 || !x.is_cuda()) throw Wrong("x is a CUDA tensor [..., cols] with cols >= 1: " + what(x));
        const at::Tensor x2 = x.dim() == 2 && x.is_contiguous() ? x : x.reshape({x.numel() / x.size(-1), x.size(-1)}).contiguous();
        require_layer(x2, w, bias);
        at::Tensor y;
        if (wants_gradient(x) || wants_gradient(w) || wants_gradient(bias)) {
            y = LayerFunction::apply(x2, w, bias.defined() ? std::optional<at::Tensor>(bias) : std::nullopt, wants_gradient(w),
                                     wants_gradient(x));
        } else {
            const c10::cuda::CUDAGuard on(x.device());
            y = layer_forward(x2, w, bias, false, false, current_stream(x)).y;
        }
        if (x.dim() != 2) {
            c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
            shape.back() = w.size(0);
            y = y.reshape(shape);
        }
        return THPVariable_Wrap(std::move(y));
    });
}

// load(path of libsnk.so, binding.SnkError)
PyObject* op_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "load(path, error)");
        return nullptr;
    }
    const char* path = PyUnicode_AsUTF8(a[0]);
    if (!path) return nullptr;
    void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!lib) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    bool ok = true;
    auto find = [&](auto& f, const char* name) {
        f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(lib, name));
        ok = ok && f;
    };
    Calls c;
    find(c.pack, "snk_q8_pack");
    find(c.unpack, "snk_q8_unpack");
    find(c.gelu, "snk_gelu_q8");
    find(c.gelu_backward, "snk_gelu_backward_q8");
    find(c.rmsnorm, "snk_rmsnorm_q8");
    find(c.rmsnorm_backward, "snk_rmsnorm_backward");
    find(c.scratch, "snk_rmsnorm_backward_scratch");
    find(c.forward, "snk_forward_q8");
    find(c.backward_weight, "snk_backward_weight_q8");
    find(c.both_scratch, "snk_q8_pack_both_scratch");
    find(c.pack_both, "snk_q8_pack_both");
    find(c.pack_blocks, "snk_q8_pack_blocks");
    find(c.matmul_scratch, "snk_q8_matmul_scratch");
    find(c.matmul, "snk_q8_matmul");
    find(c.vocab_scratch, "snk_vocab_loss_scratch");
    find(c.vocab_loss, "snk_vocab_loss");
    find(c.vocab_loss_backward, "snk_vocab_loss_backward");
    find(c.status_string, "snk_status_string");
    if (!ok) {
        PyErr_SetString(PyExc_RuntimeError, "libsnk.so lacks a call of this module");
        return nullptr;
    }
    g = c;
    Py_XSETREF(g_error, Py_NewRef(a[1]));
    Py_RETURN_NONE;
}

#define OP(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {OP("load", op_load),
                         OP("pack", op_pack),
                         OP("unpack", op_unpack),
                         OP("gelu", op_gelu),
                         OP("gelu_backward", op_gelu_backward),
                         OP("rmsnorm", op_rmsnorm),
                         OP("rmsnorm_backward", op_rmsnorm_backward),
                         OP("forward", op_forward),
                         OP("backward_weight", op_backward_weight),
                         OP("pack_both", op_pack_both),
                         OP("pack_blocks", op_pack_blocks),
                         OP("matmul", op_matmul),
                         OP("vocab_loss", op_vocab_loss),
                         OP("linear_cross_entropy", op_linear_cross_entropy),
                         OP("linear_q8", op_linear_q8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q8ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__q8ops() { return PyModule_Create(&module); }
