// Python entry points of the 8-bit activation calls on torch tensors: argument
// checks, outputs, the current stream, and the call into libsnk, in one native
// step.  (Through ctypes and torch's Python API a call took 16 to 24 us of host
// time, most of a decoding step; here 4 to 9.)  The module is built against torch's
// headers beside libsnk.so, which load() opens; q8.py and binding.py are its
// only users.  Wrong tensors raise ValueError, a status from libsnk raises
// binding.SnkError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
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
} g;

struct Wrong : std::runtime_error {   // becomes ValueError
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
    if (!ok) {
        PyErr_SetString(PyExc_RuntimeError, "libsnk.so lacks an 8-bit activation call");
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q8ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__q8ops() { return PyModule_Create(&module); }
