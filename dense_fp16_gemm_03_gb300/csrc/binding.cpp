// Python binding of the calls whose time on the GPU is about that of their
// arguments' way through Python: products with an epilogue, their gradients and
// the router with scores.  Checks, allocation of outputs and the call of the C
// ABI, nothing else; names, defaults and documentation are in linear.py and
// ragged.py.  (One row of 2048 x 1024 with bias and residual: 11 to 14 us a call through
// ctypes, of which the C call takes 2.4; the GPU takes 6.)
//
// A function returns its tensors, or the status of a call that was refused as
// a number.  Wrong shapes, types, devices and layouts raise ValueError before
// the call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "gemm_linear.h"
#include "gemm_ragged.h"

namespace {

struct Wrong : std::exception {
    std::string text;
    explicit Wrong(std::string t) : text(std::move(t)) {}
    const char *what() const noexcept override { return text.c_str(); }
};

using Shape = c10::SmallVector<int64_t, 4>;

std::string shape_text(c10::IntArrayRef shape)
{
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

const at::Tensor *tensor(PyObject *o, const char *what)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Wrong(std::string(what) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

const at::Tensor &needed(PyObject *o, const char *what)
{
    const at::Tensor *t = tensor(o, what);
    if (t == nullptr) throw Wrong(std::string(what) + " is needed");
    return *t;
}

// The matrix that a call is about: contiguous, on the current device.  Returns the device's number.
int operand(const at::Tensor &t, const char *what)
{
    if (!t.is_cuda() || t.dim() != 2 || !t.is_contiguous())
        throw Wrong(std::string(what) + " must be a contiguous CUDA tensor with 2 dimensions");
    int now = -1;
    cudaGetDevice(&now);
    if (t.get_device() != now) throw Wrong(std::string(what) + " must be on the current device");
    return now;
}

gemm_dtype_t kind_of(at::ScalarType t, bool f32 = false)
{
    if (t == at::kHalf) return GEMM_DTYPE_F16;
    if (t == at::kBFloat16) return GEMM_DTYPE_BF16;
    if (f32 && t == at::kFloat) return GEMM_DTYPE_F32;
    throw Wrong(std::string("operands must be float16 or bfloat16") + (f32 ? " or float32" : "") + ", got " + c10::toString(t));
}

void fits(const at::Tensor &t, const char *what, c10::IntArrayRef shape, at::ScalarType type, int dev)
{
    if (t.sizes() != shape || t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        throw Wrong(std::string(what) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + shape_text(shape) +
                    " on cuda:" + std::to_string(dev));
}

// The address of an argument that may be None.
void *optional(PyObject *o, const char *what, c10::IntArrayRef shape, at::ScalarType type, int dev)
{
    const at::Tensor *t = tensor(o, what);
    if (t == nullptr) return nullptr;
    fits(*t, what, shape, type, dev);
    return t->data_ptr();
}

// An output: the one given, or a new one.
at::Tensor output(PyObject *o, const char *what, c10::IntArrayRef shape, at::ScalarType type, int dev)
{
    if (const at::Tensor *t = tensor(o, what)) {
        fits(*t, what, shape, type, dev);
        return *t;
    }
    return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev))));
}

// A tensor of 32-bit elements in another one's memory, which it keeps: one allocation for several small outputs (0.8 us each,
// views by torch's own functions as much).
at::Tensor cut(const at::Tensor &base, int64_t first, c10::IntArrayRef shape, at::ScalarType type)
{
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), c10::scalarTypeToTypeMeta(type));
    impl->set_sizes_contiguous(shape);
    impl->set_storage_offset(first);
    return at::Tensor(std::move(impl));
}

struct Space {
    void *at = nullptr;
    size_t bytes = 0;
    Space(PyObject *o, int dev)
    {
        const at::Tensor *t = tensor(o, "workspace");
        if (t == nullptr) return;
        if (!t->is_cuda() || t->get_device() != dev || !t->is_contiguous())
            throw Wrong("workspace must be a contiguous CUDA tensor on cuda:" + std::to_string(dev));
        at = t->data_ptr();
        bytes = t->nbytes();
    }
};

gemm_stream_t stream_of(PyObject *o, int dev)
{
    if (o == Py_None) return reinterpret_cast<gemm_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw python_error();
    return reinterpret_cast<gemm_stream_t>(v);
}

int64_t number(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(v);
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

PyObject *wrap(const at::Tensor &t)
{
    return THPVariable_Wrap(t);
}

PyObject *tuple(std::initializer_list<at::Tensor> ts)
{
    PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (r == nullptr) throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = wrap(t);
        if (o == nullptr) {
            Py_DECREF(r);
            throw python_error();
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// One weight matrix, or one per group of rows.
struct Groups {
    bool given = false;
    int64_t count = 1;
    const int32_t *offsets = nullptr;
    Groups(PyObject *o, int dev)
    {
        const at::Tensor *t = tensor(o, "offsets");
        if (t == nullptr) return;
        given = true;
        if (t->dim() != 1 || t->size(0) < 1) throw Wrong("offsets must hold groups + 1 numbers");
        fits(*t, "offsets", t->sizes(), at::kInt, dev);
        count = t->size(0) - 1;
        offsets = static_cast<const int32_t *>(t->data_ptr());
    }
    Shape shape(std::initializer_list<int64_t> own) const  // with an extent for the groups in front
    {
        Shape s;
        if (given) s.push_back(count);
        s.append(own.begin(), own.end());
        return s;
    }
};

struct Weights {
    int64_t n, k;
    Weights(const at::Tensor &w, const Groups &g)
    {
        const int64_t dims = g.given ? 3 : 2;
        if (w.dim() != dims) throw Wrong(g.given ? "w must be [groups, n, k]" : "w must be [n, k] without offsets");
        n = w.size(dims - 2);
        k = w.size(dims - 1);
    }
};

template <class F>
PyObject *guarded(F &&f)
{
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Wrong &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

bool counted(Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "takes %zd arguments, got %zd", want, got);
    return false;
}

// (x, w, bias, residual, act, offsets, keep, y, z, workspace, stream)
PyObject *linear_nt(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    if (!counted(count, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = needed(a[0], "x"), &w = needed(a[1], "w");
        const int dev = operand(x, "x");
        const at::ScalarType type = x.scalar_type();
        const gemm_dtype_t kind = kind_of(type);
        const Groups g(a[5], dev);
        const Weights s(w, g);
        const int64_t rows = x.size(0), k = x.size(1), n = s.n;
        fits(w, "w", g.shape({n, k}), type, dev);
        const void *bias = optional(a[2], "bias", g.shape({n}), type, dev);
        const int64_t shape[2] = {rows, n};
        const void *residual = optional(a[3], "residual", shape, type, dev);
        const bool keep = truth(a[6]);
        if (!keep && a[8] != Py_None) throw Wrong("z is written with keep only");
        const Space ws(a[9], dev);
        const gemm_stream_t stream = stream_of(a[10], dev);
        const gemm_act_t act = static_cast<gemm_act_t>(number(a[4]));
        at::Tensor z;
        if (keep) z = output(a[8], "z", shape, type, dev);
        const at::Tensor y = output(a[7], "y", shape, type, dev);
        const gemm_status_t st = gemm_linear_nt(kind, act, g.count, rows, n, k, g.offsets, x.data_ptr(), w.data_ptr(), bias, residual,
                                                keep ? z.data_ptr() : nullptr, y.data_ptr(), ws.at, ws.bytes, stream);
        if (st != GEMM_OK) return PyLong_FromLong(st);
        return keep ? tuple({y, z}) : wrap(y);
    });
}

// (dy, w, z, act, offsets, bias_grad, dx, dbias, workspace, stream)
PyObject *linear_nn(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    if (!counted(count, 10)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dy = needed(a[0], "dy"), &w = needed(a[1], "w");
        const int dev = operand(dy, "dy");
        const at::ScalarType type = dy.scalar_type();
        const gemm_dtype_t kind = kind_of(type);
        const Groups g(a[4], dev);
        const Weights s(w, g);
        const int64_t rows = dy.size(0), n = dy.size(1), k = s.k;
        fits(w, "w", g.shape({n, k}), type, dev);
        const int64_t shape[2] = {rows, k};
        const void *z = optional(a[2], "z", shape, type, dev);
        const gemm_act_t act = static_cast<gemm_act_t>(number(a[3]));
        if (act != GEMM_ACT_NONE && a[2] == Py_None) throw Wrong("z is needed with act");
        const bool bias = truth(a[5]);
        if (!bias && a[7] != Py_None) throw Wrong("dbias is written with bias_grad only");
        const Space ws(a[8], dev);
        const gemm_stream_t stream = stream_of(a[9], dev);
        const at::Tensor dx = output(a[6], "dx", shape, type, dev);
        at::Tensor db;
        if (bias) db = output(a[7], "dbias", g.shape({k}), at::kFloat, dev);
        const gemm_status_t st = gemm_linear_nn(kind, act, g.count, rows, n, k, g.offsets, dy.data_ptr(), w.data_ptr(), z, dx.data_ptr(),
                                                bias ? static_cast<float *>(db.data_ptr()) : nullptr, ws.at, ws.bytes, stream);
        if (st != GEMM_OK) return PyLong_FromLong(st);
        return bias ? tuple({dx, db}) : wrap(dx);
    });
}

// (dy, z, act, offsets, bias_grad, dz, dbias, workspace, stream)
PyObject *linear_grad(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    if (!counted(count, 9)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &dy = needed(a[0], "dy");
        const int dev = operand(dy, "dy");
        const at::ScalarType type = dy.scalar_type();
        const gemm_dtype_t kind = kind_of(type);
        const Groups g(a[3], dev);
        const int64_t rows = dy.size(0), n = dy.size(1);
        const gemm_act_t act = static_cast<gemm_act_t>(number(a[2]));
        const void *z = optional(a[1], "z", dy.sizes(), type, dev);
        if (act != GEMM_ACT_NONE && a[1] == Py_None) throw Wrong("z is needed with act");
        const bool bias = truth(a[4]);
        if (!bias && a[6] != Py_None) throw Wrong("dbias is written with bias_grad only");
        const Space ws(a[7], dev);
        const gemm_stream_t stream = stream_of(a[8], dev);
        // (without act dz is dy, unless another is given, or offsets, which may leave rows out: they are zero in dz)
        const bool same = act == GEMM_ACT_NONE && !g.given && a[5] == Py_None;
        const at::Tensor dz = same ? dy : output(a[5], "dz", dy.sizes(), type, dev);
        at::Tensor db;
        if (bias) db = output(a[6], "dbias", g.shape({n}), at::kFloat, dev);
        const gemm_status_t st = gemm_linear_grad(kind, act, g.count, rows, n, g.offsets, dy.data_ptr(), z, same ? nullptr : dz.data_ptr(),
                                                  bias ? static_cast<float *>(db.data_ptr()) : nullptr, ws.at, ws.bytes, stream);
        if (st != GEMM_OK) return PyLong_FromLong(st);
        return bias ? tuple({dz, db}) : wrap(dz);
    });
}

// (logits, top, score, bias, groups, top_groups, group_top, renorm, scale, out, workspace, stream)
PyObject *route_scored(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    if (!counted(count, 12)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &logits = needed(a[0], "logits");
        // a Routing to write into has all five: one that were made here would end with the call
        constexpr const char *names[5] = {"ids", "weights", "offsets", "order", "position"};
        const bool given = a[9] != Py_None;
        if (given && (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 5)) throw Wrong("out must be a Routing");
        for (Py_ssize_t i = 0; given && i < 5; ++i) needed(PyTuple_GET_ITEM(a[9], i), names[i]);
        const int dev = operand(logits, "logits");
        const gemm_dtype_t kind = kind_of(logits.scalar_type(), true);
        const int64_t rows = logits.size(0), experts = logits.size(1);
        const int64_t top = number(a[1]), groups = number(a[4]), top_groups = number(a[5]), group_top = number(a[6]);
        if (top < 1 || top > experts) throw Wrong("top must be in [1, experts]");
        if (groups < 1 || experts % groups != 0 || top_groups < 1 || top_groups > groups)
            throw Wrong("groups must divide the experts, and top_groups be in [1, groups]");
        if (top > top_groups * (experts / groups)) throw Wrong("the groups kept hold fewer than `top` experts");
        if (group_top != 1 && group_top != 2) throw Wrong("group_top must be 1 or 2");
        const int64_t each[1] = {experts}, chosen[2] = {rows, top}, ends[1] = {experts + 1}, flat[1] = {rows * top};
        const void *bias = optional(a[3], "bias", each, at::kFloat, dev);
        const Space ws(a[10], dev);
        const gemm_stream_t stream = stream_of(a[11], dev);
        const bool renorm = truth(a[7]);
        const float scale = real(a[8]);
        const gemm_route_score_t score = static_cast<gemm_route_score_t>(number(a[2]));
        at::Tensor ids, weights, offsets, order, position;
        if (given) {
            auto to = [&](Py_ssize_t i, c10::IntArrayRef shape, at::ScalarType type) {
                return output(PyTuple_GET_ITEM(a[9], i), names[i], shape, type, dev);
            };
            ids = to(0, chosen, at::kInt);
            weights = to(1, chosen, at::kFloat);
            offsets = to(2, ends, at::kInt);
            order = to(3, flat, at::kInt);
            position = to(4, chosen, at::kInt);
        } else {
            const int64_t part = (rows * top + 3) / 4 * 4, all[1] = {4 * part + experts + 1};  // (parts of whole 16 bytes)
            const at::Tensor base = output(Py_None, "", all, at::kInt, dev);
            ids = cut(base, 0, chosen, at::kInt);
            weights = cut(base, part, chosen, at::kFloat);
            order = cut(base, 2 * part, flat, at::kInt);
            position = cut(base, 3 * part, chosen, at::kInt);
            offsets = cut(base, 4 * part, ends, at::kInt);
        }
        auto i32 = [](const at::Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); };
        const gemm_status_t st = gemm_route_scored(kind, score, rows, experts, top, groups, top_groups, int32_t(group_top), renorm ? 1 : 0, scale,
                                                   logits.data_ptr(), static_cast<const float *>(bias), i32(ids),
                                                   static_cast<float *>(weights.data_ptr()), i32(offsets), i32(order), i32(position), ws.at,
                                                   ws.bytes, stream);
        if (st != GEMM_OK) return PyLong_FromLong(st);
        if (given) {
            Py_INCREF(a[9]);
            return a[9];
        }
        return tuple({ids, weights, offsets, order, position});
    });
}

// (logits, ids, dweights, score, renorm, scale, dlogits, stream)
PyObject *route_scored_grad(PyObject *, PyObject *const *a, Py_ssize_t count)
{
    if (!counted(count, 8)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &logits = needed(a[0], "logits"), &ids = needed(a[1], "ids"), &dweights = needed(a[2], "dweights");
        const int dev = operand(logits, "logits");
        const gemm_dtype_t kind = kind_of(logits.scalar_type(), true);
        const int64_t rows = logits.size(0), experts = logits.size(1);
        if (ids.dim() != 2) throw Wrong("ids must be [rows, top]");
        const int64_t chosen[2] = {rows, ids.size(1)}, shape[2] = {rows, experts};
        fits(ids, "ids", chosen, at::kInt, dev);
        fits(dweights, "dweights", chosen, at::kFloat, dev);
        const gemm_route_score_t score = static_cast<gemm_route_score_t>(number(a[3]));
        const bool renorm = truth(a[4]);
        const float scale = real(a[5]);
        const gemm_stream_t stream = stream_of(a[7], dev);
        const at::Tensor dl = output(a[6], "dlogits", shape, at::kFloat, dev);
        const gemm_status_t st = gemm_route_scored_grad(kind, score, rows, experts, chosen[1], renorm ? 1 : 0, scale, logits.data_ptr(),
                                                        static_cast<const int32_t *>(ids.data_ptr()),
                                                        static_cast<const float *>(dweights.data_ptr()), static_cast<float *>(dl.data_ptr()),
                                                        stream);
        return st != GEMM_OK ? PyLong_FromLong(st) : wrap(dl);
    });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(linear_nt), METHOD(linear_nn),         METHOD(linear_grad), METHOD(route_scored),
                         METHOD(route_scored_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gemm_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gemm_binding()
{
    return PyModule_Create(&module);
}
