// fast_calls.cpp -- the calls of moe.py whose outputs are given, without Python
// between their arguments and the library.
//
// One decoding token's calls take 3 us on the GPU.  Without the launch, a call through
// moe.py's checks and ctypes takes 4 us on the host, and 0.25 through here.  Each
// function here looks at the same things as its namesake in moe.py and enqueues
// the call where all of them are in order (True, or the exception of a launch that
// failed); in any other case it does nothing (False), and moe.py takes the call, raises
// what there is to raise, or hands it to autograd.  Tensors on another device than the current one, other
// streams than the current one, and subclasses of Tensor are its too.
#include <Python.h>
#include <dlfcn.h>

#include <ATen/core/Tensor.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/bakron_moe.h"

namespace {

#define CALLS(X)                                                                                                          \
    X(bakron_moe_route) X(bakron_moe_route_grad) X(bakron_moe_gather) X(bakron_moe_combine) X(bakron_moe_combine_grad)    \
    X(bakron_q4_experts) X(bakron_q4_experts_grad) X(bakron_ck8_pack) X(bakron_gated_act) X(bakron_gated_act_grad)        \
    X(bakron_ck8_bytes)
struct Library {
#define X(name) decltype(&::name) name = nullptr;
    CALLS(X)
#undef X
} lib;

// Names of attributes and dictionary entries
#define NAMES(X)                                                                                                       \
    X(data) X(count) X(m) X(n) X(_group) X(rows) X(cols) X(dtype) X(ids) X(weights) X(place) X(order) X(offsets) X(dys) \
    X(dweights)
struct Names {
#define X(name) PyObject* name = nullptr;
    NAMES(X)
#undef X
} names;
PyObject *layer_type = nullptr, *checkpoint_type = nullptr, *error_type = nullptr;

// A tensor that is a plain one on the current device, without a gradient or a tangent
// to take; -1 in `device` is set by the first of a call's tensors.
const at::Tensor* plain(PyObject* o, int& device)
{
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) return nullptr;
    if (device < 0) {
        device = t.get_device();
        if (c10::hip::current_device() != device) return nullptr;
    } else if (t.get_device() != device) {
        return nullptr;
    }
    if (t.requires_grad() && c10::GradMode::is_enabled()) return nullptr;
    if (t._fw_grad(0).defined()) return nullptr;   // (a dual tensor of forward mode)
    return &t;
}

bool type_of(at::ScalarType t, bool three, int32_t& type)
{
    if (t == at::kBFloat16) type = BAKRON_Q4_BF16;
    else if (t == at::kHalf) type = BAKRON_Q4_FP16;
    else if (three && t == at::kFloat) type = BAKRON_MOE_F32;
    else return false;
    return true;
}

// rows x cols of one of the value types, its rows contiguous.
struct Matrix {
    void* p;
    int64_t rows, cols, ld;
    int32_t type;
};
bool matrix(PyObject* o, int& device, Matrix& m, bool three = false)
{
    const at::Tensor* t = plain(o, device);
    if (!t || t->dim() != 2 || !type_of(t->scalar_type(), three, m.type)) return false;
    m.rows = t->size(0);
    m.cols = t->size(1);
    if (m.cols > 1 && t->stride(1) != 1 && m.rows) return false;
    m.ld = m.rows <= 1 || m.cols == 0 ? m.cols : t->stride(0);
    if (m.ld < m.cols) return false;
    m.p = t->data_ptr();
    return true;
}
bool matrix_like(PyObject* o, int& device, Matrix& m, int64_t rows, int64_t cols, int32_t type)
{
    return matrix(o, device, m) && m.rows == rows && m.cols == cols && m.type == type;
}

// A contiguous tensor of a type, `dims` of its sizes given.
void* flat(PyObject* o, int& device, at::ScalarType type, int64_t a, int64_t b = -1)
{
    const at::Tensor* t = o ? plain(o, device) : nullptr;
    if (!t || t->scalar_type() != type || !t->is_contiguous() || t->dim() != (b < 0 ? 1 : 2) || t->size(0) != a ||
        (b >= 0 && t->size(1) != b))
        return nullptr;
    static char none;   // an empty tensor has no address, and is none that is missing
    return t->numel() ? t->data_ptr() : &none;
}

// tokens x top_k places
bool places(PyObject* o, int& device, int64_t& T, int64_t& k, const int32_t*& p)
{
    const at::Tensor* t = plain(o, device);
    if (!t || t->dim() != 2 || t->scalar_type() != at::kInt || !t->is_contiguous()) return false;
    T = t->size(0);
    k = t->size(1);
    p = static_cast<const int32_t*>(t->data_ptr());
    return k >= 1 && k <= BAKRON_MOE_MAX_PLACES;
}

bool workspace(PyObject* o, int& device, void*& p, size_t& bytes)
{
    p = nullptr;
    bytes = 0;
    if (o == Py_None) return true;   // (a call that needs one refuses, and moe.py makes it)
    const at::Tensor* t = plain(o, device);
    if (!t || !t->is_contiguous()) return false;
    p = t->data_ptr();
    bytes = t->nbytes();
    return true;
}

bool number(PyObject* o, PyObject* name, int64_t& v)
{
    PyObject* a = PyObject_GetAttr(o, name);
    if (!a) return PyErr_Clear(), false;
    v = PyLong_CheckExact(a) ? PyLong_AsLongLong(a) : -1;
    Py_DECREF(a);
    if (PyErr_Occurred()) PyErr_Clear(), v = -1;
    return v >= 0;
}
bool integer(PyObject* o, int64_t& v)
{
    if (!PyLong_CheckExact(o)) return false;
    v = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) return PyErr_Clear(), false;
    return true;
}

// The bytes of a tensor that an object keeps as its `data`.  (The object keeps the
// tensor, and the caller the object.)
void* data_of(PyObject* o, int& device, size_t* bytes = nullptr)
{
    PyObject* d = PyObject_GetAttr(o, names.data);
    if (!d) return PyErr_Clear(), nullptr;
    const at::Tensor* t = plain(d, device);
    void* p = t && t->is_contiguous() ? t->data_ptr() : nullptr;
    if (t && bytes) *bytes = t->nbytes();
    Py_DECREF(d);
    return p;
}

struct Layers {
    void* p;
    int64_t count, m, n, group;
};
bool layers(PyObject* o, int& device, Layers& w)
{
    return (PyObject*)Py_TYPE(o) == layer_type && number(o, names.count, w.count) && number(o, names.m, w.m) &&
           number(o, names.n, w.n) && number(o, names._group, w.group) && (w.p = data_of(o, device)) != nullptr;
}

// A checkpoint of so many values of that type (null: not one).
void* checkpoint(PyObject* o, int& device, int64_t rows, int64_t cols, int32_t type)
{
    int64_t r, c;
    if ((PyObject*)Py_TYPE(o) != checkpoint_type || !number(o, names.rows, r) || !number(o, names.cols, c) || r != rows || c != cols)
        return nullptr;
    PyObject* d = PyObject_GetAttr(o, names.dtype);
    if (!d) return PyErr_Clear(), nullptr;
    int32_t t;
    const bool same = THPDtype_Check(d) && type_of(reinterpret_cast<THPDtype*>(d)->scalar_type, false, t) && t == type;
    Py_DECREF(d);
    size_t bytes = 0;
    void* p = same ? data_of(o, device, &bytes) : nullptr;
    return p && bytes >= lib.bakron_ck8_bytes(rows, cols) ? p : nullptr;
}

const int32_t* count_of(PyObject* o, int& device, bool& ok)
{
    if (o == Py_None) return nullptr;
    const void* p = flat(o, device, at::kInt, 1);
    ok = ok && p;
    return static_cast<const int32_t*>(p);
}

hipStream_t stream(int device) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }

// A given output, or an object that keeps one as its `data`, counts as changed in place
// (moe.py's _written); null: none.
void written(PyObject* o)
{
    PyObject* t = !o ? nullptr : THPVariable_CheckExact(o) ? Py_NewRef(o) : PyObject_GetAttr(o, names.data);
    if (!t) return PyErr_Clear();
    const at::Tensor& v = THPVariable_Unpack(t);   // (checked before the call)
    if (!v.is_inference()) v.unsafeGetTensorImpl()->bump_version();
    Py_DECREF(t);
}

// What the library says to a call: refusals, which come before anything is enqueued, are
// moe.py's to raise (or to mend, where a workspace is what is missing).  An error of a launch
// is raised here: what the call enqueued before it must not be enqueued again.
template <class... Outputs>
PyObject* answer(const char* call, int rc, Outputs... outputs)
{
    if (rc == BAKRON_SUCCESS) {
        (written(outputs), ...);
        Py_RETURN_TRUE;
    }
    if (rc == BAKRON_ERR_NULL_POINTER || rc == BAKRON_ERR_BAD_SIZE || rc == BAKRON_ERR_WORKSPACE || rc == BAKRON_ERR_BAD_ARG)
        Py_RETURN_FALSE;
    PyObject* e = PyObject_CallFunction(error_type, "is", rc, call);
    if (e) PyErr_SetObject(error_type, e);
    Py_XDECREF(e);
    return nullptr;
}
PyObject* entry(PyObject* d, PyObject* name)
{
    return PyDict_CheckExact(d) ? PyDict_GetItemWithError(d, name) : nullptr;
}

#define ARGS(k)                                                        \
    if (n != (k) || !lib.bakron_moe_route) Py_RETURN_FALSE;             \
    int dev = -1;
#define NEED(cond) \
    if (!(cond)) Py_RETURN_FALSE
#define CALL(call, args, ...) answer(#call, lib.call args, __VA_ARGS__)

// logits, top_k, out, ws
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(4)
    Matrix l;
    int64_t k;
    NEED(matrix(a[0], dev, l, true) && integer(a[1], k) && k >= 1 && k <= BAKRON_MOE_MAX_TOP_K);
    const int64_t T = l.rows, E = l.cols;
    int32_t* ids = (int32_t*)flat(entry(a[2], names.ids), dev, at::kInt, T, k);
    float* weights = (float*)flat(entry(a[2], names.weights), dev, at::kFloat, T, k);
    int32_t* place = (int32_t*)flat(entry(a[2], names.place), dev, at::kInt, T, k);
    int32_t* order = (int32_t*)flat(entry(a[2], names.order), dev, at::kInt, T * k);
    int32_t* offsets = (int32_t*)flat(entry(a[2], names.offsets), dev, at::kInt, E + 1);
    void* ws;
    size_t bytes;
    NEED(T && ids && weights && place && order && offsets && workspace(a[3], dev, ws, bytes));
    return CALL(bakron_moe_route, (l.p, l.ld, T, l.type, E, (int32_t)k, ids, weights, place, order, offsets, ws, bytes,
                stream(dev)),
                entry(a[2], names.ids), entry(a[2], names.weights), entry(a[2], names.place), entry(a[2], names.order),
                entry(a[2], names.offsets));
}

// dweights, weights, ids, experts, out
PyObject* route_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(5)
    Matrix d;
    int64_t E;
    NEED(integer(a[3], E) && matrix(a[4], dev, d, true) && d.cols == E && d.rows);
    const at::Tensor* i = plain(a[2], dev);
    NEED(i && i->dim() == 2);
    const int64_t k = i->size(1);
    const float *g = (const float*)flat(a[0], dev, at::kFloat, d.rows, k), *w = (const float*)flat(a[1], dev, at::kFloat, d.rows, k);
    const int32_t* ids = (const int32_t*)flat(a[2], dev, at::kInt, d.rows, k);
    NEED(k >= 1 && k <= BAKRON_MOE_MAX_TOP_K && g && w && ids);
    return CALL(bakron_moe_route_grad, (g, w, ids, d.rows, E, (int32_t)k, d.p, d.ld, d.type, stream(dev)), a[4]);
}

// x, place, out
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(3)
    Matrix x, xs;
    int64_t T, k;
    const int32_t* place;
    NEED(matrix(a[0], dev, x) && places(a[1], dev, T, k, place) && x.rows == T && matrix(a[2], dev, xs) && xs.cols == x.cols &&
         xs.type == x.type);
    return CALL(bakron_moe_gather, (x.p, x.ld, T, x.type, x.cols, (int32_t)k, place, xs.p, xs.ld, xs.rows, stream(dev)), a[2]);
}

// ys, place, weights, out
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(4)
    Matrix ys, y;
    int64_t T, k;
    const int32_t* place;
    const float* w = nullptr;
    NEED(matrix(a[0], dev, ys) && places(a[1], dev, T, k, place) && matrix_like(a[3], dev, y, T, ys.cols, ys.type));
    NEED(a[2] == Py_None || (w = (const float*)flat(a[2], dev, at::kFloat, T, k)));
    return CALL(bakron_moe_combine, (ys.p, ys.ld, ys.rows, ys.type, ys.cols, (int32_t)k, place, w, T, y.p, y.ld, stream(dev)),
                a[3]);
}

// dy, ys, place, weights, out
PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(5)
    Matrix dy, ys, dys;
    int64_t T, k;
    const int32_t* place;
    NEED(matrix(a[1], dev, ys) && places(a[2], dev, T, k, place) && matrix_like(a[0], dev, dy, T, ys.cols, ys.type));
    const float* w = (const float*)flat(a[3], dev, at::kFloat, T, k);
    float* dw = (float*)flat(entry(a[4], names.dweights), dev, at::kFloat, T, k);
    PyObject* o = entry(a[4], names.dys);
    NEED(w && dw && o && matrix_like(o, dev, dys, ys.rows, ys.cols, ys.type));
    return CALL(bakron_moe_combine_grad, (dy.p, dy.ld, ys.p, ys.ld, ys.rows, ys.type, ys.cols, (int32_t)k, place, w, T, dys.p,
                dys.ld, dw, stream(dev)), o, entry(a[4], names.dweights));
}

// x, w, offsets, out, ws
PyObject* experts_of(bool grad, PyObject* const* a, Py_ssize_t n)
{
    ARGS(5)
    Matrix x, y;
    Layers w;
    void* ws;
    size_t bytes;
    NEED(matrix(a[0], dev, x) && layers(a[1], dev, w) && x.cols == (grad ? w.m : w.n) &&
         matrix_like(a[3], dev, y, x.rows, grad ? w.n : w.m, x.type) && workspace(a[4], dev, ws, bytes));
    const int32_t* offsets = (const int32_t*)flat(a[2], dev, at::kInt, w.count + 1);
    NEED(offsets);
    const auto run = grad ? lib.bakron_q4_experts_grad : lib.bakron_q4_experts;
    const int rc = run(x.p, x.ld, x.rows, x.type, w.p, w.count, w.m, w.n, w.group, offsets, y.p, y.ld, ws, bytes, stream(dev));
    return answer(grad ? "bakron_q4_experts_grad" : "bakron_q4_experts", rc, a[3]);
}
PyObject* experts(PyObject*, PyObject* const* a, Py_ssize_t n) { return experts_of(false, a, n); }
PyObject* experts_grad(PyObject*, PyObject* const* a, Py_ssize_t n) { return experts_of(true, a, n); }

// x, out
PyObject* pack(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(2)
    Matrix x;
    void* ck;
    NEED(matrix(a[0], dev, x) && (ck = checkpoint(a[1], dev, x.rows, x.cols, x.type)));
    return CALL(bakron_ck8_pack, (x.p, x.ld, x.rows, x.type, x.cols, ck, stream(dev)), a[1]);
}

// a, b, kind, checkpoints (None or a pair), count, out
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(6)
    Matrix x, y, h;
    int64_t kind;
    bool ok = true;
    NEED(matrix(a[0], dev, x) && matrix_like(a[1], dev, y, x.rows, x.cols, x.type) && integer(a[2], kind) &&
         matrix_like(a[5], dev, h, x.rows, x.cols, x.type));
    const int32_t* count = count_of(a[4], dev, ok);
    void *ca = nullptr, *cb = nullptr;
    if (a[3] != Py_None)
        ok = ok && PyTuple_CheckExact(a[3]) && PyTuple_GET_SIZE(a[3]) == 2 &&
             (ca = checkpoint(PyTuple_GET_ITEM(a[3], 0), dev, x.rows, x.cols, x.type)) &&
             (cb = checkpoint(PyTuple_GET_ITEM(a[3], 1), dev, x.rows, x.cols, x.type));
    NEED(ok);
    return CALL(bakron_gated_act, (x.p, x.ld, y.p, y.ld, x.rows, x.type, x.cols, (int32_t)kind, count, h.p, h.ld, ca, cb,
                stream(dev)), a[5], ca ? PyTuple_GET_ITEM(a[3], 0) : nullptr, cb ? PyTuple_GET_ITEM(a[3], 1) : nullptr);
}

// dh, ck_a, ck_b, kind, count, da, db
PyObject* gated_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    ARGS(7)
    Matrix d, da, db;
    int64_t kind;
    bool ok = true;
    NEED(matrix(a[0], dev, d) && integer(a[3], kind) && matrix_like(a[5], dev, da, d.rows, d.cols, d.type) &&
         matrix_like(a[6], dev, db, d.rows, d.cols, d.type));
    const int32_t* count = count_of(a[4], dev, ok);
    void *ca = checkpoint(a[1], dev, d.rows, d.cols, d.type), *cb = checkpoint(a[2], dev, d.rows, d.cols, d.type);
    NEED(ok && ca && cb);
    return CALL(bakron_gated_act_grad, (d.p, d.ld, ca, cb, d.rows, d.type, d.cols, (int32_t)kind, count, da.p, da.ld, db.p,
                db.ld, stream(dev)), a[5], a[6]);
}

// path of the library, Q4Weight, Checkpoint8, BakronError
PyObject* load(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    const char* path = n == 4 ? PyUnicode_AsUTF8(a[0]) : nullptr;
    void* h = path ? dlopen(path, RTLD_NOW | RTLD_LOCAL) : nullptr;
    if (PyErr_Occurred()) return nullptr;
    if (!h) return PyErr_SetString(PyExc_RuntimeError, "the library cannot be loaded"), nullptr;
    Library l;
#define X(name)                                                      \
    l.name = reinterpret_cast<decltype(l.name)>(dlsym(h, #name));    \
    if (!l.name) return PyErr_SetString(PyExc_RuntimeError, #name " is missing"), nullptr;
    CALLS(X)
#undef X
#define X(name)                                                      \
    if (!names.name) names.name = PyUnicode_InternFromString(#name); \
    if (!names.name) return nullptr;
    NAMES(X)
#undef X
    for (int i = 1; i < 4; ++i) Py_INCREF(a[i]);
    Py_XSETREF(layer_type, a[1]);
    Py_XSETREF(checkpoint_type, a[2]);
    Py_XSETREF(error_type, a[3]);
    lib = l;
    Py_RETURN_NONE;
}

// No C++ exception may leave a call that Python makes.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* safe(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    try {
        return F(self, a, n);
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(safe<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(load), METHOD(route), METHOD(route_grad), METHOD(gather), METHOD(combine), METHOD(combine_grad),
                         METHOD(experts), METHOD(experts_grad), METHOD(pack), METHOD(gated), METHOD(gated_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
