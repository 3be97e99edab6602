// _native: the bindings' common case without Python's share of it.
//
// A call of a few microseconds on the GPU (a decoding step's append and
// attention) cost 13 us through ctypes, most of it checks and marshalling.
// The functions here take a binding's arguments by position, check them, make
// the outputs that the caller did not give, and call the C ABI on the current
// stream.  They serve the plain case only and answer NotImplemented to all
// else: another device than the current one, wrong types or shapes, an error
// of the C call.  The Python binding then goes its own way, which has the
// messages.  No argument is kept.  Python's lock is given up while outputs are
// made and kernels launched: both may wait, for memory or for room in the launch
// queue, and what they wait for may be a function on the stream that needs it.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <cstring>

#include "fvattn_cache.h"
#include "fvattn_train.h"

namespace {

using at::Tensor;

PyObject* not_here() { Py_RETURN_NOTIMPLEMENTED; }

// Python's lock, given up for a scope (which an exception may leave).
struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// A tensor argument, or null for None; `ok` falls for anything else.
const Tensor* arg(PyObject* o, bool& ok) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
        ok = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

// On CUDA device `dev`, dense, of this type.
bool dense(const Tensor* t, int dev, at::ScalarType type, at::IntArrayRef shape) {
    return t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}

// A [rows, heads, D] view whose rows may lie apart: their stride, or -1.
long long row_stride(const Tensor* t, int dev, long long rows, long long heads, long long D) {
    if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != at::kBFloat16 || t->dim() != 3) return -1;
    const auto n = t->sizes(), st = t->strides();
    if (n[0] != rows || (heads > 0 && n[1] != heads) || n[1] < 1 || n[2] != D) return -1;
    const long long row = n[1] * D, sr = n[0] > 1 ? st[0] : row;
    if (st[2] != 1 || (n[1] > 1 && st[1] != D) || sr < row || sr % 8) return -1;
    return sr;
}

at::TensorOptions on(int dev, at::ScalarType type) {
    return at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev));
}

fvattn_stream_t stream_of(int dev) {
    return reinterpret_cast<fvattn_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

bool current(int dev) { return c10::cuda::current_device() == dev; }

// scale: None is 1 / sqrt(D)
bool scale_of(PyObject* o, long long D, float& scale) {
    if (o == Py_None) {
        scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
        return true;
    }
    if (!PyFloat_Check(o)) return false;
    const double x = PyFloat_AS_DOUBLE(o);
    scale = static_cast<float>(x);
    return x > 0.0 && std::isfinite(x);
}

bool geom_of(PyObject* o, fvattn_geom& g) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
        PyErr_Clear();
        return false;
    }
    const bool ok = b.len == static_cast<Py_ssize_t>(sizeof(g));
    if (ok) std::memcpy(&g, b.buf, sizeof(g));
    PyBuffer_Release(&b);
    return ok;
}

template <class T>
T* ptr(const Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

bool cache_of(const Tensor* k, const Tensor* v, fvattn_cache& c, int& dev) {
    if (!k || !v || !k->is_cuda() || k->dim() != 4) return false;
    dev = k->get_device();
    if (!dense(k, dev, at::kBFloat16, k->sizes()) || !dense(v, dev, at::kBFloat16, k->sizes()) || !current(dev)) return false;
    const auto n = k->sizes();
    c.pages = static_cast<int>(n[0]);
    c.Hkv = static_cast<int>(n[1]);
    c.page = static_cast<int>(n[2]);
    c.D = static_cast<int>(n[3]);
    c.k = k->data_ptr();
    c.v = v->data_ptr();
    return true;
}

// append(k_pages, v_pages, k, v, table, lens, cu, q, q_out, pos, rot, axes, halves) -> q_out
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 13) return not_here();
    bool ok = true;
    const Tensor *kp = arg(a[0], ok), *vp = arg(a[1], ok), *k = arg(a[2], ok), *v = arg(a[3], ok), *table = arg(a[4], ok),
                 *lens = arg(a[5], ok), *cu = arg(a[6], ok), *q = arg(a[7], ok), *qo = arg(a[8], ok), *pos = arg(a[9], ok),
                 *rot = arg(a[10], ok);
    fvattn_cache c;
    int dev = 0;
    if (!ok || !cache_of(kp, vp, c, dev) || !k || k->dim() != 3 || k->size(0) < 1 || !table || table->dim() != 2 ||
        table->numel() < 1)
        return not_here();
    const long long rows = k->size(0), B = table->size(0);
    const long long ks = row_stride(k, dev, rows, c.Hkv, c.D), vs = row_stride(v, dev, rows, c.Hkv, c.D);
    if (ks < 0 || vs < 0 || !dense(table, dev, at::kInt, table->sizes()) || !dense(lens, dev, at::kInt, {B}) ||
        (cu ? !dense(cu, dev, at::kInt, {B + 1}) : rows < B))
        return not_here();
    long long qs = 0, qos = 0, hq = 0;
    if (q) {
        if ((qs = row_stride(q, dev, rows, 0, c.D)) < 0) return not_here();
        hq = q->size(1);
        if (qo && ((qos = row_stride(qo, dev, rows, hq, c.D)) < 0 || (qo->data_ptr() == q->data_ptr() && qos != qs)))
            return not_here();
    } else if (qo) {
        return not_here();
    }
    fvattn_rotation r;
    if (rot) {
        if (rot->dim() != 2 || rot->size(0) < 1 || rot->size(0) > 0x7fffffff ||
            !dense(rot, dev, at::kFloat, {rot->size(0), static_cast<long long>(c.D)}))
            return not_here();
        r = {};
        r.axes = 1;
        r.pairs[0] = c.D / 2;
        if (a[11] != Py_None) {
            if (!PyTuple_CheckExact(a[11]) || PyTuple_GET_SIZE(a[11]) < 1 || PyTuple_GET_SIZE(a[11]) > 3) return not_here();
            r.axes = static_cast<int>(PyTuple_GET_SIZE(a[11]));
            for (int i = 0; i < r.axes; ++i) {
                PyObject* x = PyTuple_GET_ITEM(a[11], i);
                if (!PyLong_CheckExact(x)) return not_here();
                const long p = PyLong_AsLong(x);
                if (p < 0 || p > c.D / 2) {
                    PyErr_Clear();
                    return not_here();
                }
                r.pairs[i] = static_cast<int>(p);
            }
        }
        if (!dense(pos, dev, at::kInt, {rows, r.axes}) || (a[12] != Py_True && a[12] != Py_False)) return not_here();
        r.table = ptr<float>(rot);
        r.rows = static_cast<int>(rot->size(0));
        r.pos = ptr<int32_t>(pos);
        r.halves = a[12] == Py_True;
    } else if (pos || a[11] != Py_None) {
        return not_here();
    }
    Tensor made;
    int rc;
    {
        Unlocked unlocked;
        if (q && !qo) {
            made = at::empty({rows, hq, c.D}, on(dev, at::kBFloat16));
            qo = &made;
            qos = hq * c.D;
        }
        const auto call = made.defined() ? fvattn_cache_append_fresh : fvattn_cache_append;
        rc = call(&c, static_cast<int>(B), rows, ptr<int32_t>(cu), ptr<int32_t>(lens), ptr<int32_t>(table),
                  static_cast<int>(table->size(1)), k->data_ptr(), ks, v->data_ptr(), vs, ptr<void>(q), qs,
                  static_cast<int>(hq), ptr<void>(qo), qos, rot ? &r : nullptr, stream_of(dev));
    }
    if (rc != FVATTN_OK) return not_here();
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    PyObject* out = q ? a[8] : Py_None;
    Py_INCREF(out);
    return out;
    END_HANDLE_TH_ERRORS
}

PyObject* pair(PyObject* x, PyObject* y) {
    PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// The caller's tensor, or the one made in its place.
PyObject* given(PyObject* o, Tensor&& made) {
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    Py_INCREF(o);
    return o;
}

// attend(k_pages, v_pages, q, table, lens, scale, longest, out, lse, workspace) -> (o, lse)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) return not_here();
    bool ok = true;
    const Tensor *kp = arg(a[0], ok), *vp = arg(a[1], ok), *q = arg(a[2], ok), *table = arg(a[3], ok), *lens = arg(a[4], ok),
                 *out = arg(a[7], ok), *lse = arg(a[8], ok), *ws = arg(a[9], ok);
    fvattn_cache c;
    int dev = 0;
    float scale;
    if (!ok || !cache_of(kp, vp, c, dev) || !table || table->dim() != 2 || table->numel() < 1 ||
        !dense(table, dev, at::kInt, table->sizes()) || !scale_of(a[5], c.D, scale))
        return not_here();
    const long long B = table->size(0), width = table->size(1);
    const long long qs = row_stride(q, dev, B, 0, c.D);
    if (qs < 0 || !dense(lens, dev, at::kInt, {B})) return not_here();
    const long long hq = q->size(1);
    long long longest = width * c.page;
    if (a[6] != Py_None) {
        if (!PyLong_CheckExact(a[6])) return not_here();
        longest = PyLong_AsLongLong(a[6]);
        if (longest < 0) {
            PyErr_Clear();
            return not_here();
        }
    }
    if ((out && !dense(out, dev, at::kBFloat16, {B, hq, c.D})) || (lse && !dense(lse, dev, at::kFloat, {B, hq})) ||
        (ws && !dense(ws, dev, at::kByte, {ws->numel()})) || hq > 0x7fffffff || B > 65535)
        return not_here();
    Tensor made_out, made_lse, made_ws;
    int rc;
    {
        Unlocked unlocked;
        if (!ws) {
            const size_t need = fvattn_cache_attn_workspace_size(static_cast<int>(B), static_cast<int>(hq), c.Hkv, c.D, longest);
            if (need > 0) made_ws = at::empty({static_cast<long long>(need)}, on(dev, at::kByte));
        }
        if (!out) made_out = at::empty({B, hq, c.D}, on(dev, at::kBFloat16));
        if (!lse) made_lse = at::empty({B, hq}, on(dev, at::kFloat));
        const Tensor* w = ws ? ws : (made_ws.defined() ? &made_ws : nullptr);
        rc = fvattn_cache_attn(&c, static_cast<int>(B), static_cast<int>(hq), q->data_ptr(), qs, ptr<int32_t>(table),
                               static_cast<int>(width), ptr<int32_t>(lens), longest, scale,
                               out ? out->data_ptr() : made_out.data_ptr(), ptr<float>(lse ? lse : &made_lse),
                               ptr<void>(w), w ? static_cast<size_t>(w->numel()) : 0, stream_of(dev));
    }
    if (rc != FVATTN_OK) return not_here();
    return pair(given(a[7], std::move(made_out)), given(a[8], std::move(made_lse)));
    END_HANDLE_TH_ERRORS
}

// The tiled tensors and lists that both training calls take.
bool training_args(const fvattn_geom& g, int dev, std::initializer_list<const Tensor*> tiles, const Tensor* idx,
                   const Tensor* cnt) {
    for (const Tensor* t : tiles)
        if (!dense(t, dev, at::kBFloat16, {g.B, g.H, g.Npad, g.D})) return false;
    return dense(idx, dev, at::kInt, {g.B, g.H, g.nb, g.nb}) && dense(cnt, dev, at::kInt, {g.B, g.H, g.nb});
}

// sparse_attn_lse(g, qt, kt, vt, kv_idx, kv_cnt, scale, out, lse, workspace) -> (out, lse)
PyObject* sparse_attn_lse(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    fvattn_geom g;
    if (n != 10 || !geom_of(a[0], g)) return not_here();
    bool ok = true;
    const Tensor *q = arg(a[1], ok), *k = arg(a[2], ok), *v = arg(a[3], ok), *idx = arg(a[4], ok), *cnt = arg(a[5], ok),
                 *out = arg(a[7], ok), *lse = arg(a[8], ok), *ws = arg(a[9], ok);
    float scale;
    if (!ok || !q || !q->is_cuda()) return not_here();
    const int dev = q->get_device();
    if (!current(dev) || !training_args(g, dev, {q, k, v}, idx, cnt) || !scale_of(a[6], g.D, scale)) return not_here();
    if ((out && (!training_args(g, dev, {out}, idx, cnt) || out->data_ptr() == q->data_ptr() ||
                 out->data_ptr() == k->data_ptr() || out->data_ptr() == v->data_ptr())) ||
        (lse && !dense(lse, dev, at::kFloat, {g.B, g.H, g.Npad})) || (ws && !dense(ws, dev, at::kByte, {ws->numel()})))
        return not_here();
    Tensor made_out, made_lse, made_ws;
    int rc;
    {
        Unlocked unlocked;
        if (!out) made_out = at::empty({g.B, g.H, g.Npad, g.D}, on(dev, at::kBFloat16));
        if (!lse) made_lse = at::empty({g.B, g.H, g.Npad}, on(dev, at::kFloat));
        if (!ws) made_ws = at::empty({static_cast<long long>(fvattn_attn_workspace_size(&g))}, on(dev, at::kByte));
        const Tensor* w = ws ? ws : &made_ws;
        rc = fvattn_sparse_attn_lse(&g, q->data_ptr(), k->data_ptr(), v->data_ptr(), ptr<int32_t>(idx), ptr<int32_t>(cnt),
                                    scale, out ? out->data_ptr() : made_out.data_ptr(),
                                    ptr<float>(lse ? lse : &made_lse), nullptr, w->data_ptr(),
                                    static_cast<size_t>(w->numel()), stream_of(dev));
    }
    if (rc != FVATTN_OK) return not_here();
    return pair(given(a[7], std::move(made_out)), given(a[8], std::move(made_lse)));
    END_HANDLE_TH_ERRORS
}

// sparse_attn_bwd(g, qt, kt, vt, ot, dot, lse, kv_idx, kv_cnt, scale, workspace) -> (dq, dk, dv), all made here
PyObject* sparse_attn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    fvattn_geom g;
    if (n != 11 || !geom_of(a[0], g)) return not_here();
    bool ok = true;
    const Tensor *q = arg(a[1], ok), *k = arg(a[2], ok), *v = arg(a[3], ok), *o = arg(a[4], ok), *dout = arg(a[5], ok),
                 *lse = arg(a[6], ok), *idx = arg(a[7], ok), *cnt = arg(a[8], ok), *ws = arg(a[10], ok);
    float scale;
    if (!ok || !q || !q->is_cuda()) return not_here();
    const int dev = q->get_device();
    if (!current(dev) || !training_args(g, dev, {q, k, v, o, dout}, idx, cnt) ||
        !dense(lse, dev, at::kFloat, {g.B, g.H, g.Npad}) || !scale_of(a[9], g.D, scale) ||
        (ws && !dense(ws, dev, at::kByte, {ws->numel()})))
        return not_here();
    Tensor d[3], made_ws;
    int rc;
    {
        Unlocked unlocked;
        for (Tensor& t : d) t = at::empty({g.B, g.H, g.Npad, g.D}, on(dev, at::kBFloat16));
        if (!ws) made_ws = at::empty({static_cast<long long>(fvattn_sparse_attn_bwd_workspace_size(&g))}, on(dev, at::kByte));
        const Tensor* w = ws ? ws : &made_ws;
        rc = fvattn_sparse_attn_bwd(&g, q->data_ptr(), k->data_ptr(), v->data_ptr(), o->data_ptr(), dout->data_ptr(),
                                    ptr<float>(lse), ptr<int32_t>(idx), ptr<int32_t>(cnt), scale, d[0].data_ptr(),
                                    d[1].data_ptr(), d[2].data_ptr(), w->data_ptr(), static_cast<size_t>(w->numel()),
                                    stream_of(dev));
    }
    if (rc != FVATTN_OK) return not_here();
    PyObject *x = THPVariable_Wrap(std::move(d[0])), *y = THPVariable_Wrap(std::move(d[1])), *z = THPVariable_Wrap(std::move(d[2]));
    PyObject* t = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return t;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"sparse_attn_lse", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sparse_attn_lse)), METH_FASTCALL, nullptr},
    {"sparse_attn_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sparse_attn_bwd)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "target", FV_NATIVE_TARGET) != 0) Py_CLEAR(m);
    return m;
}
