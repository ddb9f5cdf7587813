// The Python binding's way past its own interpreter for the short calls: it reads
// shapes, strides, types and addresses off the tensors and calls the C entry, as
// sd_verify.py does for the same arguments, in 2 us instead of 10 to 17.  It takes
// only calls of which every check holds; for any other it returns None without
// calling anything, and sd_verify.py goes through the arguments itself and says
// what is wrong with them.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <dlfcn.h>

#include "../../include/sd_verify.h"

namespace {

decltype(&sd_norm_rotary) norm_rotary_fn;
decltype(&sd_norm_rotary_append_paged) append_fn;
decltype(&sd_paged_attention_e4m3) attention_fn;
decltype(&sd_paged_tree_attention) tree_fn;
decltype(&sd_compact_tree_paged) compact_fn;

using at::ScalarType;

// the arguments of one call: anything that is not as it should be clears `ok`
struct Args {
    PyObject *const *a;
    Py_ssize_t n;
    bool ok = true;
    int device = -1;

    const at::Tensor *tensor(Py_ssize_t i, bool optional = false) {
        if (!ok) return nullptr;
        if (i >= n || (optional && a[i] == Py_None)) {
            ok = ok && i < n;
            return nullptr;
        }
        if (!THPVariable_Check(a[i])) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        if (!t.defined() || !t.is_cuda() || (device >= 0 && t.get_device() != device)) {
            ok = false;
            return nullptr;
        }
        device = t.get_device();
        return &t;
    }
    double number(Py_ssize_t i) {
        if (!ok || i >= n || !(PyFloat_CheckExact(a[i]) || PyLong_CheckExact(a[i]))) {
            ok = false;
            return 0;
        }
        const double v = PyFloat_CheckExact(a[i]) ? PyFloat_AS_DOUBLE(a[i]) : PyLong_AsDouble(a[i]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    int whole(Py_ssize_t i) {
        if (!ok || i >= n || !(PyLong_CheckExact(a[i]) || PyBool_Check(a[i]))) {
            ok = false;
            return 0;
        }
        int over = 0;
        const long v = PyLong_AsLongAndOverflow(a[i], &over);
        if (over || v < INT32_MIN || v > INT32_MAX) ok = false;
        return (int)v;
    }
    void need(bool c) { ok = ok && c; }
    void *stream() { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
    void current() { need(device >= 0 && device == c10::cuda::current_device()); }
};

int dtype_of(const at::Tensor &t) {
    return t.scalar_type() == ScalarType::BFloat16 ? SD_BF16 : t.scalar_type() == ScalarType::Float ? SD_FP32 : -1;
}
bool is_i32(const at::Tensor &t, int64_t n) {
    return t.scalar_type() == ScalarType::Int && t.dim() == 1 && t.size(0) == n && t.is_contiguous();
}
void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

// [n, h, D] rows of `like`'s type with a contiguous last axis
bool rows(const at::Tensor &t, int64_t n, int64_t h, int64_t d, ScalarType type) {
    return t.dim() == 3 && t.size(0) == n && t.size(1) == h && t.size(2) == d && t.stride(2) == 1 && t.scalar_type() == type;
}

// k_pages, v_pages, page_table, scales; `type` is that of a cache without scales
struct Cache {
    sd_paged_cache c;
    sd_page_scales s;
    bool scaled;
    int B, Hkv, D;

    Cache(Args &x, const at::Tensor *k, const at::Tensor *v, const at::Tensor *table, const at::Tensor *ks, const at::Tensor *vs,
          ScalarType type) {
        if (!x.ok) return;
        scaled = ks != nullptr;
        x.need((ks != nullptr) == (vs != nullptr) && k->dim() == 4 && k->sizes() == v->sizes() && k->strides() == v->strides() &&
               k->scalar_type() == v->scalar_type() && k->scalar_type() == (scaled ? ScalarType::Float8_e4m3fn : type) &&
               table->dim() == 2 && table->scalar_type() == ScalarType::Int);
        if (!x.ok) return;
        x.need(k->stride(3) == 1 && table->stride(1) == 1 && k->size(0) <= INT32_MAX && k->size(1) <= INT32_MAX &&
               table->size(1) <= INT32_MAX && table->size(0) <= INT32_MAX);
        if (scaled)
            for (const at::Tensor *t : {ks, vs})
                x.need(t->scalar_type() == ScalarType::Float && t->dim() == 3 && t->size(0) == k->size(0) && t->size(1) == k->size(2) &&
                       t->size(2) == k->size(1) && t->is_contiguous());
        if (!x.ok) return;
        B = (int)table->size(0);
        Hkv = (int)k->size(2);
        D = (int)k->size(3);
        c = {k->data_ptr(), v->data_ptr(), {k->stride(0), k->stride(1), k->stride(2)}, static_cast<const int32_t *>(table->data_ptr()),
             table->stride(0), (int)table->size(1), (int)k->size(0), (int)k->size(1)};
        if (scaled) s = {static_cast<float *>(ks->data_ptr()), static_cast<float *>(vs->data_ptr())};
    }
};

// turns, positions, axes (None or a tuple), order, layout: what the two rotary calls share
struct Rope {
    const uint64_t *turns = nullptr;
    const int32_t *positions = nullptr;
    int64_t stride = 0;
    sd_rope_axes axes;
    const sd_rope_axes *use = nullptr;
    int rot = 0;
    sd_rope_layout layout = SD_ROPE_HALF;

    Rope(Args &x, const at::Tensor *t, const at::Tensor *pos, int64_t N, Py_ssize_t at) {
        if (!x.ok) return;
        x.need(t->scalar_type() == ScalarType::Long && t->dim() == 1 && t->is_contiguous() && t->size(0) <= 4096);
        PyObject *ax = x.a[at], *order = x.a[at + 1], *lay = x.a[at + 2];
        x.need(PyUnicode_CheckExact(order) && PyUnicode_CheckExact(lay));
        if (!x.ok) return;
        int n = 1;
        if (ax != Py_None) {
            x.need(PyTuple_CheckExact(ax) || PyList_CheckExact(ax));
            if (!x.ok) return;
            const bool list = PyList_CheckExact(ax);
            n = (int)(list ? PyList_GET_SIZE(ax) : PyTuple_GET_SIZE(ax));
            x.need(n >= 1 && n <= 4);
            axes = {};
            for (int i = 0; x.ok && i < n; ++i) {
                PyObject *v = list ? PyList_GET_ITEM(ax, i) : PyTuple_GET_ITEM(ax, i);
                x.need(PyLong_CheckExact(v));
                if (!x.ok) return;
                int over = 0;
                const long p = PyLong_AsLongAndOverflow(v, &over);
                x.need(!over && p >= 0 && p <= 4096);
                axes.pairs[i] = (int)p;
            }
            axes.n = n;
            use = &axes;
            int64_t sum = 0;
            for (int i = 0; i < n; ++i) sum += axes.pairs[i];
            x.need(sum == t->size(0));
            if (PyUnicode_CompareWithASCIIString(order, "blocks") == 0) axes.order = SD_AXES_BLOCKS;
            else if (PyUnicode_CompareWithASCIIString(order, "stripes") == 0) axes.order = SD_AXES_STRIPES;
            else x.ok = false;
        }
        if (PyUnicode_CompareWithASCIIString(lay, "interleaved") == 0) layout = SD_ROPE_INTERLEAVED;
        else x.need(PyUnicode_CompareWithASCIIString(lay, "half") == 0);
        if (pos) {
            const int64_t d = pos->dim();
            x.need(pos->scalar_type() == ScalarType::Int && ((d == 2 && pos->size(0) == n && pos->size(1) == N) ||
                                                             (d == 1 && n == 1 && pos->size(0) == N)));
            x.need(x.ok && (N <= 1 || pos->stride(d - 1) == 1));
            if (!x.ok) return;
            positions = static_cast<const int32_t *>(pos->data_ptr());
            stride = pos->stride(0);
        }
        rot = (int)(2 * t->size(0));
        turns = static_cast<const uint64_t *>(t->data_ptr());
    }
};

bool weight(const at::Tensor *w, int64_t D, ScalarType type) {
    return !w || (w->dim() == 1 && w->size(0) == D && w->scalar_type() == type && (D <= 1 || w->stride(0) == 1));
}

// Calls a C entry (none throws) without the interpreter's lock: a launch waits where the queue is full, and what it
// waits for may need the lock.
template <typename F, typename... A> PyObject *answer(F entry, A... args) {
    PyThreadState *state = PyEval_SaveThread();
    const sd_status s = entry(args...);
    PyEval_RestoreThread(state);
    return PyLong_FromLong((long)s);
}

// q q_out k k_out positions turns q_weight k_weight eps axes order layout magnitude
PyObject *norm_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Args x{a, n};
    if (n != 13) Py_RETURN_NONE;
    const at::Tensor *q = x.tensor(0), *qo = x.tensor(1), *k = x.tensor(2, true), *ko = x.tensor(3, true), *pos = x.tensor(4),
                     *turns = x.tensor(5), *wq = x.tensor(6, true), *wk = x.tensor(7, true);
    const double eps = x.number(8), m = x.number(12);
    if (!x.ok || q->dim() != 3 || (k != nullptr) != (ko != nullptr) || (k && k->dim() != 3)) Py_RETURN_NONE;
    const int64_t N = q->size(0), Hq = q->size(1), D = q->size(2), Hk = k ? k->size(1) : 0;
    const ScalarType type = q->scalar_type();
    const Rope r(x, turns, pos, N, 9);
    x.need(dtype_of(*q) >= 0 && rows(*q, N, Hq, D, type) && rows(*qo, N, Hq, D, type) &&
           (!k || (rows(*k, N, Hk, D, type) && rows(*ko, N, Hk, D, type))) && weight(wq, D, type) && weight(wk, D, type) &&
           N <= INT32_MAX && Hq <= INT32_MAX && Hk <= INT32_MAX && D <= INT32_MAX);
    x.current();
    if (!x.ok) Py_RETURN_NONE;
    return answer(norm_rotary_fn, q->data_ptr(), q->stride(0), q->stride(1), qo->data_ptr(), qo->stride(0), qo->stride(1), ptr(k),
                                 k ? k->stride(0) : 0, k ? k->stride(1) : 0, ptr(ko), ko ? ko->stride(0) : 0, ko ? ko->stride(1) : 0,
                                 ptr(wq), ptr(wk), (float)eps, r.positions, r.stride, r.use, r.turns, (float)m, (int)N, (int)Hq, (int)Hk,
                                 (int)D, r.rot, r.layout, (sd_dtype)dtype_of(*q), x.stream());
}

// q k v q_out positions turns cu_q kv_len page_table k_pages v_pages k_scale v_scale q_weight k_weight eps axes order layout magnitude
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Args x{a, n};
    if (n != 20) Py_RETURN_NONE;
    const at::Tensor *q = x.tensor(0, true), *k = x.tensor(1), *v = x.tensor(2), *qo = x.tensor(3, true), *pos = x.tensor(4, true),
                     *turns = x.tensor(5), *cu = x.tensor(6), *kv = x.tensor(7), *table = x.tensor(8), *kp = x.tensor(9),
                     *vp = x.tensor(10), *ks = x.tensor(11, true), *vs = x.tensor(12, true), *wq = x.tensor(13, true),
                     *wk = x.tensor(14, true);
    const double eps = x.number(15), m = x.number(19);
    if (!x.ok || k->dim() != 3 || (q != nullptr) != (qo != nullptr) || (q && q->dim() != 3)) Py_RETURN_NONE;
    const int64_t N = k->size(0), Hkv = k->size(1), D = k->size(2), Hq = q ? q->size(1) : 0;
    const ScalarType type = k->scalar_type();
    const Rope r(x, turns, pos, N, 16);
    const Cache c(x, kp, vp, table, ks, vs, type);
    if (!x.ok) Py_RETURN_NONE;
    x.need(dtype_of(*k) >= 0 && rows(*k, N, Hkv, D, type) && rows(*v, N, Hkv, D, type) && k->strides() == v->strides() &&
           (!q || (rows(*q, N, Hq, D, type) && rows(*qo, N, Hq, D, type) && qo->is_contiguous())) && c.Hkv == Hkv && c.D == D &&
           is_i32(*cu, (int64_t)c.B + 1) && is_i32(*kv, c.B) && weight(wq, D, type) && weight(wk, D, type) && N <= INT32_MAX &&
           Hq <= INT32_MAX);
    x.current();
    if (!x.ok) Py_RETURN_NONE;
    return answer(append_fn, ptr(q), q ? q->stride(0) : 0, q ? q->stride(1) : 0, k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1),
                            ptr(qo), ptr(wq), ptr(wk), (float)eps, r.positions, r.stride, r.use, r.turns, (float)m, r.rot, r.layout,
                            static_cast<const int32_t *>(cu->data_ptr()), static_cast<const int32_t *>(kv->data_ptr()), &c.c,
                            c.scaled ? &c.s : nullptr, (int)N, c.B, (int)Hq, (int)Hkv, (int)D, (sd_dtype)dtype_of(*k), x.stream());
}

// q k_pages v_pages k_scale v_scale page_table tree_mask cu_q kv_len max_q max_kv out scale ws causal (tree_mask None: no tree)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Args x{a, n};
    if (n != 15) Py_RETURN_NONE;
    const at::Tensor *q = x.tensor(0), *kp = x.tensor(1), *vp = x.tensor(2), *ks = x.tensor(3, true), *vs = x.tensor(4, true),
                     *table = x.tensor(5), *mask = x.tensor(6, true), *cu = x.tensor(7), *kv = x.tensor(8), *out = x.tensor(11),
                     *ws = x.tensor(13);
    const int max_q = x.whole(9), max_kv = x.whole(10), causal = x.whole(14);
    const double scale = x.number(12);
    if (!x.ok || q->dim() != 3 || (!mask && !ks)) Py_RETURN_NONE;
    const ScalarType type = q->scalar_type();
    const Cache c(x, kp, vp, table, ks, vs, type);
    if (!x.ok) Py_RETURN_NONE;
    const int64_t N = q->size(0), Hq = q->size(1), D = q->size(2);
    x.need(dtype_of(*q) >= 0 && rows(*q, N, Hq, D, type) && rows(*out, N, Hq, D, type) && out->is_contiguous() && c.D == D &&
           is_i32(*cu, (int64_t)c.B + 1) && is_i32(*kv, c.B) && N <= INT32_MAX && Hq <= INT32_MAX && ws->is_contiguous());
    if (mask) x.need(mask->scalar_type() == ScalarType::Long && mask->dim() == 1 && mask->size(0) == N && mask->is_contiguous());
    x.current();
    if (!x.ok) Py_RETURN_NONE;
    const int32_t *cup = static_cast<const int32_t *>(cu->data_ptr()), *kvp = static_cast<const int32_t *>(kv->data_ptr());
    if (mask)
        return answer(tree_fn, q->data_ptr(), q->stride(0), q->stride(1), &c.c, c.scaled ? &c.s : nullptr,
                              static_cast<const uint64_t *>(mask->data_ptr()), cup, kvp, max_q, max_kv, out->data_ptr(), (int)N, c.B,
                              (int)Hq, c.Hkv, (int)D, (sd_dtype)dtype_of(*q), (float)scale, ws->data_ptr(), ws->nbytes(), x.stream());
    return answer(attention_fn, q->data_ptr(), q->stride(0), q->stride(1), &c.c, &c.s, cup, kvp, max_q, max_kv, out->data_ptr(), (int)N,
                               c.B, (int)Hq, c.Hkv, (int)D, (sd_dtype)dtype_of(*q), (float)scale, causal ? 1 : 0, ws->data_ptr(),
                               ws->nbytes(), x.stream());
}

// k_pages v_pages page_table ctx_len path n_accepted k_scale v_scale
PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Args x{a, n};
    if (n != 8) Py_RETURN_NONE;
    const at::Tensor *kp = x.tensor(0), *vp = x.tensor(1), *table = x.tensor(2), *ctx = x.tensor(3), *path = x.tensor(4),
                     *acc = x.tensor(5), *ks = x.tensor(6, true), *vs = x.tensor(7, true);
    if (!x.ok) Py_RETURN_NONE;
    const Cache c(x, kp, vp, table, ks, vs, kp->scalar_type());
    if (!x.ok) Py_RETURN_NONE;
    const int dt = c.scaled ? (int)SD_BF16 : dtype_of(*kp);
    x.need(dt >= 0 && is_i32(*ctx, c.B) && is_i32(*acc, c.B) && path->dim() == 2 && path->size(0) == c.B && path->size(1) <= INT32_MAX &&
           path->scalar_type() == ScalarType::Int && path->is_contiguous());
    x.current();
    if (!x.ok) Py_RETURN_NONE;
    return answer(compact_fn, &c.c, c.scaled ? &c.s : nullptr, static_cast<const int32_t *>(ctx->data_ptr()),
                             static_cast<const int32_t *>(path->data_ptr()), static_cast<const int32_t *>(acc->data_ptr()), c.B,
                             (int)path->size(1), c.Hkv, c.D, (sd_dtype)dt, x.stream());
}

// bind(path of libsdverify.so): finds the entry points in the library that is already loaded
PyObject *bind(PyObject *, PyObject *arg) {
    const char *path = PyUnicode_AsUTF8(arg);
    if (!path) return nullptr;
    void *lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!lib) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    norm_rotary_fn = reinterpret_cast<decltype(norm_rotary_fn)>(dlsym(lib, "sd_norm_rotary"));
    append_fn = reinterpret_cast<decltype(append_fn)>(dlsym(lib, "sd_norm_rotary_append_paged"));
    attention_fn = reinterpret_cast<decltype(attention_fn)>(dlsym(lib, "sd_paged_attention_e4m3"));
    tree_fn = reinterpret_cast<decltype(tree_fn)>(dlsym(lib, "sd_paged_tree_attention"));
    compact_fn = reinterpret_cast<decltype(compact_fn)>(dlsym(lib, "sd_compact_tree_paged"));
    if (!norm_rotary_fn || !append_fn || !attention_fn || !tree_fn || !compact_fn) {
        PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point");
        return nullptr;
    }
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyCFunction entry() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>));
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"norm_rotary", entry<norm_rotary>(), METH_FASTCALL, nullptr},
                         {"append", entry<append>(), METH_FASTCALL, nullptr},
                         {"attend", entry<attend>(), METH_FASTCALL, nullptr},
                         {"compact", entry<compact>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_calls() { return PyModule_Create(&module); }
