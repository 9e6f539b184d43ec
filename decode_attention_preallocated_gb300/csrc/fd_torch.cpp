// fd_torch.cpp -- argument marshalling of the 4-bit cache and page calls for
// fd.py, as a Python extension: torch tensors become fd_tensor descriptors and
// addresses, what the C ABI cannot see (devices, and types and shapes of the
// int32 arrays) is checked, outputs are allocated, and libfd.so is called.  No
// arithmetic and no kernel of its own.
//
// A decode call hands over seven tensors.  Read through their Python attributes
// they take 10 us, more than the kernel of a short sequence runs, and a GPU
// that falls idle takes its next launch about 4 us later still: 1,000 positions
// of two heads, call after call, 18.0 us by attributes and 6.8 this way.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <cstring>

#include "fd.h"

namespace {

// libfd.so's calls and what fd.py lends: see bind()
struct {
    decltype(&fd_decode_fp4) decode;
    decltype(&fd_append_fp4) append;
    decltype(&fd_read_fp4) read;
    decltype(&fd_pages_reserve) reserve;
    decltype(&fd_pages_fork) fork;
    decltype(&fd_pages_free) free;
    decltype(&fd_pages_compact) compact;
    decltype(&fd_pages_copy) copy;
} fd;
PyObject *workspaces;   // {(device, stream): Workspace}
PyObject *opts_for;     // (workspace, device, stream, segments, rows, ctas, num_ctas) -> fd_opts as bytes
PyObject *empty_on;     // (shape, dtype, device, stream) -> tensor
PyObject *error;        // FdError(code, name)

struct Raised {};       // a Python exception is set

[[noreturn]] void raise(PyObject *type, const char *what) {
    PyErr_SetString(type, what);
    throw Raised{};
}

struct Ref {            // owns a reference
    PyObject *p;
    explicit Ref(PyObject *x) : p(x) {
        if (!p) throw Raised{};
    }
    Ref(const Ref &) = delete;
    ~Ref() { Py_XDECREF(p); }
};

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Raised{};
    }
    return THPVariable_Unpack(o);
}

int dtype_of(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return FD_BF16;
        case at::kFloat: return FD_F32;
        case at::kChar: return FD_I8;
        case at::kInt: return FD_I32;
        case at::kByte: return FD_U8;
        case at::kFloat8_e4m3fn: return FD_E4M3;
        default: return -1;
    }
}

// The call's device: that of its first tensor, and every other's.
struct Device {
    int index = -1;
    void on(const at::Tensor &t) {
        const int i = t.is_cuda() ? (int)t.get_device() : -1;
        if (index < 0) index = i;
        if (i < 0 || i != index) raise(PyExc_ValueError, "all tensors must be CUDA tensors on one device");
    }
};

fd_tensor describe(const at::Tensor &t, Device &dev) {
    dev.on(t);
    fd_tensor d{};
    d.dtype = dtype_of(t.scalar_type());
    if (d.dtype < 0) raise(PyExc_TypeError, "unsupported dtype");
    d.ndim = (int32_t)t.dim();
    if (d.ndim < 1 || d.ndim > 4) raise(PyExc_ValueError, "1 to 4 dimensions");
    d.data = t.data_ptr();
    for (int i = 0; i < d.ndim; ++i) {
        d.shape[i] = t.size(i);
        d.stride[i] = t.stride(i);
    }
    return d;
}

// Address of a contiguous int32 tensor [n] or, with m, [n, m]; 0 for None where
// that is allowed.
constexpr int64_t kNone = -1, kAny = -2;
int32_t *ints(PyObject *o, int64_t n, int64_t m, const char *name, Device &dev, bool none = false) {
    if (none && o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    dev.on(t);
    if (t.scalar_type() != at::kInt || t.dim() != (m == kNone ? 1 : 2) || (n != kAny && t.size(0) != n) ||
        (m >= 0 && t.size(1) != m) || !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous int32 tensor of the call's %s", name,
                     m == kNone ? "length" : "shape");
        throw Raised{};
    }
    return static_cast<int32_t *>(t.data_ptr());
}

float number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)x;
}

// An int32 argument; what does not fit is refused as the C ABI would refuse it.
int32_t whole(PyObject *o) {
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_ValueError, "an integer argument passes 32 bits");
    return (int32_t)x;
}

bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Raised{};
    return x != 0;
}

// The output a call makes: on the current stream, or by fd.py on a given one.
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, PyObject *dtype, const Device &dev, PyObject *stream) {
    if (stream == Py_None)
        return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev.index)));
    Ref size(PyTuple_New((Py_ssize_t)shape.size()));
    for (size_t i = 0; i < shape.size(); ++i) {
        PyObject *const x = PyLong_FromLongLong(shape[i]);
        if (!x) throw Raised{};
        PyTuple_SET_ITEM(size.p, (Py_ssize_t)i, x);
    }
    Ref index(PyLong_FromLong(dev.index));
    Ref t(PyObject_CallFunctionObjArgs(empty_on, size.p, dtype, index.p, stream, nullptr));
    return tensor(t.p, "out");
}

at::ScalarType scalar_of(PyObject *dtype) {
    if (!THPDtype_Check(dtype)) raise(PyExc_TypeError, "dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype *>(dtype)->scalar_type;
}

// Calls f(opts) with the call's device current.  The workspace is the given one
// or the stream's, which fd.py makes where there is none and enlarges where the
// call finds it too small.
template <typename F>
void run(const char *name, const Device &dev, PyObject *stream, PyObject *workspace, int64_t segments, int64_t rows,
         int64_t ctas, int64_t num_ctas, F f) {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev.index);
    fd_opts o{};
    const auto call = [&] {
        int rc;
        Py_BEGIN_ALLOW_THREADS
        rc = f(&o);
        Py_END_ALLOW_THREADS
        return rc;
    };
    int rc = FD_ERR_WORKSPACE;
    const bool plain = stream == Py_None && workspace == Py_None;
    if (plain) {
        void *const s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
        Ref key(Py_BuildValue("(iK)", dev.index, (unsigned long long)(uintptr_t)s));
        PyObject *found = PyDict_GetItemWithError(workspaces, key.p);   // borrowed
        if (!found && PyErr_Occurred()) throw Raised{};
        if (found) {
            // another thread may put a larger one in its place meanwhile; fd.py
            // destroys neither
            Ref ws(Py_NewRef(found));
            Ref handle(PyObject_GetAttrString(ws.p, "handle"));
            Ref value(PyObject_GetAttrString(handle.p, "value"));
            o.stream = s;
            o.ws = static_cast<fd_workspace *>(PyLong_AsVoidPtr(value.p));
            o.num_ctas = (int32_t)num_ctas;
            if (PyErr_Occurred()) throw Raised{};
            rc = call();
        }
    }
    if (!plain || rc == FD_ERR_WORKSPACE) {
        Ref b(PyObject_CallFunction(opts_for, "OiOLLLL", workspace, dev.index, stream, (long long)segments,
                                    (long long)rows, (long long)ctas, (long long)num_ctas));
        if (!PyBytes_Check(b.p) || PyBytes_GET_SIZE(b.p) != (Py_ssize_t)sizeof o) raise(PyExc_TypeError, "opts");
        memcpy(&o, PyBytes_AS_STRING(b.p), sizeof o);
        rc = call();
    }
    if (rc != FD_OK) {
        Ref e(PyObject_CallFunction(error, "is", rc, name));
        PyErr_SetObject(error, e.p);
        throw Raised{};
    }
}

// A method: no C++ exception leaves it.
template <Py_ssize_t N, PyObject *(*F)(PyObject *const *)>
PyObject *method(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        if (n != N) raise(PyExc_TypeError, "wrong number of arguments");
        return F(a);
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown failure");
        return nullptr;
    }
}

PyObject *none() { return Py_NewRef(Py_None); }

struct Cache {
    fd_tensor k, v, ks, vs;
    Cache(PyObject *const *a, Device &dev)
        : k(describe(tensor(a[0], "k_cache"), dev)), v(describe(tensor(a[1], "v_cache"), dev)),
          ks(describe(tensor(a[2], "k_scale"), dev)), vs(describe(tensor(a[3], "v_scale"), dev)) {}
};

struct Table {
    int32_t *p = nullptr, max_pages = 0;
    Table(PyObject *o, int64_t B, Device &dev) {
        if (o == Py_None) return;
        p = ints(o, B, kAny, "block_table", dev);
        max_pages = (int32_t)THPVariable_Unpack(o).size(1);
        // (an empty one has no address, which the C ABI reads as a flat cache)
        if (!p) raise(PyExc_ValueError, "block_table must have room for a page");
    }
};

// q, k, v, ks, vs, lengths, n_q, causal, scale, k_global, v_global, table, out, out_dtype, num_ctas, stream, workspace
PyObject *decode(PyObject *const *a) {
    Device dev;
    const at::Tensor &tq = tensor(a[0], "q");
    if (tq.dim() != 4) raise(PyExc_ValueError, "q must have four dimensions");
    const fd_tensor q = describe(tq, dev);
    const Cache c(a + 1, dev);
    const int64_t B = q.shape[0];
    const int32_t *lens = ints(a[5], B, kNone, "kv_lengths", dev);
    const int32_t n_q = a[6] == Py_None ? (int32_t)q.shape[1] : whole(a[6]);
    const bool causal = truth(a[7]);
    const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)q.shape[3])) : number(a[8]);
    const float kg = number(a[9]), vg = number(a[10]);
    const Table t(a[11], B, dev);
    const int32_t num_ctas = whole(a[14]);
    const at::Tensor made = a[12] == Py_None ? make(tq.sizes(), scalar_of(a[13]), a[13], dev, a[15]) : tensor(a[12], "out");
    const fd_tensor out = describe(made, dev);
    const int64_t Hkv = c.k.shape[1] > 0 ? c.k.shape[1] : 1, rows = q.shape[2] / Hkv * q.shape[1];   // over 32: two halves
    run("fd_decode_fp4", dev, a[15], a[16], B * Hkv * (rows > 32 ? 2 : 1), rows < 32 ? rows : 32,
        num_ctas > 1 ? num_ctas : 1, num_ctas, [&](const fd_opts *o) {
            return fd.decode(&q, &c.k, &c.v, &c.ks, &c.vs, kg, vg, t.p, t.max_pages, lens, n_q, causal, scale, &out, o);
        });
    return a[12] == Py_None ? THPVariable_Wrap(made) : Py_NewRef(a[12]);
}

// k_new, v_new, k, v, ks, vs, lengths, new_lengths, lengths_out, k_global, v_global, table, stream, workspace
PyObject *append(PyObject *const *a) {
    Device dev;
    const fd_tensor kn = describe(tensor(a[0], "k_new"), dev), vn = describe(tensor(a[1], "v_new"), dev);
    const Cache c(a + 2, dev);
    const int64_t B = kn.shape[0];
    const int32_t *lens = ints(a[6], B, kNone, "kv_lengths", dev);
    const int32_t *fresh = ints(a[7], B, kNone, "new_lengths", dev, true);
    int32_t *after = ints(a[8], B, kNone, "lengths_out", dev, true);
    const float kg = number(a[9]), vg = number(a[10]);
    const Table t(a[11], B, dev);
    run("fd_append_fp4", dev, a[12], a[13], 1, 1, 1, 0, [&](const fd_opts *o) {
        return fd.append(&kn, &vn, fresh, &c.k, &c.v, &c.ks, &c.vs, kg, vg, t.p, t.max_pages, lens, after, o);
    });
    return none();
}

// k, v, ks, vs, lengths, n, start, k_global, v_global, table, out, out_dtype, stream, workspace
PyObject *read(PyObject *const *a) {
    Device dev;
    const Cache c(a, dev);
    const at::Tensor &lengths = tensor(a[4], "kv_lengths");
    if (lengths.dim() != 1 || c.k.ndim != 4) raise(PyExc_ValueError, "kv_lengths [B] and a cache of four dimensions");
    const int64_t B = lengths.size(0);
    const int32_t *lens = ints(a[4], B, kNone, "kv_lengths", dev);
    const int32_t n = whole(a[5]);
    const int32_t *start = ints(a[6], B, kNone, "start", dev, true);
    const float kg = number(a[7]), vg = number(a[8]);
    const Table t(a[9], B, dev);
    at::Tensor ko, vo;
    if (a[10] == Py_None) {
        if (n < 0) raise(PyExc_ValueError, "n must not be negative");
        const int64_t shape[4] = {B, n, c.k.shape[1], 2 * c.k.shape[3]};
        const at::ScalarType type = scalar_of(a[11]);
        ko = make(shape, type, a[11], dev, a[12]);
        vo = make(shape, type, a[11], dev, a[12]);
    } else {
        Ref pair(PySequence_Fast(a[10], "out must be two tensors"));
        if (PySequence_Fast_GET_SIZE(pair.p) != 2) raise(PyExc_ValueError, "out must be two tensors");
        ko = tensor(PySequence_Fast_GET_ITEM(pair.p, 0), "out");
        vo = tensor(PySequence_Fast_GET_ITEM(pair.p, 1), "out");
        if (ko.dim() != 4 || ko.size(0) != B || ko.size(1) != n)
            raise(PyExc_ValueError, "out must be two [B, n, Hkv, d] tensors");
    }
    const fd_tensor dk = describe(ko, dev), dv = describe(vo, dev);
    run("fd_read_fp4", dev, a[12], a[13], 1, 1, 1, 0, [&](const fd_opts *o) {
        return fd.read(&c.k, &c.v, &c.ks, &c.vs, kg, vg, t.p, t.max_pages, start, lens, &dk, &dv, o);
    });
    Ref k(THPVariable_Wrap(ko)), v(THPVariable_Wrap(vo));
    return PyTuple_Pack(2, k.p, v.p);
}

// The books of a paged cache.
struct Books {
    int32_t *table, *lens = nullptr, *refs, B, max_pages, num_pages;
    Books(PyObject *t, PyObject *l, PyObject *r, Device &dev) {
        table = ints(t, kAny, kAny, "block_table", dev);
        refs = ints(r, kAny, kNone, "refs", dev);
        const at::Tensor &x = THPVariable_Unpack(t);
        const int64_t pages = THPVariable_Unpack(r).size(0);
        if (x.size(0) > INT32_MAX || x.size(1) > INT32_MAX || pages > INT32_MAX)
            raise(PyExc_ValueError, "books that pass 32 bits");
        B = (int32_t)x.size(0);
        max_pages = (int32_t)x.size(1);
        num_pages = (int32_t)pages;
        if (l) lens = ints(l, B, kNone, "kv_lengths", dev);
    }
};

// Segments of a default workspace (16 rows of head_dim 256 and two numbers each,
// for every segment and for 1024 blocks) whose room holds the scratch of reserve
// and compact.
int64_t scratch_slots(int64_t num_pages) {
    const int64_t n = 3 * num_pages / (16 * (256 + 2)) - 1000;
    return n > 1 ? n : 1;
}

// table, lengths, refs, page_size, n_new, pairs, count, stream, workspace
PyObject *reserve(PyObject *const *a) {
    Device dev;
    const Books k(a[0], a[1], a[2], dev);
    const int32_t page = whole(a[3]);
    int32_t each = 0;
    const int32_t *fresh = nullptr;
    if (THPVariable_Check(a[4])) fresh = ints(a[4], k.B, kNone, "n_new", dev);
    else each = whole(a[4]);
    PyObject *const int32 = reinterpret_cast<PyObject *>(torch::getTHPDtype(at::kInt));
    at::Tensor pairs, count;
    Ref p(a[5] == Py_None ? THPVariable_Wrap(pairs = make({k.B, 2}, at::kInt, int32, dev, a[7])) : Py_NewRef(a[5]));
    Ref c(a[6] == Py_None ? THPVariable_Wrap(count = make({1}, at::kInt, int32, dev, a[7])) : Py_NewRef(a[6]));
    int32_t *to = ints(p.p, k.B, 2, "pairs", dev), *n = ints(c.p, 1, kNone, "count", dev);
    run("fd_pages_reserve", dev, a[7], a[8], scratch_slots(k.num_pages), 1, 1, 0, [&](const fd_opts *o) {
        return fd.reserve(k.table, k.B, k.max_pages, k.lens, fresh, each, page, k.refs, k.num_pages, to, n, o);
    });
    return PyTuple_Pack(2, p.p, c.p);
}

// table, lengths, refs, page_size, src, dst, lengths of the copies, stream, workspace
PyObject *fork(PyObject *const *a) {
    Device dev;
    const Books k(a[0], a[1], a[2], dev);
    const int32_t page = whole(a[3]);
    const int32_t *src = ints(a[4], kAny, kNone, "src", dev);
    const int64_t n = THPVariable_Unpack(a[4]).size(0);
    const int32_t *dst = ints(a[5], n, kNone, "dst", dev), *given = ints(a[6], n, kNone, "lengths", dev, true);
    if (n > INT32_MAX) raise(PyExc_ValueError, "lists that pass 32 bits");
    run("fd_pages_fork", dev, a[7], a[8], 1, 1, 1, 0, [&](const fd_opts *o) {
        return fd.fork(k.table, k.B, k.max_pages, k.lens, page, k.refs, k.num_pages, src, dst, given, (int32_t)n, o);
    });
    return none();
}

// table, lengths, refs, page_size, seqs, lengths left, stream, workspace
PyObject *release(PyObject *const *a) {
    Device dev;
    const Books k(a[0], a[1], a[2], dev);
    const int32_t page = whole(a[3]);
    const int32_t *seqs = ints(a[4], kAny, kNone, "seqs", dev, true);
    const int64_t n = seqs || a[4] != Py_None ? THPVariable_Unpack(a[4]).size(0) : k.B;
    const int32_t *given = ints(a[5], n, kNone, "lengths", dev, true);
    if (n > INT32_MAX) raise(PyExc_ValueError, "lists that pass 32 bits");
    run("fd_pages_free", dev, a[6], a[7], 1, 1, 1, 0, [&](const fd_opts *o) {
        return fd.free(k.table, k.B, k.max_pages, k.lens, page, k.refs, k.num_pages, seqs, given, (int32_t)n, o);
    });
    return none();
}

// table, refs, pairs, count, stream, workspace
PyObject *compact(PyObject *const *a) {
    Device dev;
    const Books k(a[0], nullptr, a[1], dev);
    const int64_t half = k.num_pages / 2 > 1 ? k.num_pages / 2 : 1;
    PyObject *const int32 = reinterpret_cast<PyObject *>(torch::getTHPDtype(at::kInt));
    at::Tensor pairs, count;
    Ref p(a[2] == Py_None ? THPVariable_Wrap(pairs = make({half, 2}, at::kInt, int32, dev, a[4])) : Py_NewRef(a[2]));
    Ref c(a[3] == Py_None ? THPVariable_Wrap(count = make({1}, at::kInt, int32, dev, a[4])) : Py_NewRef(a[3]));
    int32_t *to = ints(p.p, half, 2, "pairs", dev), *n = ints(c.p, 1, kNone, "count", dev);
    run("fd_pages_compact", dev, a[4], a[5], scratch_slots(k.num_pages), 1, 1, 0, [&](const fd_opts *o) {
        return fd.compact(k.table, k.B, k.max_pages, k.refs, k.num_pages, to, n, o);
    });
    return PyTuple_Pack(2, p.p, c.p);
}

// pools as packed descriptors, their device, pairs, count, stream, workspace
PyObject *copy(PyObject *const *a) {
    Device dev;
    dev.index = whole(a[1]);
    const int32_t *pairs = ints(a[2], kAny, 2, "pairs", dev), *count = ints(a[3], 1, kNone, "count", dev);
    const int64_t most = THPVariable_Unpack(a[2]).size(0);
    if (!PyBytes_Check(a[0]) || most > INT32_MAX) raise(PyExc_ValueError, "packed pools and a list below 2^31 pairs");
    const auto *pools = reinterpret_cast<const fd_tensor *>(PyBytes_AS_STRING(a[0]));
    const int64_t n = PyBytes_GET_SIZE(a[0]) / (Py_ssize_t)sizeof(fd_tensor);
    run("fd_pages_copy", dev, a[4], a[5], 1, 1, 1, 0, [&](const fd_opts *o) {
        return fd.copy(pools, (int32_t)n, pairs, count, (int32_t)most, o);
    });
    return none();
}

// addresses of the eight calls, the workspaces, opts_for, empty_on, FdError
PyObject *bind(PyObject *const *a) {
    void **const to = reinterpret_cast<void **>(&fd);
    if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 8 || !PyDict_Check(a[1])) raise(PyExc_TypeError, "bind");
    for (Py_ssize_t i = 0; i < 8; ++i) to[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
    if (PyErr_Occurred()) throw Raised{};
    Py_XSETREF(workspaces, Py_NewRef(a[1]));
    Py_XSETREF(opts_for, Py_NewRef(a[2]));
    Py_XSETREF(empty_on, Py_NewRef(a[3]));
    Py_XSETREF(error, Py_NewRef(a[4]));
    return none();
}

template <Py_ssize_t N, PyObject *(*F)(PyObject *const *)>
PyMethodDef entry(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<N, F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {entry<17, decode>("decode_fp4"), entry<14, append>("append_fp4"), entry<14, read>("read_fp4"),
                         entry<9, reserve>("pages_reserve"), entry<9, fork>("pages_fork"),
                         entry<8, release>("pages_free"), entry<6, compact>("pages_compact"),
                         entry<6, copy>("pages_copy"), entry<5, bind>("bind"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_fd_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fd_torch() { return PyModule_Create(&module_def); }
