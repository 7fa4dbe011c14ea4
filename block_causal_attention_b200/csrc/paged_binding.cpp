// The paged cache's operators as Python functions over torch tensors (module _paged_binding):
// argument checks, allocation and the calls of include/bca.h.  A single token's attention takes
// the GPU 6.1 us (one token of 128 heads over 1,536 keys, D = 24); the same checks by interpreter
// steps and ctypes took 19 us a call, compiled they take 7.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/api/include/torch/version.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <sstream>

#include "../../include/bca.h"

namespace {

// What PagedCache.__init__ knows, for every later call.
struct Cache {
    bca_paged_t handle;
    int64_t hq, hkv, d, layers, pool_bytes;
    char *k_pages, *v_pages;
    at::ScalarType dtype, o_dtype;
    int device;
};
constexpr const char *kCapsule = "bca_paged_cache";

Cache *cache_of(PyObject *o) { return static_cast<Cache *>(PyCapsule_GetPointer(o, kCapsule)); }

struct Refused {};  // a Python error is set

std::string shape_text(at::IntArrayRef s) {
    std::ostringstream t;
    t << "(";
    for (size_t i = 0; i < s.size(); ++i) t << (i ? ", " : "") << s[i];
    t << ")";
    return t.str();
}

// The tensor's memory, if it is what the call needs.
void *tensor(const Cache &c, const char *name, PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
        throw Refused();
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() == type && t.is_cuda() && t.get_device() == c.device && t.sizes() == shape && t.is_contiguous())
        return t.data_ptr();
    std::ostringstream s;
    s << name << ": expected a contiguous " << c10::toString(type) << " tensor of shape " << shape_text(shape)
      << " on cuda:" << c.device << ", got " << (t.is_contiguous() ? "" : "a non-contiguous ")
      << c10::toString(t.scalar_type()) << " " << shape_text(t.sizes()) << " on " << t.device().str();
    PyErr_SetString(PyExc_ValueError, s.str().c_str());
    throw Refused();
}
void *tensor_or_null(const Cache &c, const char *name, PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : tensor(c, name, o, type, shape);
}

int64_t rows_of(const char *name, PyObject *o, int64_t dims) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
        throw Refused();
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != dims) {
        PyErr_Format(PyExc_ValueError, "%s: expected %lld dimensions, got shape %s", name, (long long)dims,
                     shape_text(t.sizes()).c_str());
        throw Refused();
    }
    return t.size(0);
}

int64_t whole(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refused();
    return x;
}

int64_t layer_of(const Cache &c, PyObject *o) {
    const int64_t layer = whole(o);
    if (layer < 0 || layer >= c.layers) {
        PyErr_Format(PyExc_ValueError, "layer %lld of %lld", (long long)layer, (long long)c.layers);
        throw Refused();
    }
    return layer;
}

// None: the current stream of the cache's device; else a cudaStream_t as a number.
cudaStream_t stream_of(const Cache &c, PyObject *o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.device).stream();
    void *s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) throw Refused();
    return static_cast<cudaStream_t>(s);
}

void gain_needs_pos(PyObject *pos, PyObject *gain, const char *name) {
    if (pos != Py_None || gain == Py_None) return;
    PyErr_Format(PyExc_ValueError, "%s needs pos: rows without positions are taken as post-prologue", name);
    throw Refused();
}

bool arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return false;
}

// cache(handle, hq, hkv, d, layers, pool_bytes, k_pages, v_pages, fp16, o_fp32, device)
PyObject *make(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 11)) return nullptr;
    int64_t x[11];
    for (int i = 0; i < 11; ++i) {
        x[i] = PyLong_AsLongLong(a[i]);
        if (x[i] == -1 && PyErr_Occurred()) return nullptr;
    }
    Cache *c = new (std::nothrow) Cache();
    if (!c) return PyErr_NoMemory();
    c->handle = reinterpret_cast<bca_paged_t>(x[0]);
    c->hq = x[1], c->hkv = x[2], c->d = x[3], c->layers = x[4], c->pool_bytes = x[5];
    c->k_pages = reinterpret_cast<char *>(x[6]), c->v_pages = reinterpret_cast<char *>(x[7]);
    c->dtype = x[8] ? at::kHalf : at::kBFloat16;
    c->o_dtype = x[9] ? at::kFloat : c->dtype;
    c->device = (int)x[10];
    PyObject *cap = PyCapsule_New(c, kCapsule, [](PyObject *o) { delete cache_of(o); });
    if (!cap) delete c;
    return cap;
}

// write(cache, k, v, table, off, start, pos, k_gain, layer, stream) -> status
PyObject *write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 10)) return nullptr;
    const Cache *c = cache_of(a[0]);
    if (!c) return nullptr;
    HANDLE_TH_ERRORS
    try {
        const int64_t layer = layer_of(*c, a[8]);
        const int64_t rows = rows_of("k", a[1], 3), seqs = rows_of("table", a[3], 2);
        const int64_t width = THPVariable_Unpack(a[3]).size(1);
        void *k = tensor(*c, "k", a[1], c->dtype, {rows, c->hkv, c->d});
        void *v = tensor(*c, "v", a[2], c->dtype, {rows, c->hkv, c->d});
        void *table = tensor(*c, "table", a[3], at::kInt, {seqs, width});
        void *off = tensor(*c, "off", a[4], at::kInt, {seqs + 1});
        void *start = tensor(*c, "start", a[5], at::kInt, {seqs});
        gain_needs_pos(a[6], a[7], "k_gain");
        void *pos = tensor_or_null(*c, "pos", a[6], at::kInt, {rows, 3});
        void *gain = tensor_or_null(*c, "k_gain", a[7], at::kFloat, {c->d});
        if (seqs > INT32_MAX || width > INT32_MAX) return PyLong_FromLong(BCA_ERR_INVALID_ARGUMENT);
        return PyLong_FromLong(bca_paged_write(
            c->handle, k, v, rows, (const int32_t *)pos, (const float *)gain, (const int32_t *)table, (int32_t)seqs,
            (int32_t)width, (const int32_t *)off, (const int32_t *)start, c->k_pages + layer * c->pool_bytes,
            c->v_pages + layer * c->pool_bytes, stream_of(*c, a[9])));
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// copy(cache, pairs (int32 [n, 2], CPU), stream) -> status
PyObject *copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 3)) return nullptr;
    const Cache *c = cache_of(a[0]);
    if (!c) return nullptr;
    HANDLE_TH_ERRORS
    try {
        const int64_t count = rows_of("pairs", a[1], 2);
        const at::Tensor &t = THPVariable_Unpack(a[1]);
        if (!t.device().is_cpu() || t.scalar_type() != at::kInt || t.size(1) != 2 || !t.is_contiguous()) {
            PyErr_SetString(PyExc_ValueError, "pairs: expected contiguous int32 [n, 2] on the host");
            return nullptr;
        }
        return PyLong_FromLong(bca_paged_copy(c->handle, t.data_ptr<int32_t>(), count, c->k_pages, c->v_pages,
                                              stream_of(*c, a[2])));
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

at::Tensor empty_on(const Cache &c, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)c.device));
}

// attend(cache, q, table, off, k_begin, k_end, seq, causal, pos, q_gain, layer, o, lse, workspace, stream)
// -> o, or a status below 0
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 15)) return nullptr;
    const Cache *c = cache_of(a[0]);
    if (!c) return nullptr;
    HANDLE_TH_ERRORS
    try {
        const int causal = PyObject_IsTrue(a[7]);
        if (causal < 0) return nullptr;
        const int64_t layer = layer_of(*c, a[10]);
        const int64_t nq = rows_of("q", a[1], 3), seqs = rows_of("table", a[2], 2), ends = rows_of("off", a[3], 1);
        const int64_t width = THPVariable_Unpack(a[2]).size(1), slices = ends - 1;
        if (slices < 0) {
            PyErr_SetString(PyExc_ValueError, "off: expected int32 [slices + 1]");
            return nullptr;
        }
        if (a[6] == Py_None && slices != seqs) {
            PyErr_SetString(PyExc_ValueError, "seq=None needs as many slices as table rows");
            return nullptr;
        }
        void *q = tensor(*c, "q", a[1], c->dtype, {nq, c->hq, c->d});
        void *table = tensor(*c, "table", a[2], at::kInt, {seqs, width});
        void *off = tensor(*c, "off", a[3], at::kInt, {ends});
        void *kb = tensor(*c, "k_begin", a[4], at::kInt, {slices});
        void *ke = tensor(*c, "k_end", a[5], at::kInt, {slices});
        void *seq = tensor_or_null(*c, "seq", a[6], at::kInt, {slices});
        gain_needs_pos(a[8], a[9], "q_gain");
        void *pos = tensor_or_null(*c, "pos", a[8], at::kInt, {nq, 3});
        void *gain = tensor_or_null(*c, "q_gain", a[9], at::kFloat, {c->d});
        void *lse = tensor_or_null(*c, "lse", a[12], at::kFloat, {c->hq, nq});
        if (seqs > INT32_MAX || width > INT32_MAX || slices > INT32_MAX)
            return PyLong_FromLong(BCA_ERR_INVALID_ARGUMENT);
        const cudaStream_t stream = stream_of(*c, a[14]);

        // What this call allocates belongs to the stream that it runs on, so that memory given
        // back at its end has its next user behind it.
        const auto current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c->device);
        std::optional<c10::cuda::CUDAStreamGuard> guard;
        if (current.stream() != stream)
            guard.emplace(c10::cuda::getStreamFromExternal(stream, (c10::DeviceIndex)c->device));
        at::Tensor o, workspace;
        void *op, *ws = nullptr;
        if (a[11] == Py_None) {
            o = empty_on(*c, {nq, c->hq, c->d}, c->o_dtype);
            op = o.data_ptr();
        } else {
            op = tensor(*c, "o", a[11], c->o_dtype, {nq, c->hq, c->d});
        }
        const int64_t bytes = (int64_t)bca_paged_workspace_bytes(c->handle, nq, (int32_t)slices, (int32_t)width);
        if (a[13] == Py_None) {
            if (bytes > 0) {
                workspace = empty_on(*c, {bytes}, at::kByte);
                ws = workspace.data_ptr();
            }
        } else {
            if (!THPVariable_Check(a[13])) {
                PyErr_SetString(PyExc_TypeError, "workspace: expected a tensor");
                return nullptr;
            }
            const at::Tensor &w = THPVariable_Unpack(a[13]);
            if (!w.is_cuda() || w.get_device() != c->device || !w.is_contiguous() || (int64_t)w.nbytes() < bytes) {
                PyErr_Format(PyExc_ValueError, "workspace: expected %lld contiguous bytes on cuda:%d", (long long)bytes,
                             c->device);
                return nullptr;
            }
            ws = w.data_ptr();
        }
        guard.reset();
        const int rc = bca_paged_attend(
            c->handle, q, nq, (const int32_t *)pos, (const float *)gain, c->k_pages + layer * c->pool_bytes,
            c->v_pages + layer * c->pool_bytes, (const int32_t *)table, (int32_t)seqs, (int32_t)width,
            (const int32_t *)off, (const int32_t *)seq, (const int32_t *)kb, (const int32_t *)ke, (int32_t)slices, causal,
            op, (float *)lse, ws, stream);
        if (rc != BCA_OK) return PyLong_FromLong(rc);
        if (a[11] == Py_None) return THPVariable_Wrap(std::move(o));
        return Py_NewRef(a[11]);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"cache", (PyCFunction)(void (*)(void))make, METH_FASTCALL, nullptr},
    {"write", (PyCFunction)(void (*)(void))write, METH_FASTCALL, nullptr},
    {"copy", (PyCFunction)(void (*)(void))copy, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
