// run_binding.cpp -- the Python binding's argument marshalling for the short calls over ragged runs (append and
// read-back), as a CPython extension.
//
// A decode step's append is two microseconds of GPU time; checking and converting its fifteen tensors in Python took
// five, here about half of one.  Checks, their order and their errors are those of csa.py; the library itself is loaded by
// csa.py, which hands over the entry points' addresses.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <exception>
#include <initializer_list>

#include "csa.h"

namespace {

struct PyError {};   // a Python error is set

decltype(&csa_kv_append_fp4) append_entry = nullptr;
decltype(&csa_kv_unpack_fp4) unpack_entry = nullptr;
PyObject *names[12];
enum { kCodes, kScales, kKeys, kSwa, kSwaScale, kSeqLen, kBlockTable, kSwaRow, kNumPages, kNumRows, kB, kMaxPages };
const char *const kNames[12] = {"codes", "scales", "keys", "swa", "swa_scale", "seq_len", "block_table", "swa_row",
                                "num_pages", "num_rows", "B", "max_pages"};
PyObject *max_seq_len_name, *cuda_stream_name;

struct Ref {
    PyObject *p;
    explicit Ref(PyObject *o) : p(o)
    {
        if (!p) throw PyError();
    }
    Ref(const Ref &) = delete;
    ~Ref() { Py_DECREF(p); }
};

int as_int(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyError();
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_SetString(PyExc_OverflowError, "value does not fit 32 bits");
        throw PyError();
    }
    return (int)v;
}

int int_attr(PyObject *o, PyObject *name)
{
    const Ref r(PyObject_GetAttr(o, name));
    return as_int(r.p);
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch tensor", name);
        throw PyError();
    }
    return THPVariable_Unpack(o);
}

// Address of a contiguous tensor on device dev; 0 for None.
template <typename T>
T *address(PyObject *o, const char *name, int dev)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    const char *wrong = !t.is_cuda() ? "%s must be a CUDA tensor (the library has no CPU path)"
                        : !t.is_contiguous() ? "%s must be contiguous"
                        : t.get_device() != dev ? "%s is not on the current device" : nullptr;
    if (wrong) {
        PyErr_Format(PyExc_ValueError, wrong, name);
        throw PyError();
    }
    return static_cast<T *>(t.data_ptr());
}

template <typename T>
T *address_attr(PyObject *o, int name, int dev)
{
    const Ref r(PyObject_GetAttr(o, names[name]));
    return address<T>(r.p, kNames[name], dev);   // the owner keeps the tensor
}

void check_array(PyObject *o, const char *name, at::ScalarType type, const char *type_name, std::initializer_list<int64_t> shape)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape)) return;
    Ref dims(PyList_New(0));
    for (const int64_t d : shape) {
        const Ref v(PyLong_FromLongLong(d));
        if (PyList_Append(dims.p, v.p) != 0) throw PyError();
    }
    PyErr_Format(PyExc_ValueError, "%s must be %s of shape %R", name, type_name, dims.p);
    throw PyError();
}

int rows_of(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (t.dim() < 1 || t.size(0) > INT_MAX) {
        PyErr_Format(PyExc_ValueError, "%s has no rows, or too many", name);
        throw PyError();
    }
    return (int)t.size(0);
}

// What every call over a run takes.
struct Call {
    csa_kv_layer layer;
    csa_batch batch;
    int dev;
    const int32_t *cu_rows;
    void *ws, *stream;
    size_t ws_bytes;
};

void check_rows(PyObject *batch, PyObject *cu_rows)
{
    const at::Tensor &t = tensor(cu_rows, "cu_rows");
    if (t.scalar_type() != at::kInt || t.numel() != (int64_t)int_attr(batch, names[kB]) + 1) {
        PyErr_SetString(PyExc_ValueError, "cu_rows must be int32 with batch.B + 1 entries");
        throw PyError();
    }
}

Call call_of(PyObject *layer, PyObject *batch, PyObject *cu_rows, PyObject *ws, PyObject *stream)
{
    Call c;
    const at::Tensor &w = tensor(ws, "ws");
    if (!w.is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "ws must be a CUDA tensor (the library has no CPU path)");
        throw PyError();
    }
    c.dev = c10::cuda::current_device();
    if (w.get_device() != c.dev) {
        PyErr_Format(PyExc_ValueError, "ws is on device %d, which is not the current one", (int)w.get_device());
        throw PyError();
    }
    c.layer.codes = address_attr<uint8_t>(layer, kCodes, c.dev);
    c.layer.scales = address_attr<uint8_t>(layer, kScales, c.dev);
    c.layer.keys = address_attr<uint8_t>(layer, kKeys, c.dev);
    c.layer.swa = address_attr<uint8_t>(layer, kSwa, c.dev);
    c.layer.swa_scale = address_attr<float>(layer, kSwaScale, c.dev);
    c.layer.num_pages = int_attr(layer, names[kNumPages]);
    c.layer.num_rows = int_attr(layer, names[kNumRows]);
    c.batch.B = int_attr(batch, names[kB]);
    c.batch.seq_len = address_attr<int32_t>(batch, kSeqLen, c.dev);
    c.batch.block_table = address_attr<int32_t>(batch, kBlockTable, c.dev);
    c.batch.max_pages = int_attr(batch, names[kMaxPages]);
    c.batch.swa_row = address_attr<int32_t>(batch, kSwaRow, c.dev);
    c.batch.max_seq_len = int_attr(batch, max_seq_len_name);
    c.cu_rows = address<int32_t>(cu_rows, "cu_rows", c.dev);
    c.ws = address<void>(ws, "ws", c.dev);
    c.ws_bytes = (size_t)w.numel();
    if (stream == Py_None) {
        c.stream = c10::cuda::getCurrentCUDAStream(c.dev).stream();
    } else {
        const Ref h(PyObject_GetAttr(stream, cuda_stream_name));
        c.stream = PyLong_AsVoidPtr(h.p);
        if (!c.stream && PyErr_Occurred()) throw PyError();
    }
    return c;
}

// Runs f, which returns the call's status; errors become Python's.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want || !append_entry || !unpack_entry) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or the library is not bound");
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const PyError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// kv_append_fp4(layer, batch, cu_rows, latent, idx_key, ws, norm_weight, rope_table, stream) -> status
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> long {
        const int rows = rows_of(a[3], "latent");
        check_rows(a[1], a[2]);
        check_array(a[3], "latent", at::kBFloat16, "torch.bfloat16", {rows, 512});
        check_array(a[4], "idx_key", at::kBFloat16, "torch.bfloat16", {rows, 128});
        if (a[6] != Py_None) check_array(a[6], "norm_weight", at::kFloat, "torch.float32", {512});
        int positions = 0;
        if (a[7] != Py_None) {
            positions = rows_of(a[7], "rope_table");
            check_array(a[7], "rope_table", at::kFloat, "torch.float32", {positions, 32, 2});
        }
        const Call c = call_of(a[0], a[1], a[2], a[5], a[8]);
        const uint16_t *latent = address<uint16_t>(a[3], "latent", c.dev), *key = address<uint16_t>(a[4], "idx_key", c.dev);
        const float *norm = address<float>(a[6], "norm_weight", c.dev), *rope = address<float>(a[7], "rope_table", c.dev);
        csa_status s;
        Py_BEGIN_ALLOW_THREADS
        s = append_entry(&c.layer, &c.batch, c.cu_rows, rows, latent, key, norm, rope, positions, c.ws, c.ws_bytes, c.stream);
        Py_END_ALLOW_THREADS
        return s;
    });
}

// kv_unpack_fp4(layer, batch, cu_rows, latent, ws, stream) -> status
PyObject *kv_unpack(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> long {
        const int rows = rows_of(a[3], "latent");
        check_rows(a[1], a[2]);
        check_array(a[3], "latent", at::kBFloat16, "torch.bfloat16", {rows, 512});
        const Call c = call_of(a[0], a[1], a[2], a[4], a[5]);
        uint16_t *latent = address<uint16_t>(a[3], "latent", c.dev);
        csa_status s;
        Py_BEGIN_ALLOW_THREADS
        s = unpack_entry(&c.layer, &c.batch, c.cu_rows, rows, latent, c.ws, c.ws_bytes, c.stream);
        Py_END_ALLOW_THREADS
        return s;
    });
}

// bind(address of csa_kv_append_fp4, address of csa_kv_unpack_fp4)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "two addresses");
        return nullptr;
    }
    void *p[2];
    for (int i = 0; i < 2; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no address");
            return nullptr;
        }
    append_entry = reinterpret_cast<decltype(append_entry)>(p[0]);
    unpack_entry = reinterpret_cast<decltype(unpack_entry)>(p[1]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"kv_append_fp4", (PyCFunction)(void (*)())kv_append, METH_FASTCALL, nullptr},
                         {"kv_unpack_fp4", (PyCFunction)(void (*)())kv_unpack, METH_FASTCALL, nullptr},
                         {"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_runs", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__runs(void)
{
    for (int i = 0; i < 12; ++i)
        if (!(names[i] = PyUnicode_InternFromString(kNames[i]))) return nullptr;
    if (!(max_seq_len_name = PyUnicode_InternFromString("max_seq_len"))) return nullptr;
    if (!(cuda_stream_name = PyUnicode_InternFromString("cuda_stream"))) return nullptr;
    PyObject *m = PyModule_Create(&module);
    // the PyTorch whose headers this was compiled with (build.py names it): csa.py refuses it under another one
    if (m && PyModule_AddStringConstant(m, "torch_version", CSA_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
