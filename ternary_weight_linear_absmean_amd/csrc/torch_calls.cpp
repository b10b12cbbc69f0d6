// torch_calls.cpp -- the binding's short way into the calls on the paged caches:
// the module `_calls`.
//
// A call through ctypes looks at seven to twelve tensors from Python and takes 9
// us of host time for a single token's attention, of which 2.5 are the launch; a
// decode step waits for it.  The functions here look at the same tensors in C++ (4 us).  They
// take what a call takes when nothing is out of the ordinary -- plain tensors,
// contiguous, of the types and shapes that the call wants, on the current GPU --
// and return NotImplemented, with nothing done, for anything else and for whatever the library
// refuses: the Python of _native.py then makes the call, or says what is wrong with it.
// A launch that the runtime reports as failed may be under way all the same (the
// runtime gives an earlier call's error too), so that status is raised here and the
// call not made again: queries rotated in place would turn twice.
//
// The library's entry points come in by address (bind), so this module is not
// linked against it.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bitlinear.h"

namespace {

struct Entries {
    decltype(&bitlinear_kv8_append) kv8_append;
    decltype(&bitlinear_kv8_append_rope) kv8_append_rope;
    decltype(&bitlinear_kv4_append) kv4_append;
    decltype(&bitlinear_kv8_read) kv8_read;
    decltype(&bitlinear_kv4_read) kv4_read;
    decltype(&bitlinear_kv8_attention) kv8_attention;
    decltype(&bitlinear_kv4_attention) kv4_attention;
    decltype(&bitlinear_kv8_attention_ws_bytes) kv8_ws;
    decltype(&bitlinear_kv4_attention_ws_bytes) kv4_ws;
} lib;

struct Unusual {};                          // left to Python

const at::Tensor &tensor(PyObject *o) {
    if (!THPVariable_CheckExact(o)) throw Unusual();
    return THPVariable_Unpack(o);
}

// GPU of a tensor that a call begins with: the current one.
int gpu_of(const at::Tensor &t) {
    if (!t.is_cuda() || t.device().index() != c10::hip::current_device()) throw Unusual();
    return t.device().index();
}

// Address of a contiguous tensor of a type and shape on a GPU.
void *at_address(const at::Tensor &t, int gpu, at::ScalarType type, at::IntArrayRef shape) {
    if (!t.is_cuda() || t.device().index() != gpu || t.scalar_type() != type || t.sizes() != shape ||
        !t.is_contiguous())
        throw Unusual();
    return t.data_ptr();
}
void *at_address(PyObject *o, int gpu, at::ScalarType type, at::IntArrayRef shape) {
    return at_address(tensor(o), gpu, type, shape);
}

bl_dtype rows_type(at::ScalarType t) {
    if (t == at::kFloat) return BL_F32;
    if (t == at::kBFloat16) return BL_BF16;
    throw Unusual();
}

bool is_none(PyObject *o) { return o == Py_None; }

struct Cache {
    int bits;
    bl_kv8 c8;
    bl_kv4 c4;
    int64_t KVH, T, D;
};
Cache cache_of(PyObject *o, int bits, int gpu) {
    if (!PyTuple_Check(o) && !PyList_Check(o)) throw Unusual();
    if (PySequence_Fast_GET_SIZE(o) != 4) throw Unusual();
    PyObject **part = PySequence_Fast_ITEMS(o);
    const at::Tensor &K = tensor(part[0]);
    if (K.dim() != 4) throw Unusual();
    const int64_t nb = K.size(0), KVH = K.size(1), T = K.size(2);
    Cache c = {bits, {}, {}, KVH, T, bits == 8 ? K.size(3) : 2 * K.size(3)};
    if (bits == 8) {
        c.c8 = {static_cast<int8_t *>(at_address(K, gpu, at::kChar, {nb, KVH, T, c.D})),
                static_cast<int8_t *>(at_address(part[1], gpu, at::kChar, {nb, KVH, c.D, T})),
                static_cast<float *>(at_address(part[2], gpu, at::kFloat, {nb, KVH})),
                static_cast<float *>(at_address(part[3], gpu, at::kFloat, {nb, KVH})), nb, KVH, T, c.D};
    } else {
        c.c4 = {static_cast<uint8_t *>(at_address(K, gpu, at::kByte, {nb, KVH, T, c.D / 2})),
                static_cast<uint8_t *>(at_address(part[1], gpu, at::kByte, {nb, KVH, T / 16, c.D, 8})),
                static_cast<uint16_t *>(at_address(part[2], gpu, at::kHalf, {nb, KVH, T, 2})),
                static_cast<uint16_t *>(at_address(part[3], gpu, at::kHalf, {nb, KVH, T, 2})), nb, KVH, T, c.D};
    }
    return c;
}

struct Seqs {
    const int32_t *q_start, *lengths, *table;
    int64_t B, max_blocks;
};
Seqs seqs_of(PyObject *q_start, PyObject *lengths, PyObject *table, int gpu) {
    const at::Tensor &t = tensor(table);
    if (t.dim() != 2) throw Unusual();
    const int64_t B = t.size(0), nb = t.size(1);
    return {static_cast<const int32_t *>(at_address(q_start, gpu, at::kInt, {B + 1})),
            static_cast<const int32_t *>(at_address(lengths, gpu, at::kInt, {B})),
            static_cast<const int32_t *>(at_address(t, gpu, at::kInt, {B, nb})), B, nb};
}

void *stream_of(int gpu) { return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(gpu)).stream(); }

// Past the dispatcher (0.3 us a tensor) where nobody looks on and nothing is to be filled.
at::Tensor fresh(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type) {
    const at::Context &torch = at::globalContext();
    if (!c10::impl::TorchDispatchModeTLS::any_modes_set() &&
        !(torch.deterministicAlgorithms() && torch.deterministicFillUninitializedMemory()))
        return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

PyObject *left() { Py_RETURN_NOTIMPLEMENTED; }
// The binding's own way of raising, raises(call, status).
PyObject *raises = nullptr;
PyObject *failed(const char *call, bl_status st) {
    if (st != BL_ERR_HIP) return left();
    PyObject *none = PyObject_CallFunction(raises, "si", call, (int)st);
    Py_XDECREF(none);
    return none ? left() : nullptr;
}

template <typename F>
bl_status without_gil(F f) {
    PyThreadState *state = PyEval_SaveThread();
    const bl_status st = f();
    PyEval_RestoreThread(state);
    return st;
}

template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        return left();
    }
}

// append(bits, k, v, q_start, lengths, table, cache, rope, q, q_out)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10) return left();
    return guarded([&]() -> PyObject * {
        const int bits = PyLong_AsLong(a[0]) == 8 ? 8 : 4;
        const at::Tensor &k = tensor(a[1]);
        const int gpu = gpu_of(k);
        const at::ScalarType type = k.scalar_type();
        const bl_dtype dt = rows_type(type);
        const Cache c = cache_of(a[6], bits, gpu);
        if (k.dim() != 3) throw Unusual();
        const int64_t rows = k.size(0);
        const void *kp = at_address(k, gpu, type, {rows, c.KVH, c.D});
        const void *vp = at_address(a[2], gpu, type, {rows, c.KVH, c.D});
        const Seqs s = seqs_of(a[3], a[4], a[5], gpu);
        bl_rope rope = {};
        if (!is_none(a[7])) {
            if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 2) throw Unusual();
            const at::Tensor &table = tensor(PyTuple_GET_ITEM(a[7], 0));
            if (table.dim() != 2) throw Unusual();
            rope.rows = table.size(0);
            rope.rot = table.size(1);
            rope.cos_sin = static_cast<const float *>(at_address(table, gpu, at::kFloat, {rope.rows, rope.rot}));
            const int pairs = PyObject_IsTrue(PyTuple_GET_ITEM(a[7], 1));
            if (pairs < 0) throw Unusual();
            rope.interleaved = pairs;
        } else if (!is_none(a[8])) {
            throw Unusual();
        }
        int64_t QH = 0;
        const void *qp = nullptr;
        void *op = nullptr;
        at::Tensor made;
        if (!is_none(a[8])) {
            const at::Tensor &q = tensor(a[8]);
            if (q.dim() != 3) throw Unusual();
            QH = q.size(1);
            qp = at_address(q, gpu, type, {rows, QH, c.D});
            if (is_none(a[9])) {
                made = fresh(q.sizes(), q, type);
                op = made.data_ptr();
            } else {
                op = at_address(a[9], gpu, type, {rows, QH, c.D});
            }
        } else if (!is_none(a[9])) {
            throw Unusual();
        }
        void *stream = stream_of(gpu);
        const bl_status st = without_gil([&] {
            if (bits == 4)
                return lib.kv4_append(kp, vp, qp, op, dt, rows, QH, s.q_start, s.lengths, s.table, s.B, s.max_blocks,
                                      &c.c4, is_none(a[7]) ? nullptr : &rope, stream);
            if (is_none(a[7]))
                return lib.kv8_append(kp, vp, dt, rows, s.q_start, s.lengths, s.table, s.B, s.max_blocks, &c.c8,
                                      stream);
            return lib.kv8_append_rope(kp, vp, qp, op, dt, rows, QH, s.q_start, s.lengths, s.table, s.B, s.max_blocks,
                                       &c.c8, &rope, stream);
        });
        if (st != BL_OK) return failed(bits == 4      ? "bitlinear_kv4_append"
                                       : is_none(a[7]) ? "bitlinear_kv8_append"
                                                       : "bitlinear_kv8_append_rope",
                                       st);
        if (made.defined()) return THPVariable_Wrap(made);
        Py_INCREF(a[9]);
        return a[9];
    });
}

// read(bits, q_start, lengths, table, cache, n_tok, dtype, k, v)
PyObject *read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) return left();
    return guarded([&]() -> PyObject * {
        const int bits = PyLong_AsLong(a[0]) == 8 ? 8 : 4;
        if ((!PyTuple_Check(a[4]) && !PyList_Check(a[4])) || PySequence_Fast_GET_SIZE(a[4]) != 4) throw Unusual();
        const at::Tensor &K = tensor(PySequence_Fast_GET_ITEM(a[4], 0));
        const int gpu = gpu_of(K);
        const Cache c = cache_of(a[4], bits, gpu);
        const Seqs s = seqs_of(a[1], a[2], a[3], gpu);
        if (!PyLong_CheckExact(a[5])) throw Unusual();
        const int64_t rows = PyLong_AsLongLong(a[5]);
        if (rows < 0) throw Unusual();
        if (!THPDtype_Check(a[6])) throw Unusual();
        const at::ScalarType type = reinterpret_cast<THPDtype *>(a[6])->scalar_type;
        const bl_dtype dt = rows_type(type);
        at::Tensor out[2];
        void *p[2];
        for (int i = 0; i < 2; ++i) {
            out[i] = is_none(a[7 + i]) ? fresh({rows, c.KVH, c.D}, K, type) : tensor(a[7 + i]);
            p[i] = at_address(out[i], gpu, type, {rows, c.KVH, c.D});
        }
        void *stream = stream_of(gpu);
        const bl_status st = without_gil([&] {
            return bits == 4 ? lib.kv4_read(&c.c4, s.q_start, s.lengths, s.table, s.B, s.max_blocks, rows, p[0], p[1], dt,
                                            stream)
                             : lib.kv8_read(&c.c8, s.q_start, s.lengths, s.table, s.B, s.max_blocks, rows, p[0], p[1], dt,
                                            stream);
        });
        if (st != BL_OK) return failed(bits == 4 ? "bitlinear_kv4_read" : "bitlinear_kv8_read", st);
        PyObject *both = PyTuple_New(2);
        if (!both) return nullptr;
        for (int i = 0; i < 2; ++i) {
            PyObject *o = a[7 + i];
            if (is_none(o)) o = THPVariable_Wrap(out[i]);
            else Py_INCREF(o);
            PyTuple_SET_ITEM(both, i, o);
        }
        return both;
    });
}

// attention(bits, q, q_start, lengths, table, cache, scale, out, ws)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9) return left();
    return guarded([&]() -> PyObject * {
        const int bits = PyLong_AsLong(a[0]) == 8 ? 8 : 4;
        const at::Tensor &q = tensor(a[1]);
        const int gpu = gpu_of(q);
        const at::ScalarType type = q.scalar_type();
        const bl_dtype dt = rows_type(type);
        const Cache c = cache_of(a[5], bits, gpu);
        if (q.dim() != 3) throw Unusual();
        const int64_t rows = q.size(0), QH = q.size(1);
        const void *qp = at_address(q, gpu, type, {rows, QH, c.D});
        const Seqs s = seqs_of(a[2], a[3], a[4], gpu);
        float scale;
        if (is_none(a[6])) {
            scale = (float)(1.0 / std::sqrt((double)c.D));
        } else {
            const double x = PyFloat_AsDouble(a[6]);
            if (PyErr_Occurred()) throw Unusual();
            scale = (float)x;
        }
        at::Tensor made, ws;
        void *op;
        if (is_none(a[7])) {
            made = fresh(q.sizes(), q, type);
            op = made.data_ptr();
        } else {
            op = at_address(a[7], gpu, type, {rows, QH, c.D});
        }
        size_t bytes;
        void *wp = nullptr;
        if (is_none(a[8])) {
            bytes = (bits == 4 ? lib.kv4_ws : lib.kv8_ws)(rows, QH, s.B, s.max_blocks, c.KVH, c.T, c.D);
            if (bytes > 0) {
                ws = fresh({(int64_t)bytes}, q, at::kByte);
                wp = ws.data_ptr();
            }
        } else {
            const at::Tensor &w = tensor(a[8]);
            bytes = (size_t)w.numel();
            wp = at_address(w, gpu, at::kByte, {w.numel()});
        }
        void *stream = stream_of(gpu);
        const bl_status st = without_gil([&] {
            return bits == 4 ? lib.kv4_attention(qp, dt, rows, QH, s.q_start, s.lengths, s.table, s.B, s.max_blocks, &c.c4,
                                                 scale, op, wp, bytes, stream)
                             : lib.kv8_attention(qp, dt, rows, QH, s.q_start, s.lengths, s.table, s.B, s.max_blocks, &c.c8,
                                                 scale, op, wp, bytes, stream);
        });
        if (st != BL_OK) return failed(bits == 4 ? "bitlinear_kv4_attention" : "bitlinear_kv8_attention", st);
        if (made.defined()) return THPVariable_Wrap(made);
        Py_INCREF(a[7]);
        return a[7];
    });
}

// bind(raises, addresses of the entry points in the order of Entries)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[sizeof(Entries) / sizeof(void *)];
    if (n != 1 + (Py_ssize_t)(sizeof p / sizeof *p)) {
        PyErr_SetString(PyExc_TypeError, "bind: wrong number of arguments");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n - 1; ++i) {
        p[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    static_assert(sizeof p == sizeof lib, "entry points are addresses");
    memcpy(&lib, p, sizeof lib);
    Py_INCREF(a[0]);
    Py_XSETREF(raises, a[0]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"read", (PyCFunction)(void (*)(void))read, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and the Python whose headers this was compiled with.
PyMODINIT_FUNC PyInit__calls() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) Py_CLEAR(m);
    return m;
}
