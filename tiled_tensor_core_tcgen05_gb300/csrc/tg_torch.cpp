// The tensor forms of a serving step's calls (rotary positions and the 8-bit
// cache): argument checks, outputs, the current stream, and the C ABI call, in
// one step. A single token's kernels take a few microseconds, less than these
// checks take in Python and the conversion of some thirty arguments by ctypes.
// Each function returns the tg_status as an int where the library refuses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <cstdint>
#include <optional>
#include <string>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tg_gemm.h"

namespace {

struct Refused {};  // a Python error has been set

[[noreturn]] void type_error(const std::string& m) {
    PyErr_SetString(PyExc_TypeError, m.c_str());
    throw Refused{};
}
[[noreturn]] void value_error(const std::string& m) {
    PyErr_SetString(PyExc_ValueError, m.c_str());
    throw Refused{};
}

std::string shape_of(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.dim() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* x, const char* name) {
    if (!THPVariable_Check(x)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(x);
}

// The kernels run on the current device, with its stream: tensors of another one are not reached from there.
void check_device(int64_t has, int64_t current, const char* name) {
    if (has != current)
        value_error(std::string(name) + " is on cuda:" + std::to_string(has) + ", but the current device is cuda:" + std::to_string(current));
}

thread_local int t_device = -1;  // the current device, once a call has asked

void on_cuda(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
    if (t_device < 0) t_device = c10::cuda::current_device();
    check_device(t.get_device(), t_device, name);
}

int64_t integer(PyObject* x) {
    const int64_t v = PyLong_AsLongLong(x);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

// One of the C ABI's int arguments.
int small(PyObject* x, const char* name) {
    const int64_t v = integer(x);
    if (v != static_cast<int>(v)) value_error(std::string(name) + " is out of range: " + std::to_string(v));
    return static_cast<int>(v);
}

double real(PyObject* x) {
    const double v = PyFloat_AsDouble(x);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}

bool truth(PyObject* x) {
    const int v = PyObject_IsTrue(x);
    if (v < 0) throw Refused{};
    return v != 0;
}

int dtype_code(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kHalf) return TG_FP16;
    if (t.scalar_type() == at::kBFloat16) return TG_BF16;
    type_error(std::string(name) + " must be float16 or bfloat16, got " + c10::toString(t.scalar_type()));
}

struct Rows {
    void* p = nullptr;
    int64_t token = 0, head = 0;
};

// A (tokens, heads, dim) tensor, contiguous along dim.
Rows rows(const at::Tensor& t, const char* name) {
    if (t.dim() != 3) value_error(std::string(name) + " must have shape (tokens, heads, dim), got " + shape_of(t));
    on_cuda(t, name);
    if (t.size(2) > 1 && t.stride(2) != 1) value_error(std::string(name) + " must be contiguous along its last dimension");
    return Rows{t.data_ptr(), t.stride(0), t.stride(1)};
}

const int32_t* ints(PyObject* x, const char* name, int64_t n, int64_t m = -1) {
    const at::Tensor& t = tensor(x, name);
    if (t.scalar_type() != at::kInt) type_error(std::string(name) + " must be int32, got " + c10::toString(t.scalar_type()));
    on_cuda(t, name);
    if (!(m < 0 ? t.dim() == 1 && t.size(0) == n : t.dim() == 2 && t.size(0) == n && t.size(1) == m))
        value_error(std::string(name) + " must have shape (" + std::to_string(n) + (m < 0 ? ",)" : ", " + std::to_string(m) + ")") + ", got " + shape_of(t));
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return static_cast<const int32_t*>(t.data_ptr());
}

const double* frequencies(PyObject* x, int64_t* rotary) {
    const at::Tensor& t = tensor(x, "inv_freq");
    if (t.scalar_type() != at::kDouble || !t.is_cuda() || t.dim() != 1 || !t.is_contiguous())
        type_error("inv_freq must be a contiguous CUDA float64 vector (radians per position of each pair)");
    on_cuda(t, "inv_freq");
    *rotary = 2 * t.size(0);
    return static_cast<const double*>(t.data_ptr());
}

// The stream of a call: the current one, or the given torch stream, which is then current for allocations.
struct Where {
    tg_stream_t handle;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    explicit Where(PyObject* stream) {
        const c10::DeviceIndex dev = c10::cuda::current_device();
        if (stream == Py_None) {
            handle = reinterpret_cast<tg_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
            return;
        }
        PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
        if (raw == nullptr) throw Refused{};
        void* p = PyLong_AsVoidPtr(raw);
        Py_DECREF(raw);
        if (p == nullptr && PyErr_Occurred()) throw Refused{};
        handle = static_cast<tg_stream_t>(p);
        guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), dev));
    }
};

struct Cache {
    void *k, *v;
    float *ks, *vs;
    int64_t pages, kv_heads, page, dim;
    int format;
};

// A cache's tensors k, v, k_scale, v_scale, looked at in every call: their storage may have been exchanged or resized
// since the last one. A cache may be made while another device is the current one.
Cache cache_of(PyObject* const* a, bool making) {
    static const char* names[4] = {"k", "v", "k_scale", "v_scale"};
    const at::Tensor* t[4];
    for (int i = 0; i < 4; ++i) t[i] = &tensor(a[i], names[i]);
    const auto type = t[0]->scalar_type();
    if (type != at::kFloat8_e4m3fn && type != at::kChar)
        type_error(std::string("codes must be float8_e4m3fn or int8, got ") + c10::toString(type));
    if (t[0]->dim() != 4 || t[0]->sizes() != t[1]->sizes() || t[1]->scalar_type() != type)
        value_error("k and v must share one (pages, kv_heads, page, dim) shape and one type");
    for (int i = 2; i < 4; ++i) {
        if (t[i]->scalar_type() != at::kFloat) type_error("scales must be float32");
        if (t[i]->dim() != 2 || t[i]->size(0) != t[0]->size(0) || t[i]->size(1) != t[0]->size(1))
            value_error("scales must have shape (" + std::to_string(t[0]->size(0)) + ", " + std::to_string(t[0]->size(1)) + ")");
    }
    for (int i = 0; i < 4; ++i) {
        if (!making) on_cuda(*t[i], names[i]);
        else if (!t[i]->is_cuda()) type_error(std::string(names[i]) + " must be a CUDA tensor");
        else if (t[i]->get_device() != t[0]->get_device()) value_error("the cache's tensors must be on one device");
        if (!t[i]->is_contiguous()) value_error(std::string(names[i]) + " must be contiguous");
    }
    return Cache{t[0]->data_ptr(), t[1]->data_ptr(), static_cast<float*>(t[2]->data_ptr()), static_cast<float*>(t[3]->data_ptr()), t[0]->size(0),
                 t[0]->size(1), t[0]->size(2), t[0]->size(3), type == at::kChar ? TG_KV_INT8 : TG_KV_E4M3};
}

// What KvCache keeps: its four tensors.
Cache cache(PyObject* t) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 4) type_error("cache must be a KvCache");
    PyObject* const a[4] = {PyTuple_GET_ITEM(t, 0), PyTuple_GET_ITEM(t, 1), PyTuple_GET_ITEM(t, 2), PyTuple_GET_ITEM(t, 3)};
    return cache_of(a, false);
}

struct Batch {
    const int32_t* table;
    int64_t width;
    const int32_t *lens, *cu;
    int64_t batch;
};

Batch batch(PyObject* table, PyObject* lens, PyObject* cu) {
    const at::Tensor& t = tensor(table, "table");
    if (t.dim() != 2) value_error("table must have shape (batch, pages a sequence), got " + shape_of(t));
    Batch b;
    b.batch = t.size(0);
    b.width = t.size(1);
    b.table = ints(table, "table", b.batch, b.width);
    b.lens = ints(lens, "lens", b.batch);
    b.cu = cu == Py_None ? nullptr : ints(cu, "cu", b.batch + 1);
    return b;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
    HANDLE_TH_ERRORS
    t_device = -1;
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, n);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// Runs a library call without the interpreter lock; a status other than TG_OK is the answer.
template <typename F, typename R>
PyObject* answer(F call, R result) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call();
    Py_END_ALLOW_THREADS
    return status == TG_OK ? result() : PyLong_FromLong(status);
}

// What torch keeps account of when a tensor is overwritten: a backward pass that saved it says so instead of reading
// other values.
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject* x) {
    if (x != Py_None) written(tensor(x, "out"));
}

PyObject* same(PyObject* x) {
    Py_INCREF(x);
    return x;
}

// (X, positions, inv_freq, amplitude, layout, backward, out, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const at::Tensor& X = tensor(a[0], "X");
        const Rows x = rows(X, "X");
        const int dtype = dtype_code(X, "X");
        int64_t rotary = 0;
        const double* freq = frequencies(a[2], &rotary);
        const int64_t T = X.size(0), H = X.size(1), D = X.size(2);
        const int32_t* pos = ints(a[1], "positions", T);
        const double amplitude = real(a[3]);
        const int layout = small(a[4], "layout"), backward = truth(a[5]);
        const Where where(a[7]);
        at::Tensor made;
        if (a[6] == Py_None) made = at::empty({T, H, D}, X.options());
        const at::Tensor& Y = a[6] == Py_None ? made : tensor(a[6], "out");
        if (Y.sizes() != X.sizes()) value_error("out has the wrong shape");
        if (Y.scalar_type() != X.scalar_type()) type_error("out has the wrong type");
        const Rows y = rows(Y, "out");
        return answer(
            [&] { return tg_rope(x.p, x.token, x.head, y.p, y.token, y.head, pos, T, H, D, freq, rotary, amplitude, layout, backward, dtype, where.handle); },
            [&] {
                written(a[6]);
                return made.defined() ? THPVariable_Wrap(std::move(made)) : same(a[6]);
            });
    });
}

// (k, v, k_scale, v_scale) -> what KvCache keeps
PyObject* cache_args(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        cache_of(a, true);
        return PyTuple_Pack(4, a[0], a[1], a[2], a[3]);
    });
}

// (cache, K, V, table, lens, cu, max_new, Q, inv_freq, amplitude, layout, out, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const Cache c = cache(a[0]);
        const at::Tensor &K = tensor(a[1], "K"), &V = tensor(a[2], "V");
        const Rows k = rows(K, "K"), v = rows(V, "V");
        const int dtype = dtype_code(K, "K");
        if (V.scalar_type() != K.scalar_type()) type_error("V must have K's type");
        const int64_t T = K.size(0);
        if (K.sizes() != V.sizes() || K.size(1) != c.kv_heads || K.size(2) != c.dim)
            value_error("K and V must have shape (total, " + std::to_string(c.kv_heads) + ", " + std::to_string(c.dim) + "), got " + shape_of(K) + " and " + shape_of(V));
        const Batch b = batch(a[3], a[4], a[5]);
        const int64_t max_new = integer(a[6]);
        int64_t rotary = 0;
        const double* freq = a[8] == Py_None ? nullptr : frequencies(a[8], &rotary);
        const double amplitude = real(a[9]);
        const int layout = small(a[10], "layout");
        const Where where(a[12]);
        at::Tensor made;
        Rows q, qo;
        int64_t heads = 0;
        if (a[7] != Py_None) {
            if (freq == nullptr) value_error("Q is only rotated: it needs inv_freq");
            const at::Tensor& Q = tensor(a[7], "Q");
            q = rows(Q, "Q");
            if (Q.scalar_type() != K.scalar_type()) type_error("Q must have K's type");
            if (Q.size(0) != T || Q.size(2) != c.dim)
                value_error("Q must have shape (" + std::to_string(T) + ", heads, " + std::to_string(c.dim) + "), got " + shape_of(Q));
            heads = Q.size(1);
            if (a[11] == Py_None) made = at::empty(Q.sizes(), Q.options());
            const at::Tensor& O = a[11] == Py_None ? made : tensor(a[11], "out");
            if (O.sizes() != Q.sizes()) value_error("out has the wrong shape");
            if (O.scalar_type() != Q.scalar_type()) type_error("out has the wrong type");
            qo = rows(O, "out");
        } else if (a[11] != Py_None) {
            value_error("out is for the rotated Q");
        }
        return answer(
            [&] {
                return tg_kv_append(c.k, c.v, c.ks, c.vs, c.pages, c.kv_heads, c.page, c.dim, c.format, k.p, k.token, k.head, v.p, v.token, v.head, b.table, b.width,
                                    b.lens, b.cu, b.batch, T, max_new, freq, rotary, amplitude, layout, q.p, q.token, q.head, qo.p, qo.token, qo.head, heads, dtype,
                                    where.handle);
            },
            [&] {
                for (int i = 0; i < 4; ++i) written(PyTuple_GET_ITEM(a[0], i));
                written(a[11]);
                return made.defined() ? THPVariable_Wrap(std::move(made)) : same(a[11]);
            });
    });
}

// (cache, table, first, cu, total, bf16, K or None, V or None, stream)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const Cache c = cache(a[0]);
        const Batch b = batch(a[1], a[2], a[3]);
        const int64_t total = integer(a[4]);
        if (total < 0) value_error("total must not be negative");
        const Where where(a[8]);
        at::Tensor made[2];
        int dtype = truth(a[5]) ? TG_BF16 : TG_FP16;
        void* to[2];
        for (int i = 0; i < 2; ++i) {
            if (a[6 + i] == Py_None) {
                made[i] = at::empty({total, c.kv_heads, c.dim}, tensor(PyTuple_GET_ITEM(a[0], 0), "k").options().dtype(dtype == TG_BF16 ? at::kBFloat16 : at::kHalf));
                to[i] = made[i].data_ptr();
                continue;
            }
            const at::Tensor& t = tensor(a[6 + i], "out");
            on_cuda(t, "out");
            if (t.dim() != 3 || t.size(0) != total || t.size(1) != c.kv_heads || t.size(2) != c.dim || !t.is_contiguous())
                value_error("out must be two contiguous tensors of shape (" + std::to_string(total) + ", " + std::to_string(c.kv_heads) + ", " + std::to_string(c.dim) + ")");
            if (dtype_code(t, "out") != dtype) type_error("out has the wrong type");
            to[i] = t.data_ptr();
        }
        return answer(
            [&] { return tg_kv_read(c.k, c.v, c.ks, c.vs, c.pages, c.kv_heads, c.page, c.dim, c.format, b.table, b.width, b.lens, b.cu, b.batch, total, to[0], to[1], dtype, where.handle); },
            [&]() -> PyObject* {
                written(a[6]);
                written(a[7]);
                PyObject* pair = PyTuple_New(2);
                for (int i = 0; pair != nullptr && i < 2; ++i)
                    PyTuple_SET_ITEM(pair, i, made[i].defined() ? THPVariable_Wrap(std::move(made[i])) : same(a[6 + i]));
                return pair;
            });
    });
}

// (Q, cache, table, lens, cu, max_new, max_len, causal, window, scale, return_lse, out, stream)
PyObject* attention_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor& Q = tensor(a[0], "Q");
        const Rows q = rows(Q, "Q");
        const int dtype = dtype_code(Q, "Q");
        const Cache c = cache(a[1]);
        const int64_t T = Q.size(0), H = Q.size(1), D = Q.size(2);
        if (D != c.dim) value_error("Q must have shape (total, heads, " + std::to_string(c.dim) + "), got " + shape_of(Q));
        const Batch b = batch(a[2], a[3], a[4]);
        const int64_t max_new = integer(a[5]), max_len = a[6] == Py_None ? b.width * c.page : integer(a[6]), window = integer(a[8]);
        const int causal = truth(a[7]);
        const double scale = a[9] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : real(a[9]);
        const bool want_lse = truth(a[10]);
        const Where where(a[12]);
        int64_t need = 0;
        const int status = tg_attention_kv_workspace(c.kv_heads, c.page, D, c.format, H, b.batch, T, max_new, max_len, window, dtype, &need);
        if (status != TG_OK) return PyLong_FromLong(status);
        at::Tensor made, lse, work;
        if (a[11] == Py_None) made = at::empty({T, H, D}, Q.options());
        const at::Tensor& O = a[11] == Py_None ? made : tensor(a[11], "out");
        if (O.sizes() != Q.sizes() || O.scalar_type() != Q.scalar_type() || !O.is_cuda() || !O.is_contiguous())
            value_error("out must be a contiguous CUDA tensor of Q's shape and type");
        on_cuda(O, "out");
        if (want_lse) lse = at::empty({T, H}, Q.options().dtype(at::kFloat));
        if (need > 0) work = at::empty({need}, Q.options().dtype(at::kByte));
        void *po = O.data_ptr(), *pw = need > 0 ? work.data_ptr() : nullptr;
        float* pl = want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
        return answer(
            [&] {
                return tg_attention_kv(q.p, q.token, q.head, po, pl, c.k, c.v, c.ks, c.vs, c.pages, c.kv_heads, c.page, c.dim, c.format, b.table, b.width, b.lens,
                                       b.cu, b.batch, T, H, max_new, max_len, causal, window, scale, dtype, pw, need, where.handle);
            },
            [&]() -> PyObject* {
                written(a[11]);
                PyObject* o = made.defined() ? THPVariable_Wrap(std::move(made)) : same(a[11]);
                if (!want_lse || o == nullptr) return o;
                PyObject* pair = PyTuple_New(2);
                if (pair == nullptr) return nullptr;
                PyTuple_SET_ITEM(pair, 0, o);
                PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(lse)));
                return pair;
            });
    });
}

// (device that a tensor has, current device, name): the check above, for a machine with one
PyObject* check_device_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        const char* name = PyUnicode_AsUTF8(a[2]);
        if (name == nullptr) return nullptr;
        check_device(integer(a[0]), integer(a[1]), name);
        Py_RETURN_NONE;
    });
}

PyMethodDef methods[] = {
    {"check_device", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(check_device_py)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"cache_args", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_args)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_read)), METH_FASTCALL, nullptr},
    {"attention_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_kv)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tg_torch() { return PyModule_Create(&module); }
