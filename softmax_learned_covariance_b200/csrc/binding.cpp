// binding.cpp -- the paged-cache calls of the Python binding in native code.
//
// A decode step of one short sequence takes the GPU a few microseconds; checking
// a dozen tensors and allocating two outputs from Python took 16 (26 before that was
// made as lean as it gets); a whole call takes 6 to 7 with these functions, which
// do the same -- check, allocate on the tensors' device and its current stream,
// call the C ABI -- and nothing else; the library's entry points are handed over
// by address (bind), so there is one loaded library and no second path.
//
// Each returns its outputs, or the library's status (an int) when it is not 0.
// Wrong types raise TypeError, wrong shapes, layouts or devices ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "parallax.h"

namespace {

using Q8Fn = decltype(&parallax_decode_paged_q8);
using AccFn = decltype(&parallax_decode_paged_acc);
using AppendFn = decltype(&parallax_kv_append);
using EvictFn = decltype(&parallax_kv_evict);
Q8Fn g_q8 = nullptr;
AccFn g_acc = nullptr;
AppendFn g_append = nullptr;
EvictFn g_evict = nullptr;

[[noreturn]] void bad_type(const char *name, const char *what) {
    TORCH_CHECK_TYPE(false, name, " must be ", what);
    abort();
}

// A tensor argument, or an undefined tensor for None where that is allowed.
at::Tensor tensor(PyObject *o, const char *name, bool may_be_none = false) {
    if (o == Py_None && may_be_none) return {};
    if (!THPVariable_Check(o)) bad_type(name, "a tensor");
    return THPVariable_Unpack(o);
}

// A tensor a kernel reads or writes whole: contiguous, on `dev`, of this type and shape.
void is(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, at::Device dev) {
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type);
    TORCH_CHECK_VALUE(t.sizes() == shape && t.device() == dev && t.is_contiguous(), name,
                      " must be a contiguous tensor of shape ", shape, " on ", dev);
}

template <typename T = void> T *at_(const at::Tensor &t) { return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr; }

struct Cache {
    at::Tensor k, v, kexp, vexp, table, seqlens;
    at::Device dev{at::kCPU};
    int64_t B, Hkv, ps, mp, np, d;
    bool q8;
};

int small(int64_t n, const char *name) {
    TORCH_CHECK_VALUE(n >= 0 && n <= 0x7fffffff, name, " is out of range: ", n);
    return (int)n;
}

Cache cache(PyObject *k, PyObject *v, PyObject *kexp, PyObject *vexp, PyObject *table, PyObject *seqlens) {
    Cache c;
    c.k = tensor(k, "kpages");
    c.v = tensor(v, "vpages");
    c.kexp = tensor(kexp, "kexp", true);
    c.vexp = tensor(vexp, "vexp", true);
    c.table = tensor(table, "block_table");
    c.seqlens = tensor(seqlens, "seqlens");
    const at::ScalarType type = c.k.scalar_type();
    c.q8 = type == at::kFloat8_e4m3fn;
    TORCH_CHECK_TYPE(c.q8 || type == at::kBFloat16, "unsupported cache dtype ", type);
    TORCH_CHECK_VALUE(c.k.is_cuda() && c.k.is_contiguous(), "kpages must be a contiguous CUDA tensor");
    TORCH_CHECK_VALUE(c.k.dim() == 4 && c.table.dim() == 2 && c.k.size(2) >= 16,
                      "kpages must be [num_pages, Hkv, page_size >= 16, d] and block_table [B, max_pages]");
    c.dev = c.k.device();
    c.np = c.k.size(0);
    c.Hkv = c.k.size(1);
    c.ps = c.k.size(2);
    c.d = c.k.size(3);
    c.B = c.table.size(0);
    c.mp = c.table.size(1);
    is(c.v, "vpages", type, c.k.sizes(), c.dev);
    if (c.q8) {
        TORCH_CHECK_VALUE(c.kexp.defined() && c.vexp.defined(), "an e4m3 cache needs kexp and vexp");
        const int64_t shape[3] = {c.np, c.Hkv, c.ps / 16};
        is(c.kexp, "kexp", at::kChar, shape, c.dev);
        is(c.vexp, "vexp", at::kChar, shape, c.dev);
    } else {
        TORCH_CHECK_VALUE(!c.kexp.defined() && !c.vexp.defined(), "a bf16 cache has no exponents");
    }
    is(c.table, "block_table", at::kInt, {c.B, c.mp}, c.dev);
    is(c.seqlens, "seqlens", at::kInt, {c.B}, c.dev);
    small(c.np, "num_pages");
    small(c.mp, "max_pages");
    small(c.B, "B");
    small(c.Hkv, "Hkv");
    return c;
}

void *stream_of(const at::Device &dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// An uninitialised tensor from torch's allocator, without the dispatcher's 0.5 us.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev) {
    return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

// steals the references
PyObject *tuple(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    bool ok = t != nullptr;
    for (PyObject *o : items) ok = ok && o != nullptr;
    for (PyObject *o : items) {
        if (ok)
            PyTuple_SET_ITEM(t, i++, o);
        else
            Py_XDECREF(o);
    }
    if (!ok) {
        Py_XDECREF(t);
        return nullptr;
    }
    return t;
}

// Other Python threads run while this one allocates and calls the library: either may
// wait there (for room in the launch queue, whose head may be a host callback that
// needs the interpreter), and torch's own calls and the ctypes ones let them as well.
struct NoGil {
    PyThreadState *state = PyEval_SaveThread();
    NoGil() = default;
    NoGil(const NoGil &) = delete;
    NoGil &operator=(const NoGil &) = delete;
    ~NoGil() { PyEval_RestoreThread(state); }
};

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, not %zd", want, n);
    return false;
}

long long whole(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}

// (q, rho, kpages, vpages, kexp, vexp, block_table, seqlens, wacc, y, lse, out_dtype, want_lse, q8) -> (y, lse)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 14)) return nullptr;
    at::ScalarType out_type = at::kFloat;
    if (a[11] != Py_None) {
        if (!THPDtype_Check(a[11])) bad_type("out_dtype", "a dtype");
        out_type = reinterpret_cast<THPDtype *>(a[11])->scalar_type;
        TORCH_CHECK_TYPE(out_type == at::kFloat || out_type == at::kBFloat16, "unsupported dtype ", out_type);
    }
    const bool want_q8 = a[13] == Py_True, want_lse = PyObject_IsTrue(a[12]) == 1;
    if (PyErr_Occurred()) return nullptr;
    TORCH_CHECK_TYPE(tensor(a[2], "kpages").scalar_type() == (want_q8 ? at::kFloat8_e4m3fn : at::kBFloat16),
                     "kpages must be ", want_q8 ? "float8_e4m3fn" : "bfloat16");
    const Cache c = cache(a[2], a[3], a[4], a[5], a[6], a[7]);
    const at::Tensor q = tensor(a[0], "q"), rho = tensor(a[1], "rho", true), wacc = tensor(a[8], "wacc", true);
    at::Tensor y = tensor(a[9], "y", true), lse = tensor(a[10], "lse", true);
    TORCH_CHECK_VALUE(q.dim() == 3, "q must be [B, Hq, d]");
    const int64_t Hq = q.size(1), shape[3] = {c.B, Hq, c.d};
    is(q, "q", at::kBFloat16, shape, c.dev);
    if (rho.defined()) is(rho, "rho", at::kBFloat16, shape, c.dev);
    if (wacc.defined()) is(wacc, "wacc", at::kFloat, {c.B, c.Hkv, c.mp * c.ps}, c.dev);
    TORCH_CHECK_VALUE(c.q8 || wacc.defined(), "wacc is required; without it use parallax_decode_paged");
    const int B = (int)c.B, hq = small(Hq, "Hq"), hkv = (int)c.Hkv, ps = small(c.ps, "page_size"), d = small(c.d, "d");
    int st;
    {
        const NoGil no_gil;
        const c10::cuda::CUDAGuard guard(c.dev);
        if (y.defined()) {
            TORCH_CHECK_TYPE(y.scalar_type() == at::kFloat || y.scalar_type() == at::kBFloat16, "unsupported dtype of y");
            is(y, "y", y.scalar_type(), shape, c.dev);
        } else {
            y = fresh(shape, out_type, c.dev);
        }
        if (lse.defined())
            is(lse, "lse", at::kFloat, {c.B, Hq}, c.dev);
        else if (want_lse)
            lse = fresh({c.B, Hq}, at::kFloat, c.dev);
        const int out = y.scalar_type() == at::kFloat ? PARALLAX_F32 : PARALLAX_BF16;
        st = c.q8 ? g_q8(at_(q), at_(rho), at_(c.k), at_(c.v), at_<signed char>(c.kexp), at_<signed char>(c.vexp),
                         at_<int>(c.table), at_<int>(c.seqlens), at_(y), at_<float>(lse), at_<float>(wacc), B, hq,
                         hkv, ps, (int)c.mp, (int)c.np, d, PARALLAX_BF16, out, stream_of(c.dev))
                  : g_acc(at_(q), at_(rho), at_(c.k), at_(c.v), at_<int>(c.table), at_<int>(c.seqlens), at_(y),
                          at_<float>(lse), at_<float>(wacc), B, hq, hkv, ps, (int)c.mp, (int)c.np, d,
                          PARALLAX_BF16, out, stream_of(c.dev));
    }
    if (st) return PyLong_FromLong(st);
    return tuple({wrap(y), wrap(lse)});
    END_HANDLE_TH_ERRORS
}

// (k, v, kpages, vpages, kexp, vexp, block_table, seqlens, counts, new_seqlens, wacc) -> new_seqlens
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 11)) return nullptr;
    const Cache c = cache(a[2], a[3], a[4], a[5], a[6], a[7]);
    const at::Tensor x[2] = {tensor(a[0], "k"), tensor(a[1], "v")}, counts = tensor(a[8], "counts", true),
                     wacc = tensor(a[10], "wacc", true);
    at::Tensor lens = tensor(a[9], "new_seqlens", true);
    TORCH_CHECK_VALUE(x[0].dim() == 4, "k must be [B, Hkv, T, d]");
    const int64_t T = x[0].size(2), shape[4] = {c.B, c.Hkv, T, c.d};
    long long strides[2][3];
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "v" : "k";
        TORCH_CHECK_TYPE(x[i].scalar_type() == at::kBFloat16, name, " must be bfloat16");
        TORCH_CHECK_VALUE(x[i].sizes() == at::IntArrayRef(shape) && x[i].device() == c.dev, name, " must be of shape ",
                          at::IntArrayRef(shape), " on ", c.dev);
        TORCH_CHECK_VALUE(x[i].stride(3) == 1 || c.d == 1, name, " must have a dense last dimension");
        // the stride of a dimension of size 1 means nothing
        for (int j = 0; j < 3; ++j) strides[i][j] = shape[j] > 1 ? x[i].stride(j) : 0;
    }
    if (counts.defined()) is(counts, "counts", at::kInt, {c.B}, c.dev);
    if (wacc.defined()) is(wacc, "wacc", at::kFloat, {c.B, c.Hkv, c.mp * c.ps}, c.dev);
    const int t = small(T, "T"), ps = small(c.ps, "page_size"), d = small(c.d, "d");
    int st;
    {
        const NoGil no_gil;
        const c10::cuda::CUDAGuard guard(c.dev);
        if (lens.defined())
            is(lens, "new_seqlens", at::kInt, {c.B}, c.dev);
        else
            lens = fresh({c.B}, at::kInt, c.dev);
        st = g_append(at_(x[0]), at_(x[1]), strides[0], strides[1], at_(c.k), at_(c.v), at_<signed char>(c.kexp),
                      at_<signed char>(c.vexp), at_<int>(c.table), at_<int>(c.seqlens), at_<int>(counts),
                      at_<int>(lens), at_<float>(wacc), (int)c.B, (int)c.Hkv, t, ps, (int)c.mp, (int)c.np, d,
                      PARALLAX_BF16, c.q8 ? PARALLAX_E4M3 : PARALLAX_BF16, stream_of(c.dev));
    }
    if (st) return PyLong_FromLong(st);
    return wrap(lens);
    END_HANDLE_TH_ERRORS
}

// (kpages, vpages, kexp, vexp, block_table, seqlens, wacc, new_table, budget, recent, new_seqlens, kept, new_wacc)
//     -> (new_seqlens, kept, new_wacc)
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 13)) return nullptr;
    const Cache c = cache(a[0], a[1], a[2], a[3], a[4], a[5]);
    const at::Tensor wacc = tensor(a[6], "wacc"), table = tensor(a[7], "new_table");
    at::Tensor lens = tensor(a[10], "new_seqlens", true), kept = tensor(a[11], "kept", true),
               nw = tensor(a[12], "new_wacc", true);
    const long long budget = whole(a[8]), recent = whole(a[9]);
    is(wacc, "wacc", at::kFloat, {c.B, c.Hkv, c.mp * c.ps}, c.dev);
    TORCH_CHECK_VALUE(table.dim() == 2, "new_table must be [B, new_max_pages]");
    const int64_t nmp = table.size(1);
    is(table, "new_table", at::kInt, {c.B, nmp}, c.dev);
    TORCH_CHECK_VALUE(1 <= budget && budget <= nmp * c.ps && 0 <= recent && recent <= budget,
                      "1 <= budget <= new_max_pages * page_size and 0 <= recent <= budget are wanted");
    const int ps = small(c.ps, "page_size"), nmax = small(nmp, "new_max_pages"), d = small(c.d, "d");
    int st;
    {
        const NoGil no_gil;
        const c10::cuda::CUDAGuard guard(c.dev);
        if (lens.defined())
            is(lens, "new_seqlens", at::kInt, {c.B}, c.dev);
        else
            lens = fresh({c.B}, at::kInt, c.dev);
        if (kept.defined())
            is(kept, "kept", at::kInt, {c.B, c.Hkv, (int64_t)budget}, c.dev);
        else
            kept = fresh({c.B, c.Hkv, (int64_t)budget}, at::kInt, c.dev).zero_();
        if (nw.defined())
            is(nw, "new_wacc", at::kFloat, {c.B, c.Hkv, nmp * c.ps}, c.dev);
        else
            nw = fresh({c.B, c.Hkv, nmp * c.ps}, at::kFloat, c.dev).zero_();
        st = g_evict(at_(c.k), at_(c.v), at_<signed char>(c.kexp), at_<signed char>(c.vexp), at_<int>(c.table),
                     at_<int>(c.seqlens), at_<float>(wacc), at_<int>(table), at_<int>(lens), at_<int>(kept),
                     at_<float>(nw), (int)c.B, (int)c.Hkv, ps, (int)c.mp, nmax, (int)c.np, d, (int)budget, (int)recent,
                     c.q8 ? PARALLAX_E4M3 : PARALLAX_BF16, stream_of(c.dev));
    }
    if (st) return PyLong_FromLong(st);
    return tuple({wrap(lens), wrap(kept), wrap(nw)});
    END_HANDLE_TH_ERRORS
}

// addresses of the library's entry points: (decode_paged_q8, decode_paged_acc, kv_append, kv_evict)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 4)) return nullptr;
    void *p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    g_q8 = reinterpret_cast<Q8Fn>(p[0]);
    g_acc = reinterpret_cast<AccFn>(p[1]);
    g_append = reinterpret_cast<AppendFn>(p[2]);
    g_evict = reinterpret_cast<EvictFn>(p[3]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(bind)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(decode)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(append)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__binding() { return PyModule_Create(&module); }
