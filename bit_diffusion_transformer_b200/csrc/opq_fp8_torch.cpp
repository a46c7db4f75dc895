// opq_fp8_torch.cpp — torch tensors to the opq_fp8_* calls of libopq.so: argument checks, outputs,
// the tensors' device and its current stream. No arithmetic happens here. It is a C extension
// rather than ctypes because the 8-bit calls are made per token and per layer: checking up to
// seven tensors and filling the cache structs from Python took 12-37 us per call, several times
// the kernels' own time; here the whole call costs a few microseconds.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <stdexcept>
#include <string>

#include "opq.h"

namespace {

constexpr int64_t kBlock = 128;
PyObject *g_opq_error = nullptr;   // the package's OPQError

// an argument error: becomes ValueError("opq: ...")
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string &msg) { throw Refused("opq: " + msg); }

std::string dims_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

int dtype_code(at::ScalarType t, const char *what) {
    if (t == at::kBFloat16) return OPQ_DTYPE_BF16;
    if (t == at::kHalf) return OPQ_DTYPE_FP16;
    refuse(std::string(what) + " must be bfloat16 or float16");
}

const at::Tensor &tensor(PyObject *o, const char *what, int64_t dim) {
    if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor on a CUDA device");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) refuse(std::string(what) + " must be a tensor on a CUDA device");
    if (t.dim() != dim) refuse(std::string(what) + " must have " + std::to_string(dim) + " dimensions");
    return t;
}
const at::Tensor &tensor(PyObject *o, const char *what, int64_t dim, at::ScalarType type) {
    const at::Tensor &t = tensor(o, what, dim);
    if (t.scalar_type() != type) refuse(std::string(what) + " must be " + at::toString(type));
    return t;
}
void same_device(const at::Tensor &t, const at::Tensor &first, const char *what) {
    if (t.device() != first.device())
        refuse(std::string(what) + " is on " + t.device().str() + ", not " + first.device().str());
}

// row stride of a matrix whose rows are contiguous (one row: its length)
int64_t row_stride(const at::Tensor &t, const char *what, bool written = false) {
    if (t.size(1) > 1 && t.stride(1) != 1) refuse(std::string(what) + ": the last dimension must be contiguous");
    if (t.size(0) <= 1) return t.size(1);
    if (written && t.stride(0) < t.size(1)) refuse(std::string(what) + ": rows overlap");
    return t.stride(0);
}

void contiguous_vector(const at::Tensor &t, int64_t n, const char *what) {
    if (t.size(0) != n || (n > 1 && t.stride(0) != 1))
        refuse(std::string(what) + " must be a contiguous [" + std::to_string(n) + "]");
}

bool overlaps(const at::Tensor &t) {
    for (int64_t i = 0; i < t.dim(); ++i)
        if (t.size(i) > 1 && t.stride(i) == 0) return true;
    return false;
}
// the stride of a dimension with one entry is never used
int64_t stride_of(const at::Tensor &t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

at::ScalarType dtype_arg(PyObject *o) {
    if (!THPDtype_Check(o)) refuse("dtype must be bfloat16 or float16");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// the stream of the call, with the tensors' device made current for its duration
struct OnDevice {
    c10::cuda::CUDAGuard guard;
    void *stream;
    explicit OnDevice(const at::Tensor &t)
        : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()) {}
};

struct Failed {
    opq_status status;
    const char *where;
};
void check(opq_status s, const char *where) {
    if (s != OPQ_OK) throw Failed{s, where};
}

PyObject *raise(const Refused &r) {
    PyErr_SetString(PyExc_ValueError, r.what());
    return nullptr;
}
PyObject *raise(const Failed &f) {
    PyObject *e = g_opq_error ? PyObject_CallFunction(g_opq_error, "is", (int)f.status, f.where) : nullptr;
    if (e) {
        PyErr_SetObject(g_opq_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, f.where);
    }
    return nullptr;
}
// no C++ exception leaves a call
#define OPQ_TRY HANDLE_TH_ERRORS try {
#define OPQ_END                  \
    }                            \
    catch (const Refused &r) {   \
        return raise(r);         \
    }                            \
    catch (const Failed &f) {    \
        return raise(f);         \
    }                            \
    END_HANDLE_TH_ERRORS

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *t = PyTuple_New(2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    return t;
}

int64_t integer(PyObject *o, const char *what) {
    const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
    if (!PyLong_Check(o) || PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(what) + " must be an integer");
    }
    return v;
}

// an uninitialised output, straight from the CUDA allocator: through the dispatcher each one costs
// another third of a microsecond, a tenth of a short call
at::Tensor new_output(at::IntArrayRef size, at::ScalarType type, const at::Tensor &like) {
    return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
}

void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse("wrong number of arguments");
}

// (x, block_rows, out or None) -> (codes, scales)
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    OPQ_TRY
    arity(n, 3);
    const at::Tensor &x = tensor(a[0], "x", 2);
    const int dt = dtype_code(x.scalar_type(), "x");
    const int64_t br = integer(a[1], "block_rows");
    if (br != 1 && br != 128) refuse("block_rows must be 1 or 128");
    const int64_t R = x.size(0), K = x.size(1);
    const int64_t kb = (K + kBlock - 1) / kBlock, rb = (R + br - 1) / br;
    at::Tensor codes, scales;
    if (a[2] == Py_None) {
        codes = new_output({R, K}, at::kFloat8_e4m3fn, x);
        scales = new_output({kb, rb}, at::kFloat, x);
    } else {
        if (!PyTuple_Check(a[2]) && !PyList_Check(a[2])) refuse("out must be (codes, scales)");
        if (PySequence_Fast_GET_SIZE(a[2]) != 2) refuse("out must be (codes, scales)");
        codes = tensor(PySequence_Fast_GET_ITEM(a[2], 0), "codes", 2, at::kFloat8_e4m3fn);
        scales = tensor(PySequence_Fast_GET_ITEM(a[2], 1), "scales", 2, at::kFloat);
        same_device(codes, x, "codes");
        same_device(scales, x, "scales");
        if (codes.sizes() != x.sizes() || scales.size(0) != kb || scales.size(1) != rb)
            refuse("out must be codes " + dims_text(x.sizes()) + " and scales " + dims_text({kb, rb}));
    }
    const int64_t ldx = row_stride(x, "x"), ldc = row_stride(codes, "codes", true), lds = row_stride(scales, "scales", true);
    OnDevice on(x);
    check(opq_fp8_quantize(x.data_ptr(), dt, R, K, ldx, br, static_cast<uint8_t *>(codes.data_ptr()), ldc,
                           static_cast<float *>(scales.data_ptr()), lds, on.stream),
          "opq_fp8_quantize");
    return pair(codes, scales);
    OPQ_END
}

// (x, x_scales, w, w_scales, bias or None, activation code, dtype, out or None) -> y
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    OPQ_TRY
    arity(n, 8);
    const at::Tensor &x = tensor(a[0], "x", 2, at::kFloat8_e4m3fn);
    const at::Tensor &xs = tensor(a[1], "x_scales", 2, at::kFloat);
    const at::Tensor &w = tensor(a[2], "w", 2, at::kFloat8_e4m3fn);
    const at::Tensor &ws = tensor(a[3], "w_scales", 2, at::kFloat);
    same_device(xs, x, "x_scales");
    same_device(w, x, "w");
    same_device(ws, x, "w_scales");
    const int64_t act = integer(a[5], "act");
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
    const int64_t kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
    if (w.size(1) != K) refuse("x has " + std::to_string(K) + " columns, w " + std::to_string(w.size(1)));
    if (xs.size(0) != kb || xs.size(1) != M)
        refuse("x_scales must be " + dims_text({kb, M}) + " (fp8_quantize with block_rows = 1)");
    if (ws.size(0) != kb || ws.size(1) != nb)
        refuse("w_scales must be " + dims_text({kb, nb}) + " (fp8_quantize with block_rows = 128)");
    at::Tensor y;
    at::ScalarType type;
    if (a[7] == Py_None) {
        type = dtype_arg(a[6]);
        dtype_code(type, "dtype");
        y = new_output({M, N}, type, x);
    } else {
        y = tensor(a[7], "out", 2);
        type = y.scalar_type();
        same_device(y, x, "out");
        if (y.size(0) != M || y.size(1) != N) refuse("out must be " + dims_text({M, N}));
    }
    const int dt = dtype_code(type, "out");
    const void *bias = nullptr;
    if (a[4] != Py_None) {
        const at::Tensor &b = tensor(a[4], "bias", 1, type);
        same_device(b, x, "bias");
        contiguous_vector(b, N, "bias");
        bias = b.data_ptr();
    }
    const int64_t ldx = row_stride(x, "x"), ldxs = row_stride(xs, "x_scales"), ldw = row_stride(w, "w"),
                  ldws = row_stride(ws, "w_scales"), ldy = row_stride(y, "out", true);
    OnDevice on(x);
    check(opq_fp8_linear(static_cast<const uint8_t *>(x.data_ptr()), ldx, static_cast<const float *>(xs.data_ptr()), ldxs,
                         M, K, static_cast<const uint8_t *>(w.data_ptr()), ldw, static_cast<const float *>(ws.data_ptr()),
                         ldws, N, bias, (int32_t)act, y.data_ptr(), dt, ldy, on.stream),
          "opq_fp8_linear");
    return THPVariable_Wrap(y);
    OPQ_END
}

struct Cache {
    opq_fp8_cache side[2];
    at::Tensor first;
    int n = 0;
    int64_t pages = 0, page = 0, heads = 0;
};

Cache read_cache(PyObject *o) {
    if (!PyTuple_Check(o) && !PyList_Check(o)) refuse("cache must be (codes, scales) or (k_codes, k_scales, v_codes, v_scales)");
    const Py_ssize_t len = PySequence_Fast_GET_SIZE(o);
    if (len != 2 && len != 4) refuse("cache must be (codes, scales) or (k_codes, k_scales, v_codes, v_scales)");
    Cache c;
    c.n = (int)len / 2;
    for (int i = 0; i < c.n; ++i) {
        const at::Tensor &codes = tensor(PySequence_Fast_GET_ITEM(o, 2 * i), "cache codes", 4, at::kFloat8_e4m3fn);
        const at::Tensor &scales = tensor(PySequence_Fast_GET_ITEM(o, 2 * i + 1), "cache scales", 4, at::kFloat);
        if (i == 0) {
            c.first = codes;
            c.pages = codes.size(0);
            c.page = codes.size(1);
            c.heads = codes.size(2);
        }
        same_device(codes, c.first, "cache codes");
        same_device(scales, c.first, "cache scales");
        const int64_t D = codes.size(3), nb = (D + kBlock - 1) / kBlock;
        if (codes.size(0) != c.pages || codes.size(1) != c.page || codes.size(2) != c.heads)
            refuse("keys and values must have the same pages, page size and heads");
        if (scales.size(0) != c.pages || scales.size(1) != c.page || scales.size(2) != c.heads || scales.size(3) != nb)
            refuse("scales must be " + dims_text({c.pages, c.page, c.heads, nb}));
        if ((D > 1 && codes.stride(3) != 1) || (nb > 1 && scales.stride(3) != 1))
            refuse("cache: the last dimension must be contiguous");
        if (overlaps(codes) || overlaps(scales)) refuse("cache: elements overlap");
        c.side[i] = {static_cast<uint8_t *>(codes.data_ptr()), static_cast<float *>(scales.data_ptr()), D,
                     stride_of(codes, 0), stride_of(codes, 1), stride_of(codes, 2),
                     stride_of(scales, 0), stride_of(scales, 1), stride_of(scales, 2)};
    }
    return c;
}

opq_rows make_rows(const at::Tensor &t, const Cache &c, int i, int64_t tokens, at::ScalarType type, const char *what,
                   bool written) {
    if (t.scalar_type() != type) refuse(std::string(what) + " must be of one type");
    same_device(t, c.first, what);
    if (t.size(0) != tokens || t.size(1) != c.heads || t.size(2) != c.side[i].head_dim)
        refuse(std::string(what) + " must be " + dims_text({tokens, c.heads, c.side[i].head_dim}));
    if (t.size(2) > 1 && t.stride(2) != 1) refuse(std::string(what) + ": the last dimension must be contiguous");
    if (written && overlaps(t)) refuse(std::string(what) + ": elements overlap");
    return {t.data_ptr(), stride_of(t, 0), stride_of(t, 1)};
}

// (k, v or None, cache, slots) -> None
PyObject *cache_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    OPQ_TRY
    arity(n, 4);
    const Cache c = read_cache(a[2]);
    if ((a[1] == Py_None ? 1 : 2) != c.n) refuse("values go with a cache of keys and values");
    const at::Tensor &k = tensor(a[0], "k", 3);
    const int dt = dtype_code(k.scalar_type(), "k");
    const int64_t T = k.size(0);
    opq_rows rows[2];
    for (int i = 0; i < c.n; ++i)
        rows[i] = make_rows(i ? tensor(a[1], "v", 3) : k, c, i, T, k.scalar_type(), i ? "v" : "k", false);
    const at::Tensor &slots = tensor(a[3], "slots", 1, at::kLong);
    same_device(slots, c.first, "slots");
    contiguous_vector(slots, T, "slots");
    OnDevice on(c.first);
    check(opq_fp8_cache_write(c.side, rows, c.n, c.pages, c.page, c.heads, dt, T,
                              static_cast<const int64_t *>(slots.data_ptr()), on.stream),
          "opq_fp8_cache_write");
    Py_RETURN_NONE;
    OPQ_END
}

// (cache, page_table, cu_rows, rows or None, starts or None, dtype, out or None) -> (k[, v])
PyObject *cache_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    OPQ_TRY
    arity(n, 7);
    const Cache c = read_cache(a[0]);
    const at::Tensor &table = tensor(a[1], "page_table", 2, at::kInt);
    const at::Tensor &cu = tensor(a[2], "cu_rows", 1, at::kInt);
    same_device(table, c.first, "page_table");
    same_device(cu, c.first, "cu_rows");
    const int64_t B = table.size(0), W = table.size(1);
    const int64_t ld = row_stride(table, "page_table");
    contiguous_vector(cu, B + 1, "cu_rows");
    const int32_t *starts = nullptr;
    if (a[4] != Py_None) {
        const at::Tensor &s = tensor(a[4], "starts", 1, at::kInt);
        same_device(s, c.first, "starts");
        contiguous_vector(s, B, "starts");
        starts = static_cast<const int32_t *>(s.data_ptr());
    }
    at::Tensor out[2];
    if (a[6] == Py_None) {
        if (a[3] == Py_None) refuse("rows (the number of output rows) or out is needed");
        const int64_t rows = integer(a[3], "rows");
        if (rows < 0) refuse("rows must not be negative");
        const at::ScalarType type = dtype_arg(a[5]);
        dtype_code(type, "dtype");
        for (int i = 0; i < c.n; ++i)
            out[i] = new_output({rows, c.heads, c.side[i].head_dim}, type, c.first);
    } else {
        if ((!PyTuple_Check(a[6]) && !PyList_Check(a[6])) || PySequence_Fast_GET_SIZE(a[6]) != c.n)
            refuse("out must hold " + std::to_string(c.n) + " tensors");
        for (int i = 0; i < c.n; ++i) out[i] = tensor(PySequence_Fast_GET_ITEM(a[6], i), "out", 3);
        if (a[3] != Py_None && integer(a[3], "rows") != out[0].size(0))
            refuse("out has " + std::to_string(out[0].size(0)) + " rows");
    }
    const at::ScalarType type = out[0].scalar_type();
    const int dt = dtype_code(type, "out");
    const int64_t rows = out[0].size(0);
    opq_rows orows[2];
    for (int i = 0; i < c.n; ++i) orows[i] = make_rows(out[i], c, i, rows, type, "out", true);
    OnDevice on(c.first);
    check(opq_fp8_cache_read(c.side, orows, c.n, c.pages, c.page, c.heads, dt, rows,
                             static_cast<const int32_t *>(cu.data_ptr()), B,
                             static_cast<const int32_t *>(table.data_ptr()), ld, W, starts, on.stream),
          "opq_fp8_cache_read");
    if (c.n == 2) return pair(out[0], out[1]);
    PyObject *t = PyTuple_New(1);
    if (t) PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(out[0]));
    return t;
    OPQ_END
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_XINCREF(cls);
    Py_XSETREF(g_opq_error, cls);
    Py_RETURN_NONE;
}

#define FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"quantize", FASTCALL(quantize), nullptr},
                           {"linear", FASTCALL(linear), nullptr},
                           {"cache_write", FASTCALL(cache_write), nullptr},
                           {"cache_read", FASTCALL(cache_read), nullptr},
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8(void) {
    PyObject *m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
