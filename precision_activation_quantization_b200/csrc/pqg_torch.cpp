// Tensor binding of the norm and cache entry points: argument checks, outputs
// and the call of the C ABI in one native function each.
//
// A decode step calls these with a few microseconds of device work; marshalling
// a call in Python costs more than that (about 26 us for the norm, against 6
// here).  The C ABI stays the boundary: its functions are looked up in the
// library that pqg.py loaded, and this module holds no arithmetic.
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>

#include "pqg.h"

namespace {

struct Library {
    decltype(&pqg_rmsnorm_quant) rmsnorm_quant;
    decltype(&pqg_scales_bytes) scales_bytes;
    decltype(&pqg_kv_write) kv_write;
    decltype(&pqg_kv_read) kv_read;
    decltype(&pqg_kv_attention) kv_attention;
    decltype(&pqg_kv_attention_workspace) kv_attention_workspace;
} lib;

template <typename F>
void find(void *handle, const char *name, F *function) {
    *function = reinterpret_cast<F>(dlsym(handle, name));
    TORCH_CHECK(*function != nullptr, "the library exports no ", name);
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}
int64_t integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_TYPE(false, name, " must be an integer that fits 64 bits");
    }
    return v;
}
double number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_TYPE(false, name, " must be a number");
    }
    return v;
}

bool half_type(const at::Tensor &t) {
    return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf;
}
int dtype_of(const at::Tensor &t) { return t.scalar_type() == at::kBFloat16 ? PQG_BF16 : PQG_FP16; }

void check_float(const at::Tensor &t, const char *name) {
    TORCH_CHECK_TYPE(half_type(t), "unsupported dtype ", t.scalar_type(), " of ", name);
}
// A dense tensor of this type and size on this device.
void check_like(const at::Tensor &t, at::ScalarType type, int64_t numel, at::Device device,
                const char *name) {
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.numel() == numel && t.device() == device &&
                          t.is_contiguous(),
                      name, " must be a contiguous ", type, " tensor of ", numel, " entries on ",
                      device);
}
void check_shape(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape,
                 at::Device device, const char *name) {
    TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == type && t.device() == device &&
                          t.is_contiguous(),
                      name, " must be a contiguous ", type, " tensor ", shape, " on ", device);
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    return at::Tensor(at::detail::empty_cuda(shape, type, device, c10::nullopt));
}

// The stream of a call: a handle, or torch's current one for None.
pqg_stream_t stream_of(PyObject *o, at::Device device) {
    if (o == Py_None)
        return reinterpret_cast<pqg_stream_t>(
            at::cuda::getCurrentCUDAStream(device.index()).stream());
    return reinterpret_cast<pqg_stream_t>(static_cast<uintptr_t>(integer(o, "stream")));
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

// (status, entry point, tensors...); steals the references it is given.
PyObject *result(int64_t status, const char *where, std::initializer_list<PyObject *> items) {
    PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(items.size()) + 2);
    PyTuple_SET_ITEM(r, 0, PyLong_FromLongLong(status));
    PyTuple_SET_ITEM(r, 1, PyUnicode_FromString(where));
    Py_ssize_t i = 2;
    for (PyObject *o : items) PyTuple_SET_ITEM(r, i++, o);
    return r;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// rmsnorm_quant(x, weight, residual, out, scales, residual_out, eps, group, out_dtype,
//               scale_fmt, layout, global_scale, stream)
PyObject *py_rmsnorm_quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 13)) return nullptr;
    const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    check_float(x, "x");
    TORCH_CHECK_VALUE(x.is_cuda() && x.is_contiguous() && x.dim() >= 2,
                      "x must be a contiguous CUDA tensor of rows");
    const at::Device device = x.device();
    const at::ScalarType type = x.scalar_type();
    const int64_t K = x.size(-1), M = K > 0 ? x.numel() / K : 0;
    check_like(weight, type, K, device, "weight");
    at::Tensor residual_out;
    const void *residual = nullptr;
    if (a[2] == Py_None) {
        TORCH_CHECK_VALUE(a[5] == Py_None, "residual_out needs a residual: without one h is x");
    } else {
        const at::Tensor &r = tensor(a[2], "residual");
        check_like(r, type, x.numel(), device, "residual");
        residual = r.data_ptr();
        if (a[5] != Py_None) {
            residual_out = tensor(a[5], "residual_out");
            check_like(residual_out, type, x.numel(), device, "residual_out");
        } else {
            residual_out = empty(x.sizes(), type, device);
        }
    }
    const double eps = number(a[6], "eps");
    const int64_t group = integer(a[7], "group");
    const int out_dtype = static_cast<int>(integer(a[8], "out_dtype"));
    const int scale_fmt = static_cast<int>(integer(a[9], "scale_fmt"));
    const int layout = static_cast<int>(integer(a[10], "layout"));
    TORCH_CHECK_VALUE(group > 0 && group <= INT32_MAX, "group must be positive");
    const int64_t bytes =
        lib.scales_bytes(1, M, K, static_cast<int>(group), scale_fmt, layout);
    if (bytes < 0) return result(bytes, "pqg_scales_bytes", {});

    const int64_t row = out_dtype == PQG_E2M1 ? K / 2 : K;
    at::Tensor out, scales;
    if (a[3] != Py_None) {
        out = tensor(a[3], "out");
        TORCH_CHECK_VALUE(static_cast<int64_t>(out.nbytes()) == M * row && out.is_contiguous() &&
                              out.device() == device,
                          "out must be a contiguous buffer of ", M * row, " bytes on x's device");
    } else {
        out = empty({M, row}, out_dtype == PQG_E4M3 ? at::kFloat8_e4m3fn
                              : out_dtype == PQG_INT8 ? at::kChar : at::kByte, device);
    }
    if (a[4] != Py_None) {
        scales = tensor(a[4], "scales");
        TORCH_CHECK_VALUE(static_cast<int64_t>(scales.nbytes()) == bytes &&
                              scales.is_contiguous() && scales.device() == device,
                          "scales must be a contiguous buffer of ", bytes, " bytes on x's device");
    } else {
        const int64_t ng = K / group, mpad = (M + 3) / 4 * 4;
        const at::ScalarType st = scale_fmt == PQG_SCALE_FP32 ? at::kFloat : at::kByte;
        scales = layout == PQG_ROW_MAJOR       ? empty({M, ng}, st, device)
                 : layout == PQG_COL_MAJOR_TMA ? empty({ng, mpad}, st, device)
                 : layout == PQG_UE8M0_PACKED  ? empty({(ng + 3) / 4, mpad}, at::kInt, device)
                                               : empty({bytes}, at::kByte, device);
    }
    const float *g = nullptr;
    if (scale_fmt == PQG_SCALE_E4M3) {
        TORCH_CHECK_VALUE(a[11] != Py_None,
                          "NVFP4 needs global_scale: a one-element fp32 tensor on x's device");
        const at::Tensor &gs = tensor(a[11], "global_scale");
        check_like(gs, at::kFloat, 1, device, "global_scale");
        g = static_cast<const float *>(gs.data_ptr());
    }
    const c10::cuda::CUDAGuard guard(device);
    const int status = lib.rmsnorm_quant(
        x.data_ptr(), residual, weight.data_ptr(),
        residual != nullptr ? residual_out.data_ptr() : nullptr, out.data_ptr(), scales.data_ptr(),
        g, M, K, static_cast<int>(group), eps, dtype_of(x), out_dtype, scale_fmt, layout,
        stream_of(a[12], device));
    if (status != PQG_OK) return result(status, "pqg_rmsnorm_quant", {});
    return result(status, "", {wrap(out), wrap(scales),
                               residual != nullptr ? wrap(residual_out) : wrap(x)});
    END_HANDLE_TH_ERRORS
}

// ---- the cache ----------------------------------------------------------------

// The description a KVCache holds, and its device.
struct Cache {
    const pqg_kv_cache *c;
    at::Device device;
    Cache(PyObject *address, PyObject *index)
        : c(reinterpret_cast<const pqg_kv_cache *>(
              static_cast<uintptr_t>(integer(address, "cache")))),
          device(at::kCUDA, static_cast<c10::DeviceIndex>(integer(index, "device"))) {}
};

// Elements between the tokens of a [T, heads, head_dim] tensor with dense heads.
int64_t token_stride(const at::Tensor &t, int64_t heads, const Cache &cache, const char *name) {
    const int64_t dim = cache.c->head_dim;
    TORCH_CHECK_VALUE(t.dim() == 3 && t.size(1) == heads && t.size(2) == dim, name,
                      " must be [tokens, ", heads, ", ", dim, "], got ", t.sizes());
    check_float(t, name);
    TORCH_CHECK_VALUE(t.device() == cache.device, name, " must be on the cache's device");
    TORCH_CHECK_VALUE(t.stride(2) == 1 && (heads == 1 || t.stride(1) == dim),
                      "the heads of a token of ", name, " must be dense");
    return t.size(0) > 1 ? t.stride(0) : heads * dim;
}

const int32_t *indexes(const at::Tensor &t, int64_t numel, const Cache &cache, const char *name) {
    check_like(t, at::kInt, numel, cache.device, name);
    return static_cast<const int32_t *>(t.data_ptr());
}

struct Table {
    const int32_t *p;
    int64_t rows, width, stride;
    Table(const at::Tensor &t, const Cache &cache) {
        TORCH_CHECK_VALUE(t.dim() == 2 && t.scalar_type() == at::kInt &&
                              t.device() == cache.device && t.size(1) >= 1 &&
                              (t.size(1) == 1 || t.stride(1) == 1),
                          "page_table must be an int32 tensor [sequences, pages] on the cache's "
                          "device with dense rows");
        p = static_cast<const int32_t *>(t.data_ptr());
        rows = t.size(0);
        width = t.size(1);
        stride = rows > 1 ? t.stride(0) : width;
    }
};

// kv_write(cache, device, k, v, slots, stream)
PyObject *py_kv_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 6)) return nullptr;
    const Cache cache(a[0], a[1]);
    const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    const int64_t ks = token_stride(k, cache.c->kv_heads, cache, "k");
    const int64_t vs = token_stride(v, cache.c->kv_heads, cache, "v");
    const int64_t T = k.size(0);
    TORCH_CHECK_VALUE(v.size(0) == T && v.scalar_type() == k.scalar_type(),
                      "k and v must hold the same tokens in the same dtype");
    const int32_t *slots = indexes(tensor(a[4], "slots"), T, cache, "slots");
    const c10::cuda::CUDAGuard guard(cache.device);
    const int status = lib.kv_write(cache.c, k.data_ptr(), v.data_ptr(), slots, T, ks, vs,
                                    dtype_of(k), stream_of(a[5], cache.device));
    return result(status, "pqg_kv_write", {});
    END_HANDLE_TH_ERRORS
}

// kv_read(cache, device, page_table, indptr, num_tokens, dtype, k_out, v_out, stream);
// dtype: PQG_BF16, PQG_FP16 or None
PyObject *py_kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 9)) return nullptr;
    const Cache cache(a[0], a[1]);
    const Table table(tensor(a[2], "page_table"), cache);
    const int32_t *indptr = indexes(tensor(a[3], "indptr"), table.rows + 1, cache, "indptr");
    const int64_t M = integer(a[4], "num_tokens");
    TORCH_CHECK_VALUE(M >= 0, "num_tokens must not be negative");
    const int64_t shape[] = {M, cache.c->kv_heads, cache.c->head_dim};
    at::ScalarType type = a[5] != Py_None && integer(a[5], "dtype") == PQG_FP16 ? at::kHalf
                                                                                : at::kBFloat16;
    for (const int i : {6, 7})
        if (a[i] != Py_None) {
            const at::Tensor &t = tensor(a[i], "an output");
            check_float(t, "an output");
            TORCH_CHECK_VALUE(a[5] == Py_None || t.scalar_type() == type,
                              "dtype differs from the given output's");
            type = t.scalar_type();
        }
    at::Tensor out[2];
    for (const int i : {0, 1}) {
        if (a[6 + i] == Py_None) {
            out[i] = empty(shape, type, cache.device);
        } else {
            out[i] = tensor(a[6 + i], "an output");
            check_shape(out[i], type, shape, cache.device, i == 0 ? "k_out" : "v_out");
        }
    }
    const c10::cuda::CUDAGuard guard(cache.device);
    const int status =
        lib.kv_read(cache.c, table.p, table.stride, table.width, indptr, table.rows,
                    out[0].data_ptr(), out[1].data_ptr(), M,
                    type == at::kBFloat16 ? PQG_BF16 : PQG_FP16, stream_of(a[8], cache.device));
    if (status != PQG_OK) return result(status, "pqg_kv_read", {});
    return result(status, "", {wrap(out[0]), wrap(out[1])});
    END_HANDLE_TH_ERRORS
}

// kv_attention(cache, device, q, page_table, seq_lens, sm_scale, max_len, out, lse,
//              return_lse, stream)
PyObject *py_kv_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 11)) return nullptr;
    const Cache cache(a[0], a[1]);
    const Table table(tensor(a[3], "page_table"), cache);
    const at::Tensor &q = tensor(a[2], "q");
    TORCH_CHECK_VALUE(q.dim() == 3 && q.size(1) >= 1 && q.size(1) % cache.c->kv_heads == 0,
                      "q must be [tokens, heads, head_dim] with a multiple of the cache's heads");
    const int64_t T = q.size(0), heads = q.size(1), B = table.rows;
    const int64_t stride = token_stride(q, heads, cache, "q");
    const int32_t *lens = indexes(tensor(a[4], "seq_lens"), B, cache, "seq_lens");
    TORCH_CHECK_VALUE(B > 0 ? T % B == 0 && T >= B : T == 0,
                      "q must hold the same number of tokens of each sequence, at least one");
    const int64_t q_len = B > 0 ? T / B : 1;
    const double sm_scale = number(a[5], "sm_scale");
    const int64_t max_len = integer(a[6], "max_len");
    const c10::cuda::CUDAGuard guard(cache.device);   // the scratch goes by the current device
    const int64_t bytes =
        lib.kv_attention_workspace(cache.c, table.width, B, q_len, heads, max_len);
    if (bytes < 0) return result(bytes, "pqg_kv_attention_workspace", {});
    at::Tensor out, lse, work;
    if (a[7] != Py_None) {
        out = tensor(a[7], "out");
        check_shape(out, q.scalar_type(), q.sizes(), cache.device, "out");
    } else {
        out = empty(q.sizes(), q.scalar_type(), cache.device);
    }
    if (a[8] != Py_None) {
        lse = tensor(a[8], "lse");
        check_shape(lse, at::kFloat, {T, heads}, cache.device, "lse");
    } else if (a[9] == Py_True) {
        lse = empty({T, heads}, at::kFloat, cache.device);
    }
    if (bytes > 0) work = empty({bytes}, at::kByte, cache.device);
    const int status = lib.kv_attention(
        cache.c, q.data_ptr(), stride, table.p, table.stride, table.width, lens, B, q_len, heads,
        static_cast<float>(sm_scale), max_len, out.data_ptr(),
        lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr,
        bytes > 0 ? work.data_ptr() : nullptr, bytes, dtype_of(q), stream_of(a[10], cache.device));
    if (status != PQG_OK) return result(status, "pqg_kv_attention", {});
    if (!lse.defined()) return result(status, "", {wrap(out)});
    return result(status, "", {wrap(out), wrap(lse)});
    END_HANDLE_TH_ERRORS
}

// load(path): the library the entry points are taken from.
PyObject *py_load(PyObject *, PyObject *path) {
    HANDLE_TH_ERRORS
    const char *name = PyUnicode_AsUTF8(path);
    if (name == nullptr) return nullptr;
    void *handle = dlopen(name, RTLD_NOW | RTLD_LOCAL);
    TORCH_CHECK(handle != nullptr, "cannot load ", name, ": ", dlerror());
    find(handle, "pqg_rmsnorm_quant", &lib.rmsnorm_quant);
    find(handle, "pqg_scales_bytes", &lib.scales_bytes);
    find(handle, "pqg_kv_write", &lib.kv_write);
    find(handle, "pqg_kv_read", &lib.kv_read);
    find(handle, "pqg_kv_attention", &lib.kv_attention);
    find(handle, "pqg_kv_attention_workspace", &lib.kv_attention_workspace);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"load", py_load, METH_O, nullptr},
    {"rmsnorm_quant", fast(py_rmsnorm_quant), METH_FASTCALL, nullptr},
    {"kv_write", fast(py_kv_write), METH_FASTCALL, nullptr},
    {"kv_read", fast(py_kv_read), METH_FASTCALL, nullptr},
    {"kv_attention", fast(py_kv_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pqg_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pqg_torch(void) { return PyModule_Create(&module); }
