// The torch side of the attention and 8-bit calls: argument checks, output and
// scratch allocation, the current stream, then the C ABI call. The same marshalling
// as the ctypes binding, compiled because a serving step makes many short calls: a
// call takes the host 5 to 7 us here and took 10 to 15 us in Python.
//
// A wrong argument raises ValueError; a refusal of the C ABI comes back as the
// status number, which the Python side turns into its exception.
#include <Python.h>
#include <dlfcn.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <bitlinear.h>

#include <algorithm>
#include <cmath>
#include <sstream>
#include <stdexcept>
#include <string>

namespace {

struct Calls {
    decltype(&bitlinear_workspace_bytes) workspace_bytes;
    decltype(&bitlinear_kv4_append) kv4_append;
    decltype(&bitlinear_kv4_read) kv4_read;
    decltype(&bitlinear_kv4_attention) kv4_attention;
    decltype(&bitlinear_forward_int8) forward_int8;
} lib;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

std::string shape_text(at::IntArrayRef s) {
    std::ostringstream o;
    o << s;
    return o.str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    return t;
}

// A contiguous tensor of this type, shape and device.
void expect(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device device) {
    if (t.scalar_type() == type && t.sizes() == shape && t.device() == device && t.is_contiguous()) return;
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor " + shape_text(shape) + " on " +
           device.str() + ", got " + c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()) + " on " + t.device().str());
}

// Row stride of t [M, heads, D] bf16 with the heads of a row side by side.
int64_t rows(const at::Tensor& t, const char* name, int64_t M, int64_t heads, int64_t D, c10::Device device) {
    if (t.scalar_type() != at::kBFloat16 || t.device() != device || t.sizes() != at::IntArrayRef({M, heads, D}))
        refuse(std::string(name) + " must be a BFloat16 tensor " + shape_text({M, heads, D}) + " on " + device.str() + ", got " +
               c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()) + " on " + t.device().str());
    if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D)) refuse(std::string(name) + " must have the heads of a row side by side");
    return M > 1 ? t.stride(0) : heads * D;  // the stride of a single row means nothing
}

struct Cache {
    bl_kv4_cache c;
    c10::Device device{c10::kCUDA, 0};
};

// a[0 .. 3]: k_codes, k_steps, v_codes, v_steps
Cache cache_of(PyObject* const* a) {
    const at::Tensor &kc = tensor(a[0], "k_codes"), &ks = tensor(a[1], "k_steps"), &vc = tensor(a[2], "v_codes"), &vs = tensor(a[3], "v_steps");
    if (kc.dim() != 4) refuse("codes must be [num_pages, kv_heads, page_size, head_dim / 2]");
    const int64_t pages = kc.size(0), heads = kc.size(1), size = kc.size(2), half = kc.size(3);
    const c10::Device dev = kc.device();
    expect(kc, "k_codes", at::kByte, {pages, heads, size, half}, dev);
    expect(vc, "v_codes", at::kByte, {pages, heads, size, half}, dev);
    expect(ks, "k_steps", at::kBFloat16, {pages, heads, size, 2 * half / 32}, dev);
    expect(vs, "v_steps", at::kBFloat16, {pages, heads, size, 2 * half / 32}, dev);
    if (heads > INT32_MAX || size > INT32_MAX || half > INT32_MAX / 2) refuse("the cache is too large");
    return {{(uint8_t*)kc.data_ptr(), (uint16_t*)ks.data_ptr(), (uint8_t*)vc.data_ptr(), (uint16_t*)vs.data_ptr(), pages, (int32_t)size,
             (int32_t)heads, (int32_t)(2 * half)},
            dev};
}

// a[0 .. 2]: page_table, kv_len, q_start
bl_kv4_batch batch_of(PyObject* const* a, c10::Device dev) {
    const at::Tensor &table = tensor(a[0], "page_table"), &len = tensor(a[1], "kv_len"), &start = tensor(a[2], "q_start");
    if (table.scalar_type() != at::kInt || table.device() != dev || table.dim() != 2) refuse("page_table must be an int32 tensor [S, W] on " + dev.str());
    const int64_t S = table.size(0), W = table.size(1);
    if (table.stride(1) != 1 && W > 1) refuse("page_table must have contiguous rows");
    expect(len, "kv_len", at::kInt, {S}, dev);
    expect(start, "q_start", at::kInt, {S + 1}, dev);
    if (S > INT32_MAX || W > INT32_MAX) refuse("page_table is too large");
    return {(const int32_t*)start.data_ptr(), (const int32_t*)len.data_ptr(), (const int32_t*)table.data_ptr(), table.stride(0), (int32_t)S, (int32_t)W};
}

int64_t whole(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be a whole number");
    }
    return v;
}

bl_stream_t stream(c10::Device dev) { return (bl_stream_t)c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

const uint16_t* bits(const at::Tensor& t) { return (const uint16_t*)t.data_ptr(); }

// C++ exceptions (wrong arguments, and torch's, such as an allocation that fails) become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

// bind(path): take the calls from the shared library
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 1, [&]() -> PyObject* {
        const char* path = PyUnicode_AsUTF8(a[0]);
        if (!path) return nullptr;
        void* h = dlopen(path, RTLD_NOW);
        if (!h) throw std::runtime_error(dlerror());
        auto get = [&](auto& f, const char* name) {
            f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
            if (!f) throw std::runtime_error(std::string(path) + " has no " + name);
        };
        get(lib.workspace_bytes, "bitlinear_workspace_bytes");
        get(lib.kv4_append, "bitlinear_kv4_append");
        get(lib.kv4_read, "bitlinear_kv4_read");
        get(lib.kv4_attention, "bitlinear_kv4_attention");
        get(lib.forward_int8, "bitlinear_forward_int8");
        Py_RETURN_NONE;
    });
}

// kv4_check(k_codes, k_steps, v_codes, v_steps) -> (kv_heads, head_dim)
PyObject* kv4_check(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        const Cache c = cache_of(a);
        return Py_BuildValue("(ii)", c.c.kv_heads, c.c.head_dim);
    });
}

// kv4_append(q, k, v, cos_sin, cache x 4, page_table, kv_len, q_start, interleaved, out)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &cs = tensor(a[3], "cos_sin");
        const Cache c = cache_of(a + 4);
        const bl_kv4_batch b = batch_of(a + 8, c.device);
        const int64_t D = c.c.head_dim, hkv = c.c.kv_heads;
        if (q.dim() != 3) refuse("q must be [M, heads, D]");
        const int64_t M = q.size(0), Hq = q.size(1);
        int64_t qs = rows(q, "q", M, Hq, D, c.device);
        const int64_t ks = rows(k, "k", M, hkv, D, c.device), vs = rows(v, "v", M, hkv, D, c.device);
        if (cs.dim() != 2) refuse("cos_sin must be [max_pos, D]");
        expect(cs, "cos_sin", at::kFloat, {cs.size(0), D}, c.device);
        const int interleaved = PyObject_IsTrue(a[11]);
        if (interleaved < 0) return nullptr;
        const c10::cuda::CUDAGuard guard(c.device);
        at::Tensor out = a[12] == Py_None ? at::empty({M, Hq, D}, q.options()) : tensor(a[12], "out");
        const int64_t os = rows(out, "out", M, Hq, D, c.device);
        const bl_status st = lib.kv4_append(bits(q), qs, bits(k), ks, bits(v), vs, M, (int32_t)Hq, (const float*)cs.data_ptr(), cs.size(0),
                                            interleaved, &c.c, &b, (uint16_t*)out.data_ptr(), os, stream(c.device));
        return st ? PyLong_FromLong(st) : wrap(out);
    });
}

// kv4_read(cache x 4, page_table, kv_len, q_start, rows)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const Cache c = cache_of(a);
        const bl_kv4_batch b = batch_of(a + 4, c.device);
        const int64_t M = whole(a[7], "rows");
        if (M < 0) refuse("rows must not be negative");
        const c10::cuda::CUDAGuard guard(c.device);
        const auto options = at::TensorOptions().dtype(at::kBFloat16).device(c.device);
        at::Tensor k = at::empty({M, c.c.kv_heads, c.c.head_dim}, options), v = at::empty({M, c.c.kv_heads, c.c.head_dim}, options);
        const bl_status st = lib.kv4_read(&c.c, &b, M, (uint16_t*)k.data_ptr(), (uint16_t*)v.data_ptr(), stream(c.device));
        if (st) return PyLong_FromLong(st);
        PyObject *pk = wrap(k), *pv = wrap(v), *both = PyTuple_Pack(2, pk, pv);
        Py_XDECREF(pk);
        Py_XDECREF(pv);
        return both;
    });
}

// kv4_attention(q, cache x 4, page_table, kv_len, q_start, max_q, scale, out, ws)
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const Cache c = cache_of(a + 1);
        const bl_kv4_batch b = batch_of(a + 5, c.device);
        const int64_t D = c.c.head_dim;
        if (q.dim() != 3) refuse("q must be [M, heads, D]");
        const int64_t M = q.size(0), Hq = q.size(1);
        const int64_t qs = rows(q, "q", M, Hq, D, c.device);
        const int64_t max_q = whole(a[8], "max_q");
        double scale = 1.0 / std::sqrt((double)D);
        if (a[9] != Py_None) {
            scale = PyFloat_AsDouble(a[9]);
            if (scale == -1.0 && PyErr_Occurred()) return nullptr;
        }
        const c10::cuda::CUDAGuard guard(c.device);
        at::Tensor out = a[10] == Py_None ? at::empty({M, Hq, D}, q.options()) : tensor(a[10], "out");
        const int64_t os = rows(out, "out", M, Hq, D, c.device);
        at::Tensor ws = a[11] == Py_None
                            ? at::empty({(int64_t)lib.workspace_bytes(BL_OP_KV4_ATTENTION, std::max<int64_t>(0, std::min(max_q, M)),
                                                                      c.c.kv_heads ? Hq / c.c.kv_heads : 0, D)},
                                        at::TensorOptions().dtype(at::kByte).device(c.device))
                            : tensor(a[11], "ws");
        if (ws.device() != c.device || !ws.is_contiguous()) refuse("ws must be contiguous, on " + c.device.str());
        const bl_status st = lib.kv4_attention(bits(q), qs, M, (int32_t)Hq, max_q, (float)scale, &c.c, &b, (uint16_t*)out.data_ptr(), os,
                                               ws.data_ptr(), ws.nbytes(), stream(c.device));
        return st ? PyLong_FromLong(st) : wrap(out);
    });
}

// forward_int8(Wq, wstep, x, rmsnorm, residual, want_acc, fp32, out, ws)
PyObject* forward_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const at::Tensor &W = tensor(a[0], "Wq"), &step = tensor(a[1], "wstep"), &x = tensor(a[2], "x");
        if (W.dim() != 2 || x.dim() != 2) refuse("Wq must be [N, K] and x [M, K]");
        const int64_t N = W.size(0), K = W.size(1), M = x.size(0);
        const c10::Device dev = x.device();
        expect(W, "Wq", at::kChar, {N, K}, dev);
        expect(step, "wstep", at::kFloat, {N}, dev);
        expect(x, "x", at::kBFloat16, {M, K}, dev);
        const uint16_t* residual = nullptr;
        if (a[4] != Py_None) {
            const at::Tensor& r = tensor(a[4], "residual");
            expect(r, "residual", at::kBFloat16, {M, N}, dev);
            residual = bits(r);
        }
        const bool rmsnorm = a[3] == Py_True, want_acc = a[5] == Py_True;
        at::ScalarType type = a[6] == Py_True ? at::kFloat : at::kBFloat16;
        const c10::cuda::CUDAGuard guard(dev);
        at::Tensor out;
        if (a[7] == Py_None) {
            out = at::empty({M, N}, x.options().dtype(type));
        } else {
            out = tensor(a[7], "out");
            if (out.scalar_type() == at::kFloat || out.scalar_type() == at::kBFloat16) type = out.scalar_type();
            expect(out, "out", type, {M, N}, dev);
        }
        at::Tensor acc = want_acc ? at::empty({M, N}, x.options().dtype(at::kInt)) : at::Tensor();
        at::Tensor ws = a[8] == Py_None ? at::empty({(int64_t)lib.workspace_bytes(BL_OP_FORWARD_INT8, M, N, K)}, x.options().dtype(at::kByte))
                                        : tensor(a[8], "ws");
        if (ws.device() != dev || !ws.is_contiguous()) refuse("ws must be contiguous, on " + dev.str());
        const bl_status st = lib.forward_int8((const int8_t*)W.data_ptr(), (const float*)step.data_ptr(), N, K, bits(x), M, rmsnorm, residual,
                                              out.data_ptr(), type == at::kFloat ? BL_FP32 : BL_BF16,
                                              want_acc ? (int32_t*)acc.data_ptr() : nullptr, ws.data_ptr(), ws.nbytes(), stream(dev));
        if (st) return PyLong_FromLong(st);
        if (!want_acc) return wrap(out);
        PyObject *po = wrap(out), *pa = wrap(acc), *both = PyTuple_Pack(2, po, pa);
        Py_XDECREF(po);
        Py_XDECREF(pa);
        return both;
    });
}

#define BL_METHOD(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {BL_METHOD(bind),          BL_METHOD(kv4_check),    BL_METHOD(kv4_append), BL_METHOD(kv4_read),
                         BL_METHOD(kv4_attention), BL_METHOD(forward_int8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
