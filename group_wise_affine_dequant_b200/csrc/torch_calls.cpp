// The serving calls from torch tensors: the argument marshalling that binding.py
// does for the other entry points, in C++. A decoding step makes these calls for every layer
// on sizes where the kernels take a few microseconds; through ctypes and tensor
// attributes the marshalling alone took 7 to 20 (one token through the router: 12 us a call,
// 4.5 so).
//
// A Python extension module `_calls` with no logic of its own: it checks what
// needs shapes, allocates outputs and workspaces, and calls libnvq's C entry
// points through the addresses that bind() is given, so that there is one loaded
// library. A function returns its outputs, or the status (an int) of a refused
// call; wrong tensors raise ValueError before anything is launched.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "../../include/nvq.h"

namespace {

// The entry points, in the order of bind().
decltype(&nv_moe_route) p_moe_route = nullptr;
decltype(&nv_kv_quantize) p_kv_quantize = nullptr;
decltype(&nv_kv_dequantize) p_kv_dequantize = nullptr;
decltype(&nv_kv_attention) p_kv_attention = nullptr;
decltype(&nv_kv_attention_workspace_size) p_kv_workspace = nullptr;

struct BadArgument : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {};  // a Python exception is set

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw BadArgument(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}
int small(PyObject* o) {  // an int argument of the C calls, clamped so that none wraps around
    const int64_t v = integer(o);
    return static_cast<int>(v < INT32_MIN ? INT32_MIN : v > INT32_MAX ? INT32_MAX : v);
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return static_cast<float>(v);
}
nv_dtype dtype_of(at::ScalarType t) {
    return t == at::kFloat ? NV_F32 : t == at::kBFloat16 ? NV_BF16 : static_cast<nv_dtype>(-1);
}
void need(bool ok, const char* what) {
    if (!ok) throw BadArgument(what);
}
// Makes a device current for a call, where it is not, and with it the stream whose handle the
// caller gave: outputs and workspaces come from that stream's memory, so that none of them is what
// another stream still uses, or may take when the call has returned.
struct On {
    c10::cuda::OptionalCUDAGuard on_device;
    c10::cuda::OptionalCUDAStreamGuard on_stream;
    nv_stream_t stream;
    On(c10::DeviceIndex device, PyObject* handle) {
        if (handle == Py_None) {
            if (device != c10::cuda::current_device()) on_device.set_index(device);
            stream = reinterpret_cast<nv_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
            return;
        }
        void* p = PyLong_AsVoidPtr(handle);
        if (!p && PyErr_Occurred()) throw PythonError();
        stream = static_cast<nv_stream_t>(p);
        on_stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), device));
    }
};
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType t, c10::DeviceIndex device) {
    return at::Tensor(at::detail::empty_cuda(shape, t, at::Device(at::kCUDA, device), std::nullopt));
}
bool is_on(const at::Tensor& t, c10::DeviceIndex device) { return t.is_cuda() && t.get_device() == device; }

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = THPVariable_Wrap(b);
    PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}
PyObject* refused(nv_status s) { return PyLong_FromLong(s); }

// Runs a call; what it throws becomes a Python exception.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t wanted, const F& f) {
    if (got != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, wanted);
        return nullptr;
    }
    if (!p_moe_route) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return nullptr;
    }
    try {
        return f();
    } catch (const BadArgument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const PythonError&) {
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

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses expected");
        return nullptr;
    }
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    p_moe_route = reinterpret_cast<decltype(p_moe_route)>(p[0]);
    p_kv_quantize = reinterpret_cast<decltype(p_kv_quantize)>(p[1]);
    p_kv_dequantize = reinterpret_cast<decltype(p_kv_dequantize)>(p[2]);
    p_kv_attention = reinterpret_cast<decltype(p_kv_attention)>(p[3]);
    p_kv_workspace = reinterpret_cast<decltype(p_kv_workspace)>(p[4]);
    Py_RETURN_NONE;
}

// moe_route(logits, topk, score, bias, groups, topk_groups, group_top, renormalize, scale, ids, weights, stream)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const at::Tensor& z = tensor(a[0], "logits");
        need(z.is_cuda() && z.dim() == 2 && z.is_contiguous(), "logits must be a contiguous CUDA tensor [T, E]");
        const c10::DeviceIndex device = z.get_device();
        const int64_t T = z.size(0), E = z.size(1);
        const int topk = small(a[1]);
        const float* bias = nullptr;
        if (a[3] != Py_None) {
            const at::Tensor& b = tensor(a[3], "bias");
            need(is_on(b, device) && b.scalar_type() == at::kFloat && b.numel() == E && b.is_contiguous(),
                 "bias must be contiguous fp32 [E] on the logits' device");
            bias = static_cast<const float*>(b.data_ptr());
        }
        const On on(device, a[11]);
        auto output = [&](PyObject* o, at::ScalarType t, const char* what) {
            if (o == Py_None) return fresh({T, topk < 0 || topk > E ? 0 : topk}, t, device);  // 0: about to be refused
            const at::Tensor& x = tensor(o, what);
            need(is_on(x, device) && x.scalar_type() == t && x.dim() == 2 && x.size(0) == T && x.size(1) == topk &&
                     x.is_contiguous(),
                 "ids and weights must be contiguous int32 and fp32 [T, topk] on the logits' device");
            return x;
        };
        const at::Tensor ids = output(a[9], at::kInt, "ids"), weights = output(a[10], at::kFloat, "weights");
        const nv_status st = p_moe_route(z.data_ptr(), dtype_of(z.scalar_type()), T, E, bias, small(a[2]), small(a[4]),
                                         small(a[5]), small(a[6]), topk, small(a[7]), real(a[8]),
                                         static_cast<uint32_t*>(ids.data_ptr()), static_cast<float*>(weights.data_ptr()),
                                         on.stream);
        return st == NV_OK ? pair(ids, weights) : refused(st);
    });
}

// The cache and the step descriptor, from eight arguments: k_codes, k_scales, v_codes,
// v_scales, pages, starts, lens, flags.
struct Cache {
    c10::DeviceIndex device;
    uint8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    nv_kv_mode mode;
    int64_t P, H, block, D;
    const int32_t *pages, *starts, *lens;
    int64_t max_pages, S;
    uint32_t* flags;

    explicit Cache(PyObject* const* a) {
        const at::Tensor& kc = tensor(a[0], "k_codes");
        const at::Tensor& ks = tensor(a[1], "k_scales");
        const at::Tensor& vc = tensor(a[2], "v_codes");
        const at::Tensor& vs = tensor(a[3], "v_scales");
        const at::Tensor& pg = tensor(a[4], "pages");
        const at::Tensor& sts = tensor(a[5], "starts");
        const at::Tensor& ln = tensor(a[6], "lens");
        need(kc.is_cuda(), "the cache must be on a CUDA device");
        device = kc.get_device();
        for (const at::Tensor* t : {&kc, &ks, &vc, &vs, &pg, &sts, &ln})
            need(is_on(*t, device) && t->is_contiguous(),
                 "the cache, pages, starts and lens must be contiguous CUDA tensors on one device");
        const at::ScalarType type = kc.scalar_type();
        need(kc.dim() == 4 && kc.sizes() == vc.sizes() && vc.scalar_type() == type &&
                 (type == at::kChar || type == at::kFloat8_e4m3fn),
             "k_codes and v_codes must be int8 or float8_e4m3fn [P, H, block, D] alike");
        mode = type == at::kChar ? NV_KV_INT8 : NV_KV_E4M3;
        P = kc.size(0);
        H = kc.size(1);
        block = kc.size(2);
        D = kc.size(3);
        for (const at::Tensor* t : {&ks, &vs})
            need(t->scalar_type() == at::kFloat && t->dim() == 2 && t->size(0) == P && t->size(1) == H,
                 "k_scales and v_scales must be fp32 [P, H]");
        need(pg.dim() == 2 && sts.dim() == 1 && ln.dim() == 1 && sts.size(0) == pg.size(0) + 1 && ln.size(0) == pg.size(0),
             "pages [S, max_pages], starts [S + 1] and lens [S] expected");
        need(pg.scalar_type() == at::kInt && sts.scalar_type() == at::kInt && ln.scalar_type() == at::kInt,
             "pages, starts and lens must be int32");
        S = pg.size(0);
        max_pages = pg.size(1);
        flags = nullptr;
        if (a[7] != Py_None) {
            const at::Tensor& f = tensor(a[7], "flags");
            need(is_on(f, device) && f.scalar_type() == at::kInt && f.numel() >= 1,
                 "flags must be an int32 CUDA tensor on the cache's device");
            flags = static_cast<uint32_t*>(f.data_ptr());
        }
        need(H <= INT32_MAX && block <= INT32_MAX && D <= INT32_MAX, "sizes beyond 32 bits");
        k_codes = static_cast<uint8_t*>(kc.data_ptr());
        v_codes = static_cast<uint8_t*>(vc.data_ptr());
        k_scales = static_cast<float*>(ks.data_ptr());
        v_scales = static_cast<float*>(vs.data_ptr());
        pages = static_cast<const int32_t*>(pg.data_ptr());
        starts = static_cast<const int32_t*>(sts.data_ptr());
        lens = static_cast<const int32_t*>(ln.data_ptr());
    }
    // Row stride of a step's tensor [rows, heads, D]: dense heads, any distance between rows.
    int64_t stride(const at::Tensor& t, int64_t heads) const {
        need(is_on(t, device) && t.dim() == 3 && t.size(1) == heads && t.size(2) == D,
             "the step's tensors must be [rows, heads, D] on the cache's device");
        need((t.stride(2) == 1 || D <= 1) && (t.stride(1) == D || heads <= 1), "the heads of a row must be dense");
        return t.size(0) > 1 ? t.stride(0) : heads * D;
    }
};

// kv_quantize(k, v, <cache and steps>, stream)
PyObject* kv_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor& k = tensor(a[0], "k");
        const at::Tensor& v = tensor(a[1], "v");
        const Cache c(a + 2);
        const int64_t ks = c.stride(k, c.H), vs = c.stride(v, c.H);
        need(k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type(), "k and v must be alike");
        const On on(c.device, a[10]);
        return refused(p_kv_quantize(k.data_ptr(), v.data_ptr(), ks, vs, dtype_of(k.scalar_type()), k.size(0), c.k_codes,
                                     c.k_scales, c.v_codes, c.v_scales, c.mode, c.P, static_cast<int>(c.H),
                                     static_cast<int>(c.block), static_cast<int>(c.D), c.pages, c.max_pages, c.starts,
                                     c.lens, c.S, c.flags, on.stream));
    });
}

// kv_dequantize(<cache and steps>, rows, dtype, k, v (outputs or None), stream)
PyObject* kv_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const Cache c(a);
        const int64_t rows = integer(a[8]);
        const auto* dt = THPDtype_Check(a[9]) ? reinterpret_cast<THPDtype*>(a[9]) : nullptr;
        need(dt != nullptr, "dtype must be a torch.dtype");
        const at::ScalarType type = dt->scalar_type;
        need(rows >= 0, "rows must not be negative");
        const On on(c.device, a[12]);
        auto output = [&](PyObject* o) {
            if (o == Py_None) return fresh({rows, c.H, c.D}, type, c.device);
            const at::Tensor& x = tensor(o, "out");
            need(is_on(x, c.device) && x.scalar_type() == type && x.dim() == 3 && x.size(0) == rows && x.size(1) == c.H &&
                     x.size(2) == c.D && x.is_contiguous(),
                 "out must be two contiguous [rows, H, D] tensors of the dtype on the cache's device");
            return x;
        };
        const at::Tensor k = output(a[10]), v = output(a[11]);
        const nv_status st = p_kv_dequantize(c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.mode, c.P,
                                             static_cast<int>(c.H), static_cast<int>(c.block), static_cast<int>(c.D),
                                             c.pages, c.max_pages, c.starts, c.lens, c.S, dtype_of(type), rows,
                                             k.data_ptr(), v.data_ptr(), c.flags, on.stream);
        return st == NV_OK ? pair(k, v) : refused(st);
    });
}

// kv_attention(q, <cache and steps>, scale, causal, window, max_q, workspace, out, stream)
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const Cache c(a + 1);
        need(q.dim() == 3, "q must be [rows, Hq, D]");
        const int64_t rows = q.size(0), Hq = q.size(1), qs = c.stride(q, Hq);
        need(Hq <= INT32_MAX, "sizes beyond 32 bits");
        const nv_dtype dt = dtype_of(q.scalar_type());
        const float scale = a[9] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.D))) : real(a[9]);
        const int window = small(a[11]);
        const int64_t max_q = integer(a[12]);
        const int H = static_cast<int>(c.H), block = static_cast<int>(c.block), D = static_cast<int>(c.D);
        const On on(c.device, a[15]);
        at::Tensor out;
        if (a[14] == Py_None) {
            out = fresh({rows, Hq, c.D}, q.scalar_type(), c.device);
        } else {
            out = tensor(a[14], "out");
            need(is_on(out, c.device) && out.scalar_type() == q.scalar_type() && out.sizes() == q.sizes() && out.is_contiguous(),
                 "out must be contiguous and like q");
        }
        at::Tensor workspace;
        if (a[13] == Py_None) {
            const size_t bytes = p_kv_workspace(dt, rows, static_cast<int>(Hq), H, block, D, c.max_pages, c.S, max_q);
            if (bytes) workspace = fresh({static_cast<int64_t>(bytes)}, at::kByte, c.device);
        } else {
            workspace = tensor(a[13], "workspace");
            need(is_on(workspace, c.device) && workspace.is_contiguous(),
                 "workspace must be a contiguous CUDA tensor on the cache's device");
        }
        const nv_status st = p_kv_attention(
            q.data_ptr(), qs, dt, rows, static_cast<int>(Hq), c.k_codes, c.k_scales, c.v_codes, c.v_scales, c.mode, c.P, H,
            block, D, c.pages, c.max_pages, c.starts, c.lens, c.S, scale, small(a[10]), window, max_q,
            workspace.defined() ? workspace.data_ptr() : nullptr, workspace.defined() ? workspace.nbytes() : 0,
            out.data_ptr(), c.flags, on.stream);
        return st == NV_OK ? THPVariable_Wrap(out) : refused(st);
    });
}

template <class F>
constexpr PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"moe_route", fast(moe_route), METH_FASTCALL, nullptr},
                         {"kv_quantize", fast(kv_quantize), METH_FASTCALL, nullptr},
                         {"kv_dequantize", fast(kv_dequantize), METH_FASTCALL, nullptr},
                         {"kv_attention", fast(kv_attention), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
