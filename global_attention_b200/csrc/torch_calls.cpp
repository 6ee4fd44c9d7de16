// torch_calls.cpp — the calls of a decode step (include/zgcm_qkrope.h, include/zgcm_kv8.h) for torch tensors:
// the module global_attention_b200._calls, under the functions of the same names in __init__.py.
//
// A decode step is a handful of calls of a few microseconds each on the device.  Checking tensors and making
// outputs from Python took 10 to 30 us a call, several times the kernels; here it takes 1 to 3.  The rules
// are those of the rest of the binding: every tensor's type, layout, shape and device is checked
// before the library is called, a wrong one raises TypeError, a status of the library is returned as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "zgcm_kv8.h"
#include "zgcm_qkrope.h"

namespace {

using at::Tensor;

struct Refused {   // becomes a TypeError
    std::string what;
};

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const Tensor& tensor(PyObject* o, const char* name, int64_t rank) {
    if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a torch tensor"};
    const Tensor& t = THPVariable_Unpack(o);
    if (t.dim() != rank) throw Refused{std::string(name) + " must be a tensor of rank " + std::to_string(rank)};
    return t;
}

void on_device(const Tensor& t, const char* name, int index) {
    if (!t.is_cuda()) throw Refused{std::string(name) + " must be a CUDA tensor"};
    if (t.get_device() != index)
        throw Refused{std::string(name) + " must be on the device of the other tensors (cuda:" + std::to_string(index) + ")"};
}

void is(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
    if (t.scalar_type() != dtype || t.sizes() != shape)
        throw Refused{std::string(name) + " must have dtype " + at::toString(dtype) + " and shape " + shape_text(shape) + ", not " +
                      at::toString(t.scalar_type()) + " " + shape_text(t.sizes())};
}

// a contiguous tensor of that type and shape
const Tensor& dense(PyObject* o, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
    const Tensor& t = tensor(o, name, (int64_t)shape.size());
    is(t, name, dtype, shape);
    if (!t.is_contiguous()) throw Refused{std::string(name) + " must be contiguous"};
    return t;
}

bool given(PyObject* o) { return o != Py_None; }

int zgcm_type(at::ScalarType t, const char* name) {
    switch (t) {
        case at::kBFloat16: return ZGCM_BF16;
        case at::kHalf: return ZGCM_FP16;
        case at::kFloat: return ZGCM_FP32;
        default: throw Refused{std::string(name) + " must be bfloat16, float16 or float32"};
    }
}

// [T, H, D] with contiguous rows; the stride of a dimension of one is not looked at (torch lets it be anything).
// out: no two elements in one place
zgcm_rows rows(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape, bool out = false) {
    is(t, name, dtype, shape);
    const int64_t T = shape[0], H = shape[1], D = shape[2];
    if (D > 1 && t.stride(2) != 1) throw Refused{std::string(name) + " must have contiguous rows"};
    const int64_t ts = T > 1 ? t.stride(0) : 0, hs = H > 1 ? t.stride(1) : 0;
    if (out && T > 0) {
        const bool t_first = ts <= hs;
        int64_t reach = D;
        for (int i = 0; i < 2; ++i) {
            const bool is_t = (i == 0) == t_first;
            const int64_t s = is_t ? ts : hs, n = is_t ? T : H;
            if (n > 1) {
                if (s < reach) throw Refused{std::string(name) + " must not overlap itself"};
                reach += s * (n - 1);
            }
        }
    }
    return zgcm_rows{t.data_ptr(), ts, hs};
}

// on the current device and stream (at::empty, through the dispatcher, took 1.5 us: as long as the launch)
Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype) {
    return at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                     dtype, std::nullopt);
}

bool off(const Tensor& t) { return (reinterpret_cast<uintptr_t>(t.const_data_ptr()) & 15u) != 0; }

// int32 positions, counts and lists may begin anywhere (a slice of a longer tensor), the library wants them at 16 bytes: others
// are copied, on the stream of the call (`Here` lives), into `copy`
const int* ints(const Tensor& t, Tensor& copy) {
    if (!off(t)) return t.const_data_ptr<int>();
    copy = fresh(t.sizes(), at::kInt);
    copy.copy_(t);
    return copy.const_data_ptr<int>();
}

int to_int(PyObject* o) {   // as the C int the library takes; larger ones are the largest
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v > 2147483647LL ? 2147483647 : v < -2147483648LL ? -2147483647 - 1 : (int)v;
}

double to_double(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

int as_int(int64_t n, const char* what) {   // a size the library takes as an int
    if (n > 2147483647LL) throw Refused{std::string(what) + " is too large"};
    return (int)n;
}

// The device `index` and the stream of the call, current while this lives: what is allocated in between belongs
// to the stream that writes it, so that a workspace freed at the return is not handed out before the kernels end.
class Here {
public:
    Here(PyObject* stream, int index) : device_((c10::DeviceIndex)index) {
        if (stream == Py_None) {
            handle_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
            return;
        }
        const long long on = number(stream, "device_index");
        if (on != index)
            throw Refused{"stream must be on the device of the tensors (cuda:" + std::to_string(index) + ")"};
        handle_ = reinterpret_cast<cudaStream_t>((uintptr_t)number(stream, "cuda_stream"));
        stream_.reset_stream(c10::cuda::getStreamFromExternal(handle_, (c10::DeviceIndex)index));
    }
    void* handle() const { return handle_; }

private:
    static long long number(PyObject* o, const char* name) {
        PyObject* x = PyObject_GetAttrString(o, name);
        const long long v = x ? PyLong_AsLongLong(x) : -1;
        Py_XDECREF(x);
        if (PyErr_Occurred()) throw python_error();
        return v;
    }
    c10::cuda::CUDAGuard device_;
    c10::cuda::OptionalCUDAStreamGuard stream_;
    cudaStream_t handle_ = nullptr;
};

template <typename F> PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_TypeError, e.what.c_str());
        return nullptr;
    } catch (...) {   // Python's own, torch's (out of memory)
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

bool count_args(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, not %zd", want, n);
    return false;
}

PyObject* status(int st) { return PyLong_FromLong(st); }

PyObject* pair(const Tensor& a, const Tensor& b) {
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = x ? THPVariable_Wrap(b) : nullptr;
    PyObject* t = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

struct Qk {
    const Tensor &q, &k;
    int64_t T, Hq, Hkv, D;
    at::ScalarType dtype;
    int x_type, index;
    zgcm_rows rq, rk;
    const float *gamma_q, *gamma_k;
    const Tensor& pos;
};

Qk qk_inputs(PyObject* const* a) {   // q, k, gamma_q, gamma_k, pos
    const Tensor &q = tensor(a[0], "q", 3), &k = tensor(a[1], "k", 3);
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    for (const int64_t n : {T, Hq, Hkv, D}) as_int(n, "a dimension");
    const at::ScalarType dtype = q.scalar_type();
    const int x_type = zgcm_type(dtype, "q");
    const zgcm_rows rq = rows(q, "q", dtype, {T, Hq, D}), rk = rows(k, "k", dtype, {T, Hkv, D});
    const Tensor &gq = dense(a[2], "gamma_q", at::kFloat, {D}), &gk = dense(a[3], "gamma_k", at::kFloat, {D});
    const Tensor& pos = dense(a[4], "pos", at::kInt, {T});
    on_device(q, "q", q.is_cuda() ? q.get_device() : -1);
    const int index = q.get_device();
    on_device(k, "k", index);
    on_device(gq, "gamma_q", index);
    on_device(gk, "gamma_k", index);
    on_device(pos, "pos", index);
    return Qk{q, k, T, Hq, Hkv, D, dtype, x_type, index, rq, rk, gq.const_data_ptr<float>(), gk.const_data_ptr<float>(), pos};
}

// (q, k, gamma_q, gamma_k, pos, rope_dims, rope_base, eps, out_dtype, qr, kr, stream)
PyObject* qk_norm_rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_args(n, 12)) return nullptr;
    return guarded([&]() -> PyObject* {
        at::ScalarType out = at::kFloat;
        if (given(a[8])) {
            if (!THPDtype_Check(a[8])) throw Refused{"out_dtype must be a torch dtype"};
            out = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
        } else if (given(a[9]) || given(a[10])) {
            out = tensor(given(a[9]) ? a[9] : a[10], "qr", 3).scalar_type();
        } else {
            out = tensor(a[0], "q", 3).scalar_type();
        }
        const int y_type = zgcm_type(out, "out_dtype");
        // the outputs' own checks come first where they are given: a CPU test sees them
        if (given(a[9])) rows(tensor(a[9], "qr", 3), "qr", out, tensor(a[0], "q", 3).sizes(), true);
        if (given(a[10])) rows(tensor(a[10], "kr", 3), "kr", out, tensor(a[1], "k", 3).sizes(), true);
        const Qk x = qk_inputs(a);
        const Here here(a[11], x.index);
        const Tensor qr = given(a[9]) ? THPVariable_Unpack(a[9]) : fresh({x.T, x.Hq, x.D}, out);
        const Tensor kr = given(a[10]) ? THPVariable_Unpack(a[10]) : fresh({x.T, x.Hkv, x.D}, out);
        on_device(qr, "qr", x.index);
        on_device(kr, "kr", x.index);
        Tensor copy;
        const int st = zgcm_qk_norm_rope_fwd(x.rq, x.rk, x.gamma_q, x.gamma_k, ints(x.pos, copy), (int)x.T, (int)x.Hq, (int)x.Hkv,
                                             (int)x.D, x.x_type, y_type, to_int(a[5]), to_double(a[6]), (float)to_double(a[7]),
                                             rows(qr, "qr", out, {x.T, x.Hq, x.D}), rows(kr, "kr", out, {x.T, x.Hkv, x.D}),
                                             here.handle());
        return st == ZGCM_OK ? pair(qr, kr) : status(st);
    });
}

const char* const kGrads[] = {"dq", "dk", "dgamma_q", "dgamma_k"};

// (q, k, gamma_q, gamma_k, pos, dqr, dkr, rope_dims, rope_base, eps, dq, dk, dgamma_q, dgamma_k, workspace, stream); the
// four gradients are given together or not at all
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_args(n, 16)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Tensor &q0 = tensor(a[0], "q", 3), &k0 = tensor(a[1], "k", 3), &dqr = tensor(a[5], "dqr", 3);
        const at::ScalarType dy = dqr.scalar_type();
        const int y_type = zgcm_type(dy, "dqr");
        const zgcm_rows rdqr = rows(dqr, "dqr", dy, q0.sizes()), rdkr = rows(tensor(a[6], "dkr", 3), "dkr", dy, k0.sizes());
        const bool have = given(a[10]) || given(a[11]) || given(a[12]) || given(a[13]);
        if (have) {
            rows(tensor(a[10], "dq", 3), "dq", q0.scalar_type(), q0.sizes(), true);
            rows(tensor(a[11], "dk", 3), "dk", q0.scalar_type(), k0.sizes(), true);
            dense(a[12], "dgamma_q", at::kFloat, {q0.size(2)});
            dense(a[13], "dgamma_k", at::kFloat, {q0.size(2)});
        }
        if (given(a[14])) dense(a[14], "workspace", at::kByte, {tensor(a[14], "workspace", 1).numel()});
        const Qk x = qk_inputs(a);
        on_device(dqr, "dqr", x.index);
        on_device(THPVariable_Unpack(a[6]), "dkr", x.index);
        const Here here(a[15], x.index);
        Tensor g[4];
        for (int i = 0; i < 4; ++i) {
            if (have)
                g[i] = THPVariable_Unpack(a[10 + i]);
            else
                g[i] = i < 2 ? fresh({x.T, i ? x.Hkv : x.Hq, x.D}, x.dtype) : fresh({x.D}, at::kFloat);
            on_device(g[i], kGrads[i], x.index);
        }
        const int64_t need = (int64_t)zgcm_qk_norm_rope_bwd_workspace_size((int)x.T);
        const Tensor ws = given(a[14]) ? THPVariable_Unpack(a[14]) : fresh({need}, at::kByte);
        on_device(ws, "workspace", x.index);
        Tensor copy;
        const int st = zgcm_qk_norm_rope_bwd(x.rq, x.rk, x.gamma_q, x.gamma_k, ints(x.pos, copy), rdqr, rdkr, (int)x.T, (int)x.Hq,
                                             (int)x.Hkv, (int)x.D, x.x_type, y_type, to_int(a[7]), to_double(a[8]), (float)to_double(a[9]),
                                             rows(g[0], "dq", x.dtype, {x.T, x.Hq, x.D}),
                                             rows(g[1], "dk", x.dtype, {x.T, x.Hkv, x.D}), g[2].data_ptr<float>(),
                                             g[3].data_ptr<float>(), ws.data_ptr(), (size_t)ws.numel(), here.handle());
        if (st != ZGCM_OK) return status(st);
        PyObject* d = PyDict_New();
        for (int i = 0; d && i < 4; ++i) {
            PyObject* t = THPVariable_Wrap(g[i]);
            if (!t || PyDict_SetItemString(d, kGrads[i], t) != 0) Py_CLEAR(d);
            Py_XDECREF(t);
        }
        return d;
    });
}

// a cache: the address of its zgcm_kv8_cache, and one of its tensors (its device)
struct Cache {
    const zgcm_kv8_cache* c;
    int index;
    at::ScalarType key;
};

Cache cache_of(PyObject* addr, PyObject* any) {
    const void* p = PyLong_AsVoidPtr(addr);
    if (!p) {
        if (PyErr_Occurred()) throw python_error();
        throw Refused{"not a cache"};
    }
    const auto* c = static_cast<const zgcm_kv8_cache*>(p);
    const Tensor& t = THPVariable_Unpack(any);
    return Cache{c, t.is_cuda() ? (int)t.get_device() : -1, c->key_type == ZGCM_BF16 ? at::kBFloat16 : at::kHalf};
}

// [n_seq, N, Hkv, D] with contiguous rows
const Tensor& tokens(PyObject* o, const char* name, const Cache& c, at::ScalarType dtype, int64_t N, long long (&s)[3]) {
    const Tensor& t = tensor(o, name, 4);
    is(t, name, dtype, {c.c->n_seq, N, c.c->Hkv, c.c->D});
    if (c.c->D > 1 && t.stride(3) != 1) throw Refused{std::string(name) + " must have contiguous rows"};
    for (int i = 0; i < 3; ++i) s[i] = t.size(i) > 1 ? t.stride(i) : 0;
    on_device(t, name, c.index);
    return t;
}

const Tensor* optional(PyObject* o, const char* name, at::ScalarType dtype, at::IntArrayRef shape, int index) {
    if (!given(o)) return nullptr;
    const Tensor& t = dense(o, name, dtype, shape);
    on_device(t, name, index);
    return &t;
}

// (cache address, tensor of it, k, v, pos, count, stream)
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_args(n, 7)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Cache c = cache_of(a[0], a[1]);
        const int64_t N = tensor(a[2], "k", 4).size(1);
        long long ks[3], vs[3];
        const Tensor &k = tokens(a[2], "k", c, c.key, N, ks), &v = tokens(a[3], "v", c, at::kBFloat16, N, vs);
        const Tensor& pos = dense(a[4], "pos", at::kInt, {c.c->n_seq});
        on_device(pos, "pos", c.index);
        const Tensor* count = optional(a[5], "count", at::kInt, {c.c->n_seq}, c.index);
        const Here here(a[6], c.index);
        Tensor copies[2];
        const int* at = ints(pos, copies[0]);
        return status(zgcm_kv8_append(c.c, k.const_data_ptr(), ks[0], ks[1], ks[2], v.const_data_ptr(), vs[0], vs[1], vs[2], at,
                                      count ? ints(*count, copies[1]) : nullptr, as_int(N, "the number of tokens"),
                                      here.handle()));
    });
}

// (cache address, tensor of it, q, g, pos, blocks, window, scale, out, lse, workspace, stream)
PyObject* attn_decode_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_args(n, 12)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Cache c = cache_of(a[0], a[1]);
        const int64_t B = c.c->n_seq, D = c.c->D, Hq = tensor(a[2], "q", 3).size(1);
        const Tensor& q = dense(a[2], "q", c.key, {B, Hq, D});
        const Tensor& pos = dense(a[4], "pos", at::kInt, {B});
        const int n_list = given(a[5]) ? as_int(tensor(a[5], "blocks", 3).size(2), "the list") : -1;
        on_device(q, "q", c.index);
        on_device(pos, "pos", c.index);
        const Tensor* g = optional(a[3], "g", at::kBFloat16, {B, Hq, D}, c.index);
        const Tensor* list = optional(a[5], "blocks", at::kInt, {B, c.c->Hkv, n_list}, c.index);
        optional(a[8], "out", at::kBFloat16, {B, Hq, D}, c.index);
        optional(a[9], "lse", at::kFloat, {B, Hq}, c.index);
        if (given(a[10])) optional(a[10], "workspace", at::kByte, {tensor(a[10], "workspace", 1).numel()}, c.index);
        const int window = to_int(a[6]), heads = as_int(Hq, "the number of heads");
        const Here here(a[11], c.index);
        const Tensor out = given(a[8]) ? THPVariable_Unpack(a[8]) : fresh({B, Hq, D}, at::kBFloat16);
        const Tensor lse = given(a[9]) ? THPVariable_Unpack(a[9]) : fresh({B, Hq}, at::kFloat);
        void* ws = nullptr;
        size_t bytes = 0;
        Tensor mine;
        if (given(a[10])) {
            const Tensor& t = THPVariable_Unpack(a[10]);
            ws = t.data_ptr();
            bytes = (size_t)t.numel();
        } else if ((bytes = zgcm_attn_decode_kv8_workspace_size(c.c, heads, window, n_list)) > 0) {
            mine = fresh({(int64_t)bytes}, at::kByte);
            ws = mine.data_ptr();
        }
        Tensor copies[2];
        const int* at = ints(pos, copies[0]);
        // an empty list is not read: only that there is one counts
        const int* blocks = !list ? nullptr : n_list == 0 ? at : ints(*list, copies[1]);
        const int st = zgcm_attn_decode_kv8(c.c, q.const_data_ptr(), g ? g->const_data_ptr() : nullptr, at, blocks,
                                            n_list < 0 ? 0 : n_list, heads, window, (float)to_double(a[7]),
                                            out.data_ptr(), lse.data_ptr<float>(), ws, bytes, here.handle());
        return st == ZGCM_OK ? pair(out, lse) : status(st);
    });
}

// (cache address, tensor of it, q, pos, n_select, n_first, n_last, window, out, stream)
PyObject* kv8_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!count_args(n, 10)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Cache c = cache_of(a[0], a[1]);
        const int64_t B = c.c->n_seq, Hq = tensor(a[2], "q", 3).size(1);
        const Tensor& q = dense(a[2], "q", c.key, {B, Hq, c.c->D});
        const Tensor& pos = dense(a[3], "pos", at::kInt, {B});
        const int n_select = to_int(a[4]);
        const int64_t shape[3] = {B, c.c->Hkv, n_select < 0 ? 0 : n_select};
        on_device(q, "q", c.index);
        on_device(pos, "pos", c.index);
        optional(a[8], "out", at::kInt, shape, c.index);
        const Here here(a[9], c.index);
        const Tensor out = given(a[8]) ? THPVariable_Unpack(a[8]) : fresh(shape, at::kInt);
        const Tensor made = off(out) ? fresh(shape, at::kInt) : out;
        Tensor copy;
        const int st = zgcm_kv8_select(c.c, q.const_data_ptr(), ints(pos, copy), as_int(Hq, "the number of heads"), to_int(a[7]),
                                       n_select, to_int(a[5]), to_int(a[6]), made.data_ptr<int>(), here.handle());
        if (st != ZGCM_OK) return status(st);
        if (!made.is_same(out)) out.copy_(made);
        return THPVariable_Wrap(out);
    });
}

#define CALL(f) \
    { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {CALL(qk_norm_rope_fwd), CALL(qk_norm_rope_bwd), CALL(kv8_append), CALL(attn_decode_kv8),
                          CALL(kv8_select), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
