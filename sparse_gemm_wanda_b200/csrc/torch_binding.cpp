// Argument marshalling of the calls that run between the products of a decoder
// block (patch_hybrid_linear, _linear_group, _gated, patch_block_norm), as a
// CPython module over PyTorch tensors.  Checks, output allocation and the call
// into the C ABI, nothing else: at decode sizes a call's kernels take 2 to 8 us
// and the same steps through ctypes and tensor attributes took 12 to 23.
//
// The functions of the C ABI arrive as addresses (`bind`), so this module and
// the ctypes binding drive one library.  Work goes to the current stream of
// the current device, outputs are allocated there.  Refused arguments raise
// ValueError; a status other than PATCH_OK is returned as an int for the
// caller to raise.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <stdint.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <string>

#include "patch.h"

namespace {

decltype(&patch_hybrid_linear_group) g_linear = nullptr;
decltype(&patch_hybrid_gated) g_gated = nullptr;
decltype(&patch_block_norm) g_norm = nullptr;

constexpr Py_ssize_t kMaxGroup = 8;

// Raises ValueError with the parts joined (no streams: PyTorch's libraries
// carry a second copy of their locale machinery, which crashes here).
std::string text(const char *v) { return v; }
std::string text(const std::string &v) { return v; }
std::string text(int64_t v) { return std::to_string(v); }
std::string text(c10::Device d) {
    return d.is_cuda() ? "cuda:" + std::to_string(static_cast<int>(d.index())) : c10::DeviceTypeName(d.type(), true);
}
std::string text(at::ScalarType t) { return c10::toString(t); }
template <class... Args>
[[noreturn]] void refuse(const Args &...args) {
    std::string message;
    ((message += text(args)), ...);
    PyErr_SetString(PyExc_ValueError, message.c_str());
    throw python_error();
}

// the tensor of a Python argument; null for None
const at::Tensor *tensor(PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
    return &THPVariable_Unpack(o);
}

bool is_real(const at::Tensor &t) { return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat; }
bool is_fp32(const at::Tensor *t) { return t && t->scalar_type() == at::kFloat; }

// the call's device, from its first tensor; it has to be the current one
c10::Device device_of(const at::Tensor *t, const char *name) {
    if (!t || !t->is_cuda()) refuse(name, " must be a CUDA tensor");
    if (t->device().index() != c10::cuda::current_device())
        refuse(name, " is on ", t->device(), ", the current device is cuda:",
               static_cast<int64_t>(c10::cuda::current_device()));
    return t->device();
}

void *current_stream(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// address of an optional contiguous [n] bf16 / fp32 vector
const void *vector(const at::Tensor *t, int64_t n, c10::Device dev, const char *name) {
    if (!t) return nullptr;
    if (t->device() != dev || !is_real(*t) || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
        refuse(name, " must be a contiguous bf16 or fp32 vector of ", n, " on ", dev);
    return t->const_data_ptr();
}

// row stride of an [M, C] tensor of contiguous rows
template <class TypeOk>
int64_t row_step(const at::Tensor &t, int64_t M, int64_t C, c10::Device dev, const char *name, const TypeOk &type_ok) {
    if (t.device() != dev || t.dim() != 2 || t.size(0) != M || t.size(1) != C || !type_ok(t))
        refuse(name, " must be [", M, ", ", C, "] of its type on ", dev);
    const int64_t step = M <= 1 ? C : t.stride(0);
    if ((C > 1 && t.stride(1) != 1) || step < C) refuse(name, " must have contiguous rows that do not overlap");
    return step;
}

// address and row stride of an optional input of that form
template <class TypeOk>
const void *rows(const at::Tensor *t, int64_t M, int64_t C, c10::Device dev, const char *name, int64_t *step,
                 const TypeOk &type_ok) {
    *step = t ? row_step(*t, M, C, dev, name, type_ok) : 0;
    return t ? t->const_data_ptr() : nullptr;
}

// A new tensor, without at::empty's way through the dispatcher (0.3 to 0.5 us of
// the 5 to 7 that a small call takes on the host).
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
    return at::detail::empty_cuda(sizes, type, dev, std::nullopt);
}

// The output of a call: the caller's (checked), or a new tensor in `fresh`.  A
// tensor that still shares its storage with a lazy clone gets its own here, so
// outputs come before the addresses of inputs, which may be the same tensor.
PyObject *output(PyObject *given, int64_t M, int64_t C, at::ScalarType type, c10::Device dev, const char *name,
                 at::Tensor *fresh, void **ptr, int64_t *step) {
    if (const at::Tensor *t = tensor(given, name)) {
        *step = row_step(*t, M, C, dev, name, [type](const at::Tensor &x) { return x.scalar_type() == type; });
        *ptr = t->mutable_data_ptr();
        Py_INCREF(given);
        return given;
    }
    *fresh = empty({M, C}, type, dev);
    *ptr = fresh->mutable_data_ptr();
    *step = C;
    return THPVariable_Wrap(*fresh);
}

// (handle, N, K, is FP8) of a PackedWeight
struct Packed {
    const patch_packed *handle;
    int64_t N, K;
    bool fp8;
};
Packed packed(PyObject *info) {
    if (!PyTuple_Check(info) || PyTuple_GET_SIZE(info) != 4) refuse("a packed weight is expected");
    Packed p;
    p.handle = static_cast<const patch_packed *>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(info, 0)));
    p.N = PyLong_AsLongLong(PyTuple_GET_ITEM(info, 1));
    p.K = PyLong_AsLongLong(PyTuple_GET_ITEM(info, 2));
    p.fp8 = PyObject_IsTrue(PyTuple_GET_ITEM(info, 3)) == 1;
    if (PyErr_Occurred()) throw python_error();
    return p;
}

// X [M, K] bf16, or e4m3 codes with their token scales
struct Input {
    c10::Device dev = c10::Device(c10::kCUDA, 0);
    int64_t M;
    const at::Tensor *X, *x_scales;
    const void *x() const { return X->const_data_ptr(); }
    const float *scales() const { return x_scales ? x_scales->const_data_ptr<float>() : nullptr; }
};
Input input(const Packed *ps, Py_ssize_t count, PyObject *X_o, PyObject *scales_o) {
    const at::Tensor *X = tensor(X_o, "X"), *sx = tensor(scales_o, "x_scales");
    Input in;
    in.X = X;
    in.x_scales = sx;
    in.dev = device_of(X, "X");
    if (X->dim() != 2 || !X->is_contiguous()) refuse("X must be a contiguous [M, K] tensor");
    in.M = X->size(0);
    for (Py_ssize_t i = 0; i < count; ++i)
        if (X->size(1) != ps[i].K) refuse("X has ", X->size(1), " columns, the packed weight ", ps[i].K);
    if (!sx) {
        if (X->scalar_type() != at::kBFloat16)
            refuse("X has dtype ", X->scalar_type(), ", expected bfloat16 (or e4m3 codes with x_scales)");
        return in;
    }
    if (X->scalar_type() != at::kByte && X->scalar_type() != at::kFloat8_e4m3fn)
        refuse("X has dtype ", X->scalar_type(), ", expected e4m3 codes (x_scales is given)");
    for (Py_ssize_t i = 0; i < count; ++i)
        if (!ps[i].fp8) refuse("x_scales needs FP8 handles (patch_pack_fp8)");
    if (sx->device() != in.dev || sx->scalar_type() != at::kFloat || sx->dim() != 1 || sx->size(0) != in.M ||
        !sx->is_contiguous())
        refuse("x_scales must be a contiguous fp32 vector of ", in.M, " on ", in.dev);
    return in;
}

// the i-th of an optional sequence of `count`, else None
PyObject *item(PyObject *seq, Py_ssize_t i, Py_ssize_t count, const char *name) {
    if (seq == Py_None) return Py_None;
    if (!PyList_Check(seq) && !PyTuple_Check(seq)) refuse(name, " must be a list");
    if (PySequence_Fast_GET_SIZE(seq) != count) refuse(name, ": one per handle");
    return PySequence_Fast_GET_ITEM(seq, i);
}

template <class Call>
patch_status without_gil(const Call &call) {
    PyThreadState *state = PyEval_SaveThread();
    const patch_status st = call();
    PyEval_RestoreThread(state);
    return st;
}

// a list that owns its references until it is returned
struct Results {
    PyObject *list;
    explicit Results(Py_ssize_t n) : list(PyList_New(n)) {
        if (!list) throw python_error();
    }
    ~Results() { Py_XDECREF(list); }
    PyObject *give() {
        PyObject *l = list;
        list = nullptr;
        return l;
    }
};

// linear(infos, X, x_scales, biases, activation, alpha, residuals, outs, out_fp32)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) refuse("linear: 9 arguments");
    PyObject *infos = a[0];
    if (!PyList_Check(infos) && !PyTuple_Check(infos)) refuse("the packed weights must be a list");
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(infos);
    if (count < 1 || count > kMaxGroup) refuse("1 to 8 packed weights are expected");
    Packed ps[kMaxGroup];
    const patch_packed *handles[kMaxGroup];
    for (Py_ssize_t i = 0; i < count; ++i) {
        ps[i] = packed(PySequence_Fast_GET_ITEM(infos, i));
        handles[i] = ps[i].handle;
    }
    const Input in = input(ps, count, a[1], a[2]);
    const int32_t act = static_cast<int32_t>(PyLong_AsLong(a[4]));
    const float alpha = static_cast<float>(PyFloat_AsDouble(a[5]));
    const bool fp32 = PyObject_IsTrue(a[8]) == 1;
    if (PyErr_Occurred()) throw python_error();
    const at::ScalarType type = fp32 ? at::kFloat : at::kBFloat16;
    patch_epilogue epis[kMaxGroup];
    void *ys[kMaxGroup];
    at::Tensor fresh;
    Results out(count);
    for (Py_ssize_t i = 0; i < count; ++i)
        PyList_SET_ITEM(out.list, i, output(item(a[7], i, count, "outs"), in.M, ps[i].N, type, in.dev, "out", &fresh,
                                            &ys[i], &epis[i].y_stride));
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor *bias = tensor(item(a[3], i, count, "biases"), "bias");
        const at::Tensor *res = tensor(item(a[6], i, count, "residuals"), "residual");
        patch_epilogue &e = epis[i];
        e.bias = vector(bias, ps[i].N, in.dev, "bias");
        e.residual = rows(res, in.M, ps[i].N, in.dev, "residual", &e.residual_stride, is_real);
        e.alpha = alpha;
        e.activation = act;
        e.bias_is_fp32 = is_fp32(bias);
        e.residual_is_fp32 = is_fp32(res);
    }
    void *stream = current_stream(in.dev);
    const patch_status st = without_gil([&] {
        return g_linear(handles, static_cast<int32_t>(count), in.x(), in.scales(), in.M, ys, fp32, epis, stream);
    });
    return st == PATCH_OK ? out.give() : PyLong_FromLong(st);
    END_HANDLE_TH_ERRORS
}

// gated(gate, up, X, x_scales, bias_gate, bias_up, activation, out, out_fp32)
PyObject *gated(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) refuse("gated: 9 arguments");
    const Packed ps[2] = {packed(a[0]), packed(a[1])};
    const int64_t N = ps[0].N;
    if (ps[1].N != N) refuse("the gate has ", N, " rows, the up projection ", ps[1].N);
    const Input in = input(ps, 2, a[2], a[3]);
    const at::Tensor *bg = tensor(a[4], "bias_gate"), *bu = tensor(a[5], "bias_up");
    if (bg && bu && bg->scalar_type() != bu->scalar_type()) refuse("bias_gate and bias_up must have one dtype");
    const int32_t act = static_cast<int32_t>(PyLong_AsLong(a[6]));
    const bool fp32 = PyObject_IsTrue(a[8]) == 1;
    if (PyErr_Occurred()) throw python_error();
    at::Tensor fresh;
    void *y;
    int64_t step;
    THPObjectPtr out(output(a[7], in.M, N, fp32 ? at::kFloat : at::kBFloat16, in.dev, "out", &fresh, &y, &step));
    const void *bgp = vector(bg, N, in.dev, "bias_gate"), *bup = vector(bu, N, in.dev, "bias_up");
    void *stream = current_stream(in.dev);
    const patch_status st = without_gil([&] {
        return g_gated(ps[0].handle, ps[1].handle, in.x(), in.scales(), in.M, y, step, fp32, bgp, bup,
                       is_fp32(bg) || is_fp32(bu), act, stream);
    });
    return st == PATCH_OK ? out.release() : PyLong_FromLong(st);
    END_HANDLE_TH_ERRORS
}

// (kind, weight, bias, eps) with kind "rms" or "layer", or None
patch_norm norm_spec(PyObject *spec, int64_t C, c10::Device dev, const char *name) {
    patch_norm s{PATCH_NORM_NONE, 0, nullptr, nullptr, 0.0f};
    if (spec == Py_None) return s;
    if (!PyTuple_Check(spec) || PyTuple_GET_SIZE(spec) != 4) refuse(name, " must be (kind, weight, bias, eps)");
    PyObject *kind = PyTuple_GET_ITEM(spec, 0);
    if (PyUnicode_Check(kind) && PyUnicode_CompareWithASCIIString(kind, "rms") == 0)
        s.kind = PATCH_NORM_RMS;
    else if (PyUnicode_Check(kind) && PyUnicode_CompareWithASCIIString(kind, "layer") == 0)
        s.kind = PATCH_NORM_LAYER;
    else
        refuse(name, ": the kind is \"rms\" or \"layer\"");
    const at::Tensor *w = tensor(PyTuple_GET_ITEM(spec, 1), name), *b = tensor(PyTuple_GET_ITEM(spec, 2), name);
    if (w && b && w->scalar_type() != b->scalar_type()) refuse(name, ": weight and bias must have one dtype");
    s.weight = vector(w, C, dev, name);
    s.bias = vector(b, C, dev, name);
    s.is_fp32 = is_fp32(w) || is_fp32(b);
    s.eps = static_cast<float>(PyFloat_AsDouble(PyTuple_GET_ITEM(spec, 3)));
    if (PyErr_Occurred()) throw python_error();
    return s;
}

// block_norm(branch, residual, gate, scale, post, pre, z_type, want_h, h_fp32, out_h, out_z)
// -> (h or None, z or None, scales or None)
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 11) refuse("block_norm: 11 arguments");
    const at::Tensor *branch = tensor(a[0], "branch"), *res = tensor(a[1], "residual"), *gate = tensor(a[2], "gate");
    const c10::Device dev = device_of(branch, "branch");
    if (branch->dim() != 2) refuse("branch must be [M, C]");
    const int64_t M = branch->size(0), C = branch->size(1);
    patch_block_norm_args p = {};
    p.scale = static_cast<float>(PyFloat_AsDouble(a[3]));
    p.z_type = static_cast<int32_t>(PyLong_AsLong(a[6]));
    const bool want_h = PyObject_IsTrue(a[7]) == 1;
    p.h_is_fp32 = PyObject_IsTrue(a[8]) == 1;
    if (PyErr_Occurred()) throw python_error();
    at::Tensor fresh;
    THPObjectPtr h, z, scales;
    if (want_h)
        h = THPObjectPtr(output(a[9], M, C, p.h_is_fp32 ? at::kFloat : at::kBFloat16, dev, "out_h", &fresh, &p.h,
                                &p.h_stride));
    else if (a[9] != Py_None)
        refuse("out_h without want_h");
    if (p.z_type != PATCH_Z_NONE) {
        const at::ScalarType type = p.z_type == PATCH_Z_BF16 ? at::kBFloat16 : p.z_type == PATCH_Z_FP32 ? at::kFloat : at::kByte;
        z = THPObjectPtr(output(a[10], M, C, type, dev, "out_z", &fresh, &p.z, &p.z_stride));
        if (p.z_type == PATCH_Z_E4M3) {
            at::Tensor s = empty({M}, at::kFloat, dev);
            p.z_scales = s.mutable_data_ptr<float>();
            scales = THPObjectPtr(THPVariable_Wrap(s));
        }
    } else if (a[10] != Py_None) {
        refuse("out_z without a pre norm");
    }
    p.branch = rows(branch, M, C, dev, "branch", &p.branch_stride, is_real);
    p.residual = rows(res, M, C, dev, "residual", &p.residual_stride, is_real);
    p.gate_tokens = 1;
    if (gate) {
        const int64_t R = gate->dim() == 2 ? gate->size(0) : 1;
        if (R < 1 || M % R != 0) refuse("gate has ", R, " rows, which do not divide ", M, " tokens");
        if (gate->dim() == 2)
            p.gate = rows(gate, R, C, dev, "gate", &p.gate_stride, is_real);
        else
            p.gate = vector(gate, C, dev, "gate");
        p.gate_tokens = M / R > 1 ? M / R : 1;
    }
    p.post = norm_spec(a[4], C, dev, "post");
    p.pre = norm_spec(a[5], C, dev, "pre");
    p.branch_is_fp32 = is_fp32(branch);
    p.residual_is_fp32 = is_fp32(res);
    p.gate_is_fp32 = is_fp32(gate);
    void *stream = current_stream(dev);
    const patch_status st = without_gil([&] { return g_norm(&p, M, C, stream); });
    if (st != PATCH_OK) return PyLong_FromLong(st);
    PyObject *r = PyTuple_New(3);
    if (!r) throw python_error();
    auto put = [r](Py_ssize_t i, THPObjectPtr &o) {
        if (!o) Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, i, o ? o.release() : Py_None);
    };
    put(0, h);
    put(1, z);
    put(2, scales);
    return r;
    END_HANDLE_TH_ERRORS
}

// bind(address of patch_hybrid_linear_group, of patch_hybrid_gated, of patch_block_norm)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 3) refuse("bind: 3 arguments");
    g_linear = reinterpret_cast<decltype(g_linear)>(PyLong_AsVoidPtr(a[0]));
    g_gated = reinterpret_cast<decltype(g_gated)>(PyLong_AsVoidPtr(a[1]));
    g_norm = reinterpret_cast<decltype(g_norm)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) throw python_error();
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                           {"linear", fast(linear), METH_FASTCALL, nullptr},
                           {"gated", fast(gated), METH_FASTCALL, nullptr},
                           {"block_norm", fast(block_norm), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_patch_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__patch_torch(void) {
    PyObject *m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", PATCH_BUILT_FOR) != 0) Py_CLEAR(m);
    return m;
}
