// ops_binding.cpp: the Python side of include/based_ops.h (argument marshalling only).
//
// A single-token call takes the GPU one to three microseconds, and reading a dozen tensors'
// metadata through Python and ctypes takes the host ten. So these functions read it from the
// tensors themselves: check it, allocate what the caller did not pass, and call the C functions
// of libbased_gb300.so on the current stream of the inputs' device. linear_attention_gb300/ops.py
// declares them, with their defaults and documentation.
#include <Python.h>
// torch after Python
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/based_ops.h"

namespace {

using at::ScalarType;
using at::Tensor;
using Sizes = c10::IntArrayRef;

struct Refusal {};  // a Python exception is set

[[noreturn]] void refuse(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Refusal();
}

const char *name_of(ScalarType t) { return c10::toString(t); }
std::string shape_of(Sizes s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
// NULL for None
const Tensor *optional_tensor(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

int type_code(ScalarType t, const char *what) {
    switch (t) {
        case ScalarType::Float: return BASED_F32;
        case ScalarType::BFloat16: return BASED_BF16;
        case ScalarType::Half: return BASED_F16;
        default: refuse(PyExc_TypeError, std::string(what) + " must be float32, bfloat16 or float16, got " + name_of(t));
    }
}
ScalarType dtype_arg(PyObject *o) {
    if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "expected a torch.dtype");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}
int choice(PyObject *o, const char *what, std::initializer_list<std::pair<const char *, int>> table) {
    if (PyUnicode_Check(o))
        for (const auto &e : table)
            if (PyUnicode_CompareWithASCIIString(o, e.first) == 0) return e.second;
    std::string names;
    for (const auto &e : table) names += (names.empty() ? "" : ", ") + std::string(e.first);
    refuse(PyExc_ValueError, std::string(what) + " must be one of " + names);
}
int mode_arg(PyObject *o) { return choice(o, "mode", {{"sigmoid", BASED_GATE_SIGMOID}, {"log", BASED_GATE_LOG}}); }
int act_arg(PyObject *o) {
    return choice(o, "act", {{"silu", BASED_ACT_SILU}, {"sigmoid", BASED_ACT_SIGMOID}, {"none", BASED_ACT_NONE}});
}
int64_t int_arg(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refusal();
    return v;
}
// an int of the C functions; what does not fit becomes a size that they refuse
int small(int64_t v) { return v > INT32_MAX || v < INT32_MIN ? -1 : static_cast<int>(v); }
double float_arg(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refusal();
    return v;
}

// t is a CUDA tensor of this shape and type on this device whose last axis has stride 1.
void input(const Tensor &t, const char *name, Sizes shape, ScalarType type, int dev) {
    if (!t.is_cuda() || t.get_device() != dev)
        refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the device of the other inputs");
    if (t.layout() != c10::kStrided) refuse(PyExc_ValueError, std::string(name) + " must be a dense tensor");
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_of(shape) + ", got " + shape_of(t.sizes()));
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
    if (t.stride(-1) != 1 && t.size(-1) != 1 && t.numel() != 0)
        refuse(PyExc_ValueError, "the last axis of " + std::string(name) + " must have stride 1");
}
// The address of a contiguous tensor of this shape and type; NULL for none.
void *whole(const Tensor *t, const char *name, Sizes shape, ScalarType type, int dev) {
    if (!t) return nullptr;
    if (t->scalar_type() != type)
        refuse(PyExc_TypeError, std::string(name) + " must be " + name_of(type) + ", got " + name_of(t->scalar_type()));
    if (!t->is_cuda() || t->get_device() != dev || t->sizes() != shape || !t->is_contiguous())
        refuse(PyExc_ValueError, std::string(name) + " must be a contiguous " + name_of(type) + " CUDA tensor of shape " + shape_of(shape));
    return t->data_ptr();
}

// t (..., C) as rows: their number and common stride.
struct Rows {
    int64_t n = 1, stride = 0;
    Rows(const Tensor &t, const char *name) {
        // from the last leading axis up: an axis of more than one row continues the one below it
        bool any = false;
        for (int64_t i = t.dim() - 2; i >= 0; --i) {
            const int64_t size = t.size(i);
            if (size != 1) {
                if (!any)
                    stride = t.stride(i);
                else if (t.stride(i) != stride * n && t.numel() != 0)
                    refuse(PyExc_ValueError, "the leading axes of " + std::string(name) + " must have one common stride");
                any = true;
            }
            n *= size;
        }
        if (!any) stride = t.dim() ? t.size(-1) : 0;  // one row
    }
};

// Device and stream of a call. On a side stream, what the call allocates comes from that stream's pool.
struct Place {
    int dev;
    std::optional<c10::cuda::CUDAGuard> device;
    std::optional<c10::cuda::CUDAStreamGuard> side;
    cudaStream_t stream = nullptr;

    // Tensors are checked to be CUDA ones first: nothing here touches a device for host tensors.
    Place(const Tensor &t, const char *name, PyObject *s) {
        if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
        dev = t.get_device();
        if (c10::cuda::current_device() != dev) device.emplace(static_cast<c10::DeviceIndex>(dev));
        if (s == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
            return;
        }
        int64_t v[3];
        const char *const attr[3] = {"stream_id", "device_index", "device_type"};
        for (int i = 0; i < 3; ++i) {
            PyObject *a = PyObject_GetAttrString(s, attr[i]);
            if (!a) throw Refusal();
            v[i] = PyLong_AsLongLong(a);
            Py_DECREF(a);
            if (v[i] == -1 && PyErr_Occurred()) throw Refusal();
        }
        if (v[1] != dev) refuse(PyExc_ValueError, "stream must be one of the inputs' device");
        const auto st = c10::cuda::CUDAStream::unpack3(v[0], static_cast<c10::DeviceIndex>(v[1]), static_cast<c10::DeviceType>(v[2]));
        side.emplace(st);
        stream = st.stream();
    }
    Tensor empty(Sizes shape, ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev))));
    }
    // the tensor that was passed, checked, or a new one
    Tensor output(PyObject *given, const char *name, Sizes shape, ScalarType type) const {
        if (given == Py_None) return empty(shape, type);
        const Tensor &t = tensor(given, name);
        whole(&t, name, shape, type, dev);
        return t;
    }
    based_stream_t raw() const { return reinterpret_cast<based_stream_t>(stream); }
};

PyObject *g_check;  // the function that raises for a return code

void check(int rc, const char *what) {
    if (rc == 0) return;
    PyObject *r = PyObject_CallFunction(g_check, "is", rc, what);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
    throw Refusal();
}

// The value of an output that no row or token adds to: `from`, or zero.
void settle(const Tensor &to, const Tensor *from) {
    if (!from)
        to.zero_();
    else if (from->data_ptr() != to.data_ptr())
        to.copy_(*from);
}

PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject *none() { return Py_NewRef(Py_None); }
PyObject *wrap_or_none(Tensor t) { return t.defined() ? wrap(std::move(t)) : none(); }
// a tuple of new references
template <typename... P>
PyObject *tuple(P... p) {
    PyObject *items[] = {p...};
    PyObject *t = PyTuple_New(sizeof...(p));
    for (size_t i = 0; i < sizeof...(p); ++i) PyTuple_SET_ITEM(t, i, items[i]);
    return t;
}

constexpr ScalarType kF32 = ScalarType::Float;

int64_t saved_rows(int64_t T) { return (T + BASED_SCAN_SAVE_ROWS - 1) / BASED_SCAN_SAVE_ROWS; }

// gate, x, mode, state, lengths, save, out, final_state, stream
PyObject *scan_fwd(PyObject *const *a) {
    const Tensor &gate = tensor(a[0], "gate"), &x = tensor(a[1], "x");
    if (x.dim() != 3) refuse(PyExc_ValueError, "expected gate and x of shape (B,T,D)");
    const ScalarType type = x.scalar_type();
    const int code = type_code(type, "x"), mode = mode_arg(a[2]);
    const Place at(x, "x", a[8]);
    const Sizes shape = x.sizes();
    const int64_t B = shape[0], T = shape[1], D = shape[2];
    input(x, "x", shape, type, at.dev);
    input(gate, "gate", shape, type, at.dev);
    const int save = PyObject_IsTrue(a[5]);
    if (save < 0) throw Refusal();
    void *state = whole(optional_tensor(a[3], "state"), "state", {B, D}, kF32, at.dev);
    void *lengths = whole(optional_tensor(a[4], "lengths"), "lengths", {B}, ScalarType::Int, at.dev);
    const Tensor y = at.output(a[6], "out", shape, type), last = at.output(a[7], "final_state", {B, D}, kF32);
    Tensor saved;
    if (save) saved = at.empty({B, saved_rows(T), D}, kF32);
    if ((B == 0 || T == 0) && D > 0) {  // the C functions take at least one row
        settle(last, optional_tensor(a[3], "state"));
        return tuple(wrap(y), wrap(last), wrap_or_none(saved));
    }
    check(based_scan_fwd(gate.data_ptr(), gate.stride(0), gate.stride(1), x.data_ptr(), x.stride(0), x.stride(1), small(B),
                         small(T), small(D), code, mode, static_cast<float *>(state), static_cast<int32_t *>(lengths),
                         y.data_ptr(), static_cast<float *>(last.data_ptr()),
                         save ? static_cast<float *>(saved.data_ptr()) : nullptr, at.raw()),
          "based_scan_fwd");
    return tuple(wrap(y), wrap(last), wrap_or_none(saved));
}

// gate, x, dy, saved, mode, dfinal, lengths, stream
PyObject *scan_bwd(PyObject *const *a) {
    const Tensor &gate = tensor(a[0], "gate"), &x = tensor(a[1], "x"), &dy = tensor(a[2], "dy");
    if (x.dim() != 3) refuse(PyExc_ValueError, "expected gate, x and dy of shape (B,T,D)");
    const ScalarType type = x.scalar_type();
    const int code = type_code(type, "x"), mode = mode_arg(a[4]);
    const Place at(x, "x", a[7]);
    const Sizes shape = x.sizes();
    const int64_t B = shape[0], T = shape[1], D = shape[2];
    input(x, "x", shape, type, at.dev);
    input(gate, "gate", shape, type, at.dev);
    input(dy, "dy", shape, type, at.dev);
    if (a[3] == Py_None) refuse(PyExc_ValueError, "based_scan_bwd needs the saved states of based_scan_fwd(..., save=True)");
    void *saved = whole(&tensor(a[3], "saved"), "saved", {B, saved_rows(T), D}, kF32, at.dev);
    void *dfinal = whole(optional_tensor(a[5], "dfinal"), "dfinal", {B, D}, kF32, at.dev);
    void *lengths = whole(optional_tensor(a[6], "lengths"), "lengths", {B}, ScalarType::Int, at.dev);
    const Tensor dgate = at.empty(shape, type), dx = at.empty(shape, type), dstate = at.empty({B, D}, kF32);
    if ((B == 0 || T == 0) && D > 0) {
        settle(dstate, optional_tensor(a[5], "dfinal"));
        return tuple(wrap(dgate), wrap(dx), wrap(dstate));
    }
    check(based_scan_bwd(gate.data_ptr(), gate.stride(0), gate.stride(1), x.data_ptr(), x.stride(0), x.stride(1),
                         dy.data_ptr(), dy.stride(0), dy.stride(1), static_cast<float *>(saved), small(B), small(T), small(D),
                         code, mode, static_cast<float *>(dfinal), static_cast<int32_t *>(lengths), dgate.data_ptr(),
                         dx.data_ptr(), static_cast<float *>(dstate.data_ptr()), at.raw()),
          "based_scan_bwd");
    return tuple(wrap(dgate), wrap(dx), wrap(dstate));
}

// gate, x, pool, mode, slots, out, stream
PyObject *scan_step(PyObject *const *a) {
    const Tensor &gate = tensor(a[0], "gate"), &x = tensor(a[1], "x"), &pool = tensor(a[2], "pool");
    if (x.dim() != 2 || pool.dim() != 2) refuse(PyExc_ValueError, "expected gate and x of shape (N,D) and pool of shape (S,D)");
    const ScalarType type = x.scalar_type();
    const int code = type_code(type, "x"), mode = mode_arg(a[3]);
    const Place at(x, "x", a[6]);
    const Sizes shape = x.sizes();
    const int64_t N = shape[0], D = shape[1], S = pool.size(0);
    input(x, "x", shape, type, at.dev);
    input(gate, "gate", shape, type, at.dev);
    void *states = whole(&pool, "pool", {S, D}, kF32, at.dev);
    void *slots = whole(optional_tensor(a[4], "slots"), "slots", {N}, ScalarType::Int, at.dev);
    const Tensor y = at.output(a[5], "out", shape, type);
    if (N == 0 && D > 0) return wrap(y);
    check(based_scan_step(gate.data_ptr(), gate.stride(0), x.data_ptr(), x.stride(0), small(N), small(D), small(S), code, mode,
                          static_cast<float *>(states), static_cast<int32_t *>(slots), y.data_ptr(), at.raw()),
          "based_scan_step");
    return wrap(y);
}

// weight and bias (C), which share a type
struct NormParams {
    int code;
    void *weight, *bias;
    const Tensor *w, *b;
    NormParams(PyObject *pw, PyObject *pb, int64_t C, ScalarType none, int dev) {
        w = optional_tensor(pw, "weight"), b = optional_tensor(pb, "bias");
        const ScalarType type = w ? w->scalar_type() : b ? b->scalar_type() : none;
        code = type_code(type, "weight and bias");
        weight = whole(w, "weight", {C}, type, dev);
        bias = whole(b, "bias", {C}, type, dev);
    }
};

// x, groups, weight, bias, gate, act, eps, out_dtype, out, stream
PyObject *norm_fwd(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x"), *gate = optional_tensor(a[4], "gate");
    if (x.dim() < 1) refuse(PyExc_ValueError, "expected x of shape (..., C)");
    const ScalarType xtype = x.scalar_type();
    const ScalarType type = gate ? gate->scalar_type() : a[7] != Py_None ? dtype_arg(a[7]) : xtype;
    if (a[7] != Py_None && dtype_arg(a[7]) != type)
        refuse(PyExc_TypeError, std::string("the output has the type of gate, ") + name_of(type));
    const int code = type_code(type, "the output"), xcode = type_code(xtype, "x"), act = act_arg(a[5]);
    const int64_t groups = int_arg(a[1]), C = x.size(-1);
    const float eps = static_cast<float>(float_arg(a[6]));
    const Place at(x, "x", a[9]);
    input(x, "x", x.sizes(), xtype, at.dev);
    if (gate) input(*gate, "gate", x.sizes(), type, at.dev);
    const Rows rx(x, "x"), rg(gate ? *gate : x, "gate");
    const NormParams par(a[2], a[3], C, type, at.dev);
    const Tensor y = at.output(a[8], "out", x.sizes(), type);
    if (rx.n == 0 && C > 0) return wrap(y);
    check(based_norm_fwd(x.data_ptr(), rx.stride, xcode, gate ? gate->data_ptr() : nullptr, rg.stride, par.weight, par.bias,
                         par.code, rx.n, small(C), small(groups), eps, act, y.data_ptr(), code, at.raw()),
          "based_norm_fwd");
    return wrap(y);
}

// What a call needs and was not passed, as bytes of a tensor.
Tensor workspace(PyObject *given, size_t bytes, const Place &at) {
    if (given == Py_None) return at.empty({static_cast<int64_t>(bytes)}, ScalarType::Byte);
    const Tensor &t = tensor(given, "workspace");
    if (!t.is_cuda() || t.get_device() != at.dev || !t.is_contiguous())
        refuse(PyExc_ValueError, "workspace must be a contiguous CUDA tensor on the device of the inputs");
    return t;
}

// dy, x, groups, weight, bias, gate, act, eps, workspace, stream
PyObject *norm_bwd(PyObject *const *a) {
    const Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), *gate = optional_tensor(a[5], "gate");
    if (x.dim() < 1) refuse(PyExc_ValueError, "expected x of shape (..., C)");
    const ScalarType xtype = x.scalar_type(), type = dy.scalar_type();
    const int code = type_code(type, "dy"), xcode = type_code(xtype, "x"), act = act_arg(a[6]);
    const int64_t groups = int_arg(a[2]), C = x.size(-1);
    const float eps = static_cast<float>(float_arg(a[7]));
    const Place at(x, "x", a[9]);
    const Sizes shape = x.sizes();
    input(x, "x", shape, xtype, at.dev);
    input(dy, "dy", shape, type, at.dev);
    if (gate) input(*gate, "gate", shape, type, at.dev);
    const Rows rx(x, "x"), rd(dy, "dy"), rg(gate ? *gate : x, "gate");
    const NormParams par(a[3], a[4], C, type, at.dev);
    const Tensor dx = at.empty(shape, xtype);
    Tensor dgate, dweight, dbias, ws;
    if (gate) dgate = at.empty(shape, type);
    if (par.w) dweight = at.empty({C}, par.w->scalar_type());
    if (par.b) dbias = at.empty({C}, par.b->scalar_type());
    if (rx.n == 0 && C > 0) {
        if (par.w) settle(dweight, nullptr);
        if (par.b) settle(dbias, nullptr);
        return tuple(wrap(dx), wrap_or_none(dgate), wrap_or_none(dweight), wrap_or_none(dbias));
    }
    const bool sums = par.w || par.b;
    if (sums) ws = workspace(a[8], a[8] == Py_None ? based_norm_bwd_workspace_size(rx.n, small(C), small(groups)) : 0, at);
    check(based_norm_bwd(dy.data_ptr(), rd.stride, x.data_ptr(), rx.stride, xcode, gate ? gate->data_ptr() : nullptr, rg.stride,
                         par.weight, par.bias, par.code, rx.n, small(C), small(groups), eps, act, dx.data_ptr(),
                         gate ? dgate.data_ptr() : nullptr, par.w ? dweight.data_ptr() : nullptr,
                         par.b ? dbias.data_ptr() : nullptr, code, sums ? ws.data_ptr() : nullptr, sums ? ws.nbytes() : 0,
                         at.raw()),
          "based_norm_bwd");
    return tuple(wrap(dx), wrap_or_none(dgate), wrap_or_none(dweight), wrap_or_none(dbias));
}

// whether ids are 64 bits wide
int ids_type(const Tensor &ids) {
    if (ids.scalar_type() != ScalarType::Int && ids.scalar_type() != ScalarType::Long)
        refuse(PyExc_TypeError, std::string("ids must be int32 or int64, got ") + name_of(ids.scalar_type()));
    return ids.scalar_type() == ScalarType::Long;
}
// ids in order, as a copy where they are strided (ids[:, :-1] of a batch)
Tensor ids_in_order(const Tensor &ids, int dev) {
    if (!ids.is_cuda() || ids.get_device() != dev)
        refuse(PyExc_ValueError, "ids must be a CUDA tensor on the device of the other inputs");
    return ids.contiguous();
}
// the shape of ids with one more axis
c10::SmallVector<int64_t, 6> with_channels(const Tensor &ids, int64_t D) {
    c10::SmallVector<int64_t, 6> s(ids.sizes().begin(), ids.sizes().end());
    s.push_back(D);
    return s;
}

// ids, table, scale, out, stream
PyObject *embed_fwd(PyObject *const *a) {
    const Tensor &given = tensor(a[0], "ids"), &table = tensor(a[1], "table");
    if (table.dim() != 2) refuse(PyExc_ValueError, "expected a table of shape (V,D)");
    const ScalarType type = table.scalar_type();
    const int code = type_code(type, "table"), wide = ids_type(given);
    const float scale = static_cast<float>(float_arg(a[2]));
    const Place at(table, "table", a[4]);
    const int64_t V = table.size(0), D = table.size(1);
    const Tensor ids = ids_in_order(given, at.dev);
    input(table, "table", table.sizes(), type, at.dev);
    const Tensor y = at.output(a[3], "out", with_channels(ids, D), type);
    if (ids.numel() == 0 && V > 0 && D > 0) return wrap(y);
    check(based_embed_fwd(ids.data_ptr(), wide, table.data_ptr(), table.stride(0), ids.numel(), small(V), small(D), code, scale,
                          y.data_ptr(), at.raw()),
          "based_embed_fwd");
    return wrap(y);
}

// ids, dy, rows, scale, dtype, out, workspace, stream
PyObject *embed_bwd(PyObject *const *a) {
    const Tensor &given = tensor(a[0], "ids"), &dy = tensor(a[1], "dy");
    if (dy.dim() < 1) refuse(PyExc_ValueError, "expected dy of shape (..., D)");
    const ScalarType type = dtype_arg(a[4]);
    const int code = type_code(dy.scalar_type(), "dy"), gcode = type_code(type, "the gradient"), wide = ids_type(given);
    const int64_t V = int_arg(a[2]), D = dy.size(-1), N = given.numel();
    const float scale = static_cast<float>(float_arg(a[3]));
    const Place at(dy, "dy", a[7]);
    const Tensor ids = ids_in_order(given, at.dev);
    input(dy, "dy", with_channels(ids, D), dy.scalar_type(), at.dev);
    const Rows rd(dy, "dy");
    if (V < 0) refuse(PyExc_ValueError, "rows must not be negative");
    const Tensor dtable = at.output(a[5], "out", {V, D}, type);
    if (N == 0 && V > 0 && D > 0) {
        settle(dtable, nullptr);
        return wrap(dtable);
    }
    const Tensor ws = workspace(a[6], a[6] == Py_None ? based_embed_bwd_workspace_size(N, small(V), small(D)) : 0, at);
    check(based_embed_bwd(ids.data_ptr(), wide, dy.data_ptr(), rd.stride, N, small(V), small(D), code, scale, dtable.data_ptr(),
                          gcode, ws.data_ptr(), ws.nbytes(), at.raw()),
          "based_embed_bwd");
    return wrap(dtable);
}

// q, k (..., HK, K) and v (..., H, V) of one type, beta and gate (..., H)
struct DeltaInputs {
    const Tensor &q, &k, &v, &beta, *gate;
    int code;
    ScalarType type;
    int64_t H, HK, K, V;
    DeltaInputs(PyObject *const *a, int dims)
        : q(tensor(a[0], "q")), k(tensor(a[1], "k")), v(tensor(a[2], "v")), beta(tensor(a[3], "beta")), gate(optional_tensor(a[4], "gate")) {
        if (q.dim() != dims || v.dim() != dims)
            refuse(PyExc_ValueError, dims == 4 ? "expected q and k of shape (B,T,HK,K) and v of shape (B,T,H,V)"
                                               : "expected q and k of shape (N,HK,K) and v of shape (N,H,V)");
        type = v.scalar_type(), code = type_code(type, "v");
        H = v.size(dims - 2), V = v.size(dims - 1), HK = q.size(dims - 2), K = q.size(dims - 1);
    }
    void check(int dev) const {
        c10::SmallVector<int64_t, 4> keys(v.sizes().begin(), v.sizes().end()), heads(v.sizes().begin(), v.sizes().end() - 1);
        keys[keys.size() - 2] = HK, keys[keys.size() - 1] = K;
        input(v, "v", v.sizes(), type, dev);
        input(q, "q", keys, type, dev);
        input(k, "k", keys, type, dev);
        input(beta, "beta", heads, type, dev);
        if (gate) input(*gate, "gate", heads, type, dev);
    }
    const void *gate_data() const { return gate ? gate->data_ptr() : nullptr; }
    int64_t gate_stride(int i) const { return gate ? gate->stride(i) : 0; }
};
// a scale; None selects the default
float scale_arg(PyObject *o) { return o == Py_None ? 0.0f : static_cast<float>(float_arg(o)); }

// q, k, v, beta, gate, scale, state, lengths, save, out, final_state, workspace, stream
PyObject *delta_fwd(PyObject *const *a) {
    const DeltaInputs in(a, 4);
    const float scale = scale_arg(a[5]);
    const Place at(in.v, "v", a[12]);
    in.check(at.dev);
    const int64_t B = in.v.size(0), T = in.v.size(1), H = in.H, K = in.K, V = in.V;
    const int save = PyObject_IsTrue(a[8]);
    if (save < 0) throw Refusal();
    void *state = whole(optional_tensor(a[6], "state"), "state", {B, H, K, V}, kF32, at.dev);
    void *lengths = whole(optional_tensor(a[7], "lengths"), "lengths", {B}, ScalarType::Int, at.dev);
    const Tensor o = at.output(a[9], "out", in.v.sizes(), in.type), last = at.output(a[10], "final_state", {B, H, K, V}, kF32);
    Tensor saved;
    if (save) saved = at.empty({static_cast<int64_t>(based_delta_saved_size(small(B), small(T), small(H), small(K), small(V), in.code))}, ScalarType::Byte);
    const auto result = [&] {
        return tuple(wrap(o), wrap(last), wrap_or_none(saved));
    };
    if ((B == 0 || T == 0) && H > 0 && K > 0 && V > 0) {
        settle(last, optional_tensor(a[6], "state"));
        return result();
    }
    const Tensor ws = workspace(a[11], a[11] == Py_None ? based_delta_workspace_size(small(B), small(T), small(H), small(in.HK), small(K), small(V), in.code, 0) : 0, at);
    check(based_delta_fwd(in.q.data_ptr(), in.q.stride(0), in.q.stride(1), in.q.stride(2), in.k.data_ptr(), in.k.stride(0), in.k.stride(1),
                          in.k.stride(2), in.v.data_ptr(), in.v.stride(0), in.v.stride(1), in.v.stride(2), in.beta.data_ptr(),
                          in.beta.stride(0), in.beta.stride(1), in.gate_data(), in.gate_stride(0), in.gate_stride(1), small(B), small(T),
                          small(H), small(in.HK), small(K), small(V), in.code, scale, static_cast<float *>(state),
                          static_cast<int32_t *>(lengths), o.data_ptr(), static_cast<float *>(last.data_ptr()),
                          save ? saved.data_ptr() : nullptr, ws.data_ptr(), ws.nbytes(), at.raw()),
          "based_delta_fwd");
    return result();
}

// q, k, v, beta, gate, dout, saved, scale, dfinal, lengths, workspace, stream
PyObject *delta_bwd(PyObject *const *a) {
    const DeltaInputs in(a, 4);
    const Tensor &dout = tensor(a[5], "dout");
    const float scale = scale_arg(a[7]);
    const Place at(in.v, "v", a[11]);
    in.check(at.dev);
    input(dout, "dout", in.v.sizes(), in.type, at.dev);
    const int64_t B = in.v.size(0), T = in.v.size(1), H = in.H, K = in.K, V = in.V;
    if (a[6] == Py_None) refuse(PyExc_ValueError, "based_delta_bwd needs what based_delta_fwd(..., save=True) saved");
    void *saved = whole(&tensor(a[6], "saved"), "saved", {static_cast<int64_t>(based_delta_saved_size(small(B), small(T), small(H), small(K), small(V), in.code))},
                        ScalarType::Byte, at.dev);
    void *dfinal = whole(optional_tensor(a[8], "dfinal"), "dfinal", {B, H, K, V}, kF32, at.dev);
    void *lengths = whole(optional_tensor(a[9], "lengths"), "lengths", {B}, ScalarType::Int, at.dev);
    const Tensor dq = at.empty(in.q.sizes(), in.type), dk = at.empty(in.q.sizes(), in.type), dv = at.empty(in.v.sizes(), in.type),
                 dbeta = at.empty({B, T, H}, in.type), dstate = at.empty({B, H, K, V}, kF32);
    Tensor dgate;
    if (in.gate) dgate = at.empty({B, T, H}, in.type);
    const auto result = [&] { return tuple(wrap(dq), wrap(dk), wrap(dv), wrap(dbeta), wrap_or_none(dgate), wrap(dstate)); };
    if ((B == 0 || T == 0) && H > 0 && K > 0 && V > 0) {
        settle(dstate, optional_tensor(a[8], "dfinal"));
        return result();
    }
    const Tensor ws = workspace(a[10], a[10] == Py_None ? based_delta_workspace_size(small(B), small(T), small(H), small(in.HK), small(K), small(V), in.code, 1) : 0, at);
    check(based_delta_bwd(in.q.data_ptr(), in.q.stride(0), in.q.stride(1), in.q.stride(2), in.k.data_ptr(), in.k.stride(0), in.k.stride(1),
                          in.k.stride(2), in.v.data_ptr(), in.v.stride(0), in.v.stride(1), in.v.stride(2), in.beta.data_ptr(),
                          in.beta.stride(0), in.beta.stride(1), in.gate_data(), in.gate_stride(0), in.gate_stride(1), dout.data_ptr(),
                          dout.stride(0), dout.stride(1), dout.stride(2), saved, small(B), small(T), small(H), small(in.HK), small(K), small(V), in.code, scale, static_cast<float *>(dfinal),
                          static_cast<int32_t *>(lengths), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dbeta.data_ptr(),
                          in.gate ? dgate.data_ptr() : nullptr, static_cast<float *>(dstate.data_ptr()), ws.data_ptr(), ws.nbytes(), at.raw()),
          "based_delta_bwd");
    return result();
}

// q, k, v, beta, gate, pool, scale, slots, out, stream
PyObject *delta_step(PyObject *const *a) {
    const DeltaInputs in(a, 3);
    const Tensor &pool = tensor(a[5], "pool");
    if (pool.dim() != 4) refuse(PyExc_ValueError, "expected pool of shape (S,H,K,V)");
    const float scale = scale_arg(a[6]);
    const Place at(in.v, "v", a[9]);
    in.check(at.dev);
    const int64_t N = in.v.size(0), S = pool.size(0);
    void *states = whole(&pool, "pool", {S, in.H, in.K, in.V}, kF32, at.dev);
    void *slots = whole(optional_tensor(a[7], "slots"), "slots", {N}, ScalarType::Int, at.dev);
    const Tensor o = at.output(a[8], "out", in.v.sizes(), in.type);
    if (N == 0 && in.H > 0 && in.K > 0 && in.V > 0) return wrap(o);
    check(based_delta_step(in.q.data_ptr(), in.q.stride(0), in.q.stride(1), in.k.data_ptr(), in.k.stride(0), in.k.stride(1), in.v.data_ptr(),
                           in.v.stride(0), in.v.stride(1), in.beta.data_ptr(), in.beta.stride(0), in.gate_data(), in.gate_stride(0),
                           small(N), small(in.H), small(in.HK), small(in.K), small(in.V), small(S), in.code, scale,
                           static_cast<float *>(states), static_cast<int32_t *>(slots), o.data_ptr(), at.raw()),
          "based_delta_step");
    return wrap(o);
}

// x, weight, residual, eps, quantize, out, sum_out, stream
PyObject *rms_fwd(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x"), *weight = optional_tensor(a[1], "weight"), *residual = optional_tensor(a[2], "residual");
    if (x.dim() < 1) refuse(PyExc_ValueError, "expected x of shape (..., C)");
    const ScalarType type = x.scalar_type(), stype = residual ? residual->scalar_type() : type, ptype = weight ? weight->scalar_type() : type;
    const int code = type_code(type, "x"), scode = type_code(stype, "residual"), pcode = type_code(ptype, "weight");
    const int quantize = PyObject_IsTrue(a[4]);
    if (quantize < 0) throw Refusal();
    const int64_t C = x.size(-1);
    const float eps = static_cast<float>(float_arg(a[3]));
    const Place at(x, "x", a[7]);
    const Sizes shape = x.sizes();
    input(x, "x", shape, type, at.dev);
    if (residual) input(*residual, "residual", shape, stype, at.dev);
    void *w = whole(weight, "weight", {C}, ptype, at.dev);
    const Rows rx(x, "x"), rr(residual ? *residual : x, "residual");
    const Tensor y = at.output(a[5], "out", shape, quantize ? ScalarType::Float8_e4m3fn : type);
    Tensor sum, scales;
    if (residual) sum = at.output(a[6], "sum_out", shape, stype);
    if (!residual && a[6] != Py_None) refuse(PyExc_ValueError, "sum_out needs a residual");
    if (quantize) scales = at.empty(shape.slice(0, shape.size() - 1), kF32);
    if (rx.n > 0 || C == 0)
        check(based_rms_fwd(x.data_ptr(), rx.stride, residual ? residual->data_ptr() : nullptr, rr.stride, scode, w, pcode, rx.n, small(C), eps,
                            residual ? sum.data_ptr() : nullptr, y.data_ptr(), code, quantize ? static_cast<float *>(scales.data_ptr()) : nullptr,
                            at.raw()),
              "based_rms_fwd");
    PyObject *const total = residual ? wrap(sum) : Py_NewRef(a[0]);
    return tuple(wrap(y), total, wrap_or_none(scales));
}

// dy, s, weight, dsum, eps, workspace, stream
PyObject *rms_bwd(PyObject *const *a) {
    const Tensor &dy = tensor(a[0], "dy"), &s = tensor(a[1], "s"), *weight = optional_tensor(a[2], "weight"), *dsum = optional_tensor(a[3], "dsum");
    if (s.dim() < 1) refuse(PyExc_ValueError, "expected s of shape (..., C)");
    const ScalarType type = dy.scalar_type(), stype = s.scalar_type(), ptype = weight ? weight->scalar_type() : type;
    const int code = type_code(type, "dy"), scode = type_code(stype, "s"), pcode = type_code(ptype, "weight");
    const int64_t C = s.size(-1);
    const float eps = static_cast<float>(float_arg(a[4]));
    const Place at(s, "s", a[6]);
    const Sizes shape = s.sizes();
    input(s, "s", shape, stype, at.dev);
    input(dy, "dy", shape, type, at.dev);
    if (dsum) input(*dsum, "dsum", shape, stype, at.dev);
    void *w = whole(weight, "weight", {C}, ptype, at.dev);
    const Rows rs(s, "s"), rd(dy, "dy"), rg(dsum ? *dsum : s, "dsum");
    const Tensor ds = at.empty(shape, stype);
    Tensor dx, dweight, ws;
    if (type != stype) dx = at.empty(shape, type);
    if (weight) dweight = at.empty({C}, ptype);
    if (rs.n == 0 && C > 0) {
        if (weight) settle(dweight, nullptr);
    } else {
        if (weight) ws = workspace(a[5], a[5] == Py_None ? based_rms_bwd_workspace_size(rs.n, small(C)) : 0, at);
        check(based_rms_bwd(dy.data_ptr(), rd.stride, s.data_ptr(), rs.stride, scode, w, pcode, dsum ? dsum->data_ptr() : nullptr, rg.stride, rs.n,
                            small(C), eps, ds.data_ptr(), dx.defined() ? dx.data_ptr() : nullptr, weight ? dweight.data_ptr() : nullptr, code,
                            weight ? ws.data_ptr() : nullptr, weight ? ws.nbytes() : 0, at.raw()),
              "based_rms_bwd");
    }
    PyObject *const first = wrap(ds);
    return tuple(first, dx.defined() ? wrap(dx) : Py_NewRef(first), wrap_or_none(dweight));
}

// A number for all rows, or a tensor with one for each
struct PerRow {
    void *data = nullptr;
    double all = 0;
    PerRow(PyObject *o, const char *name, double none, int64_t N, ScalarType type, int dev) : all(none) {
        if (THPVariable_Check(o))
            data = whole(&THPVariable_Unpack(o), name, {N}, type, dev);
        else if (o != Py_None)
            all = float_arg(o);
    }
};

// logits, u, temperature, top_k, top_p, min_p, out, stream
PyObject *sample(PyObject *const *a) {
    const Tensor &logits = tensor(a[0], "logits"), &u = tensor(a[1], "u");
    if (logits.dim() != 2) refuse(PyExc_ValueError, "expected logits of shape (N,V)");
    const ScalarType type = logits.scalar_type();
    const int code = type_code(type, "logits");
    const int64_t N = logits.size(0), V = logits.size(1);
    const Place at(logits, "logits", a[7]);
    input(logits, "logits", logits.sizes(), type, at.dev);
    void *const random = whole(&u, "u", {N}, kF32, at.dev);
    const PerRow temperature(a[2], "temperature", 1.0, N, kF32, at.dev), top_k(a[3], "top_k", 0.0, N, ScalarType::Int, at.dev),
        top_p(a[4], "top_p", 1.0, N, kF32, at.dev), min_p(a[5], "min_p", 0.0, N, kF32, at.dev);
    if (!(top_k.all >= INT32_MIN && top_k.all <= INT32_MAX) || top_k.all != static_cast<int>(top_k.all)) refuse(PyExc_ValueError, "top_k must be a whole number");
    const Tensor tokens = at.output(a[6], "out", {N}, ScalarType::Int), probs = at.empty({N}, kF32);
    if (N > 0 || V == 0)
        check(based_sample(logits.data_ptr(), logits.stride(0), code, small(N), small(V), static_cast<float *>(random),
                           static_cast<float *>(temperature.data), static_cast<float>(temperature.all), static_cast<int32_t *>(top_k.data),
                           static_cast<int>(top_k.all), static_cast<float *>(top_p.data), static_cast<float>(top_p.all),
                           static_cast<float *>(min_p.data), static_cast<float>(min_p.all), static_cast<int32_t *>(tokens.data_ptr()),
                           static_cast<float *>(probs.data_ptr()), at.raw()),
              "based_sample");
    return tuple(wrap(tokens), wrap(probs));
}

// A Python function of COUNT positional arguments. Nothing is thrown past it: torch's errors (such
// as memory that cannot be had) become Python's.
template <PyObject *(*F)(PyObject *const *), int COUNT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != COUNT) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", COUNT, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refusal &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_check(PyObject *, PyObject *fn) {
    Py_XSETREF(g_check, Py_NewRef(fn));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int COUNT>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&entry<F, COUNT>)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<scan_fwd, 9>("scan_fwd"),
                           method<scan_bwd, 8>("scan_bwd"),
                           method<scan_step, 7>("scan_step"),
                           method<norm_fwd, 10>("norm_fwd"),
                           method<norm_bwd, 10>("norm_bwd"),
                           method<embed_fwd, 5>("embed_fwd"),
                           method<embed_bwd, 8>("embed_bwd"),
                           method<delta_fwd, 13>("delta_fwd"),
                           method<delta_bwd, 12>("delta_bwd"),
                           method<delta_step, 10>("delta_step"),
                           method<rms_fwd, 8>("rms_fwd"),
                           method<rms_bwd, 7>("rms_bwd"),
                           method<sample, 8>("sample"),
                           {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "based_ops_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_based_ops_binding() { return PyModule_Create(&g_module); }
