// Tensor-side marshalling of the decayed attention and the rotary embedding.
//
// A single-token call of these operators runs for a few microseconds, less than
// an argument-by-argument check in Python costs, so the checks of shapes, types,
// devices and overlaps, the allocation of outputs and the call into libblin's C
// functions are done here.  No part of the computation is.
//
// Every function takes its arguments by position (the Python wrappers give them
// names and defaults) and returns the output, or the C function's status as an
// int when that is not BLIN_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <string>
#include <vector>

#include "../../include/blin.h"

namespace {

using at::Tensor;

struct Refused {
    PyObject *type;
    std::string what;
};
[[noreturn]] void value_error(const std::string &w) { throw Refused{PyExc_ValueError, w}; }
[[noreturn]] void type_error(const std::string &w) { throw Refused{PyExc_TypeError, w}; }
[[noreturn]] void runtime_error(const std::string &w) { throw Refused{PyExc_RuntimeError, w}; }

std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + (v.size() == 1 ? ",)" : ")");
}

// A tensor with `dims` dimensions, each of which the library's ints can hold.
const Tensor &operand(PyObject *o, const char *name, int64_t dims, const char *shape) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
    const Tensor &t = THPVariable_Unpack(o);
    if (t.dim() != dims) value_error(std::string(name) + " must be a " + shape + " tensor");
    for (const int64_t n : t.sizes())
        if (n > INT32_MAX) value_error(std::string(name) + "'s dimensions must be below 2^31 (got " + text(t.sizes()) + ")");
    return t;
}
void same_kind(const Tensor &t, const char *name, at::IntArrayRef shape, const Tensor &as) {
    if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
    if (t.sizes() != shape || t.scalar_type() != as.scalar_type() || t.device() != as.device() || t.stride(-1) != 1)
        value_error(std::string(name) + " must be a " + at::toString(as.scalar_type()) + " tensor of shape " + text(shape) +
                    " on " + as.device().str() + ", last dimension contiguous (got " + at::toString(t.scalar_type()) + ", " +
                    text(t.sizes()) + ", " + t.device().str() + ", strides " + text(t.strides()) + ")");
}
blin_dtype dtype_of(const Tensor &t) {
    if (t.scalar_type() == at::kFloat) return BLIN_F32;
    if (t.scalar_type() == at::kBFloat16) return BLIN_BF16;
    type_error(std::string("unsupported dtype ") + at::toString(t.scalar_type()) + " (float32 or bfloat16)");
}
// The library launches on the current device: the call's tensors must live there.
void on_current_device(const Tensor &t) {
    const int cur = c10::cuda::current_device();
    if (t.device().index() != cur)
        value_error("tensors are on " + t.device().str() + " but the current device is cuda:" + std::to_string(cur) +
                    "; call under torch.cuda.device(...)");
}
// An optional contiguous tensor of a type and shape; NULL when it is None.
const void *optional(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const Tensor &as) {
    if (o == Py_None) return nullptr;
    if (THPVariable_Check(o)) {
        const Tensor &t = THPVariable_Unpack(o);
        if (t.scalar_type() == type && t.sizes() == shape && t.device() == as.device() && t.is_contiguous())
            return t.const_data_ptr();
    }
    value_error(std::string(name) + " must be a contiguous " + at::toString(type) + " tensor of shape " + text(shape) + " on " +
                as.device().str());
}
// Would autograd have to record an operation on this tensor?
bool recorded(const Tensor &t) { return at::GradMode::is_enabled() && t.requires_grad(); }
// Tells autograd that a call has written to a tensor of the caller's.
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
bool same_place(const Tensor &a, const Tensor &b) { return a.const_data_ptr() == b.const_data_ptr() && a.strides() == b.strides(); }
// An output must not overlap an input: contiguous tensors are compared by address range, strided views,
// which may interleave without sharing an element, only by start address.
void no_overlap(const Tensor &out, const Tensor &in) {
    const char *a = static_cast<const char *>(out.const_data_ptr()), *b = static_cast<const char *>(in.const_data_ptr());
    if (out.numel() == 0 || in.numel() == 0) return;
    if (a == b || (out.is_contiguous() && in.is_contiguous() && a < b + in.nbytes() && b < a + out.nbytes()))
        value_error("out must not overlap the inputs");
}
void check_out(const Tensor &out, const Tensor &like) {
    if (out.scalar_type() != like.scalar_type() || out.sizes() != like.sizes() || out.device() != like.device() ||
        out.stride(-1) != 1)
        value_error(std::string("out must be a ") + at::toString(like.scalar_type()) + " tensor of shape " + text(like.sizes()) +
                    " on " + like.device().str() + ", last dimension contiguous");
}
const Tensor &given_out(PyObject *o, const Tensor &like) {
    if (!THPVariable_Check(o)) value_error("out must be a tensor");
    const Tensor &t = THPVariable_Unpack(o);
    check_out(t, like);
    return t;
}
// [B, H, N, d], or [B, H, d], which has no token stride
blin_layout layout(const Tensor &t) {
    const auto s = t.strides();
    return blin_layout{t.dim() == 4 ? s[2] : t.size(-1), s[1], s[0]};
}

// The call's stream: the current one, or the handle that the wrapper hands over.  Memory that the call makes
// belongs to its stream (the current stream's may still be in use there by work that the call's does not wait
// for); what it returns is kept until the current stream, where it is most likely read, has also done with it.
// What the caller hands over is kept until the call's stream has done with it: on its own stream the memory of a
// tensor that goes out of use right after the call would be given away while the call may still read it.
class CallStream {
    c10::cuda::CUDAStream current_, used_;
    c10::cuda::OptionalCUDAStreamGuard guard_;

    static c10::cuda::CUDAStream chosen(PyObject *o, const c10::cuda::CUDAStream &current) {
        if (o == Py_None) return current;
        cudaStream_t s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
        if (PyErr_Occurred()) {
            PyErr_Clear();
            type_error("stream must be a torch.cuda.Stream");
        }
        return s == current.stream() ? current : c10::cuda::getStreamFromExternal(s, current.device_index());
    }

public:
    CallStream(PyObject *o, const Tensor &like)
        : current_(c10::cuda::getCurrentCUDAStream(like.device().index())), used_(chosen(o, current_)) {
        if (used_ != current_) guard_.reset_stream(used_);
    }
    cudaStream_t stream() const { return used_.stream(); }
    void keep(const Tensor &t) const {
        if (used_ != current_) t.record_stream(used_);
    }
    void keep(PyObject *o) const {
        if (o != Py_None) keep(THPVariable_Unpack(o));
    }
    Tensor output(at::IntArrayRef shape, const Tensor &like) const {
        Tensor t = at::empty(shape, like.options().memory_format(at::MemoryFormat::Contiguous));
        if (used_ != current_) t.record_stream(current_);
        return t;
    }
};
int64_t integer(PyObject *o, const char *name) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    if (v > INT32_MAX || v < INT32_MIN) value_error(std::string(name) + " is out of range");
    return v;
}
float number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be a number");
    }
    return static_cast<float>(v);
}
void integers(PyObject *o, const char *name, int *to, int n) {
    PyObject *seq = PySequence_Fast(o, "");
    if (seq == nullptr || PySequence_Fast_GET_SIZE(seq) != n) {
        Py_XDECREF(seq);
        PyErr_Clear();
        value_error(std::string(name) + " must hold " + std::to_string(n) + " integers");
    }
    struct Hold {
        PyObject *p;
        ~Hold() { Py_DECREF(p); }
    } hold{seq};
    for (int i = 0; i < n; ++i) to[i] = static_cast<int>(integer(PySequence_Fast_GET_ITEM(seq, i), name));
}
void expect_args(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}
// Runs the body; a refusal or a C++ exception becomes a Python one, torch's own those that torch makes of them.
template <typename F>
PyObject *guarded(F &&body) {
    try {
        return body();
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}
// What a prefill and a step share: q, k, v, log_decay, the pool and the slots.
struct Call {
    const Tensor &q, &k, &v;
    blin_dtype dt;
    int64_t B, H, d;
    const float *lg;
    float *pool = nullptr;
    int64_t slots = 0;
    const int *slot_of;
    const Tensor *state = nullptr;

    Call(PyObject *const *a, int64_t dims, const char *shape, PyObject *st, PyObject *sl)
        : q(operand(a[0], "q", dims, shape)), k(operand(a[1], "k", dims, shape)), v(operand(a[2], "v", dims, shape)) {
        dt = dtype_of(q);
        same_kind(q, "q", q.sizes(), q);
        same_kind(k, "k", q.sizes(), q);
        same_kind(v, "v", q.sizes(), q);
        on_current_device(q);
        B = q.size(0), H = q.size(1), d = q.size(-1);
        lg = static_cast<const float *>(optional(a[3], "log_decay", at::kFloat, {H}, q));
        if (lg == nullptr) value_error("log_decay is needed");
        if (st != Py_None) {
            state = THPVariable_Check(st) ? &THPVariable_Unpack(st) : nullptr;
            if (state == nullptr || state->dim() != 4 || state->scalar_type() != at::kFloat || state->size(1) != H ||
                state->size(2) != d || state->size(3) != d || state->device() != q.device() || !state->is_contiguous())
                value_error("state must be a contiguous float32 [slots, " + std::to_string(H) + ", " + std::to_string(d) + ", " +
                            std::to_string(d) + "] tensor on " + q.device().str());
            pool = static_cast<float *>(state->data_ptr());
            slots = state->size(0);
            if (slots < 1 || slots > INT32_MAX)  // an empty tensor has no address: it would pass for no state at all
                value_error("state must hold between 1 and 2^31 - 1 slots (got " + std::to_string(slots) + ")");
        }
        slot_of = static_cast<const int *>(optional(sl, "slots", at::kInt, {B}, q));
        if (recorded(q) || recorded(k) || recorded(v) || recorded(THPVariable_Unpack(a[3])) || (state && recorded(*state)))
            no_gradient();
    }
    [[noreturn]] static void no_gradient() {
        runtime_error("the decayed attention has no gradient: call it under torch.no_grad(), or with tensors that require none");
    }
    void keep(const CallStream &on, PyObject *lg, PyObject *sl) const {
        on.keep(q), on.keep(k), on.keep(v), on.keep(lg), on.keep(sl);
        if (state) on.keep(*state);
    }
    Tensor output(PyObject *o, const CallStream &on) const {
        if (o == Py_None) return on.output(q.sizes(), q);
        const Tensor &t = given_out(o, q);
        if (recorded(t)) no_gradient();
        no_overlap(t, q), no_overlap(t, k), no_overlap(t, v);
        if (state) no_overlap(t, *state);
        on.keep(t);
        return t;
    }
    bool dense(const Tensor &out) const {
        return q.is_contiguous() && k.is_contiguous() && v.is_contiguous() && out.is_contiguous();
    }
    // The output, or the status of a call that failed.
    PyObject *answer(blin_status rc, const Tensor &out, PyObject *given) const {
        if (rc != BLIN_OK) return PyLong_FromLong(rc);
        if (state) written(*state);
        if (given != Py_None) written(out);
        return THPVariable_Wrap(out);
    }
    blin_decay_layouts layouts(const Tensor &out) const { return {layout(q), layout(k), layout(v), layout(out)}; }
};

// q, k, v, log_decay, state, slots, lengths, scale, out, workspace, stream
PyObject *decay_prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        expect_args(n, 11);
        const Call c(a, 4, "[B, H, N, d]", a[4], a[5]);
        const int64_t N = c.q.size(2);
        const int *lengths = static_cast<const int *>(optional(a[6], "lengths", at::kInt, {c.B}, c.q));
        const CallStream on(a[10], c.q);
        c.keep(on, a[3], a[5]), on.keep(a[6]);
        const Tensor out = c.output(a[8], on);
        if (N == 0 && c.B > 0 && c.H > 0) return THPVariable_Wrap(out);  // no tokens: nothing to read, no address to give
        const size_t need = blin_decay_workspace_size((int)c.B, (int)c.H, (int)N, (int)c.d, c.dt);
        Tensor scratch;
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[9] != Py_None) {
            if (!THPVariable_Check(a[9])) value_error("workspace must be a tensor");
            const Tensor &w = THPVariable_Unpack(a[9]);
            if (w.device() != c.q.device() || !w.is_contiguous())
                value_error("workspace must be a contiguous tensor on " + c.q.device().str());
            on.keep(w);
            ws = w.data_ptr();
            ws_bytes = w.nbytes();
        } else if (need > 16) {
            scratch = at::empty({(int64_t)need}, c.q.options().dtype(at::kByte));
            ws = scratch.data_ptr();
            ws_bytes = need;
        }
        const blin_decay_layouts lay = c.layouts(out);
        const blin_status rc =
            blin_decay_prefill(c.q.const_data_ptr(), c.k.const_data_ptr(), c.v.const_data_ptr(), out.data_ptr(), c.dt, (int)c.B,
                               (int)c.H, (int)N, (int)c.d, c.lg, number(a[7], "scale"), c.dense(out) ? nullptr : &lay, lengths,
                               c.pool, (int)c.slots, c.slot_of, ws, ws_bytes, on.stream());
        if (rc == BLIN_OK && a[9] != Py_None) written(THPVariable_Unpack(a[9]));
        return c.answer(rc, out, a[8]);
    });
}

// q, k, v, log_decay, state, slots, scale, out, stream
PyObject *decay_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        expect_args(n, 9);
        const Call c(a, 3, "[B, H, d]", a[4], a[5]);
        if (c.state == nullptr) value_error("a step needs a state");
        const CallStream on(a[8], c.q);
        c.keep(on, a[3], a[5]);
        const Tensor out = c.output(a[7], on);
        const blin_decay_layouts lay = c.layouts(out);
        const blin_status rc =
            blin_decay_step(c.q.const_data_ptr(), c.k.const_data_ptr(), c.v.const_data_ptr(), out.data_ptr(), c.dt, (int)c.B,
                            (int)c.H, (int)c.d, c.lg, number(a[6], "scale"), c.dense(out) ? nullptr : &lay, c.pool, (int)c.slots,
                            c.slot_of, on.stream());
        return c.answer(rc, out, a[7]);
    });
}

// q, k, rope_split, grid, t0, positions, theta, inverse, out, stream; NotImplemented where autograd has to record
// the call
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        expect_args(n, 10);
        const bool two = a[1] != Py_None;
        const Tensor &q = operand(a[0], "q", 4, "[B, Hq, N, d]");
        const Tensor &k = two ? operand(a[1], "k", 4, "[B, Hk, N, d]") : q;
        const blin_dtype dt = dtype_of(q);
        const int64_t B = q.size(0), N = q.size(2), d = q.size(3);
        same_kind(q, "q", q.sizes(), q);
        same_kind(k, "k", {B, k.size(1), N, d}, q);
        on_current_device(q);
        if ((a[3] == Py_None) == (a[5] == Py_None)) value_error("give either grid or positions");
        blin_geom g = {};
        g.Hgt = g.Wid = g.block_frames = 1;
        g.theta = number(a[6], "theta");
        integers(a[2], "rope_split", g.rope_split, 3);
        const int *pos = nullptr;
        int shared = 0;
        if (a[5] != Py_None) {
            shared = THPVariable_Check(a[5]) && THPVariable_Unpack(a[5]).dim() == 2;
            pos = static_cast<const int *>(shared ? optional(a[5], "positions", at::kInt, {N, 3}, q)
                                                  : optional(a[5], "positions", at::kInt, {B, N, 3}, q));
        } else {
            int t[3];
            integers(a[3], "grid", t, 3);
            g.T = t[0], g.Hgt = t[1], g.Wid = t[2];
        }
        const int inverse = PyObject_IsTrue(a[7]);
        if (inverse < 0) {
            PyErr_Clear();
            type_error("inverse must be True or False");
        }
        const bool record = recorded(q) || (two && recorded(k));
        if (record && a[8] == Py_None) Py_RETURN_NOTIMPLEMENTED;
        const CallStream on(a[9], q);
        on.keep(q), on.keep(k), on.keep(a[5]);
        Tensor out[2];
        const Tensor *in[2] = {&q, &k};
        const int outs = two ? 2 : 1;
        if (a[8] == Py_None) {
            for (int i = 0; i < outs; ++i) out[i] = on.output(in[i]->sizes(), q);
        } else {
            PyObject *o[2] = {a[8], nullptr};
            const bool seq = PyTuple_Check(a[8]) || PyList_Check(a[8]);
            if ((seq ? PySequence_Size(a[8]) : 1) != outs) value_error("out must hold " + std::to_string(outs) + " tensor(s)");
            for (int i = 0; i < outs && seq; ++i) o[i] = PyTuple_Check(a[8]) ? PyTuple_GET_ITEM(a[8], i) : PyList_GET_ITEM(a[8], i);
            for (int i = 0; i < outs; ++i) {
                out[i] = given_out(o[i], *in[i]);
                if (record || recorded(out[i]))
                    runtime_error("rope with out= has no gradient: call it under torch.no_grad(), or with tensors that require none");
                for (int j = 0; j < outs; ++j)
                    if (i != j || !same_place(out[i], *in[i])) no_overlap(out[i], *in[j]);
            }
            if (two) no_overlap(out[0], out[1]);
            for (int i = 0; i < outs; ++i) on.keep(out[i]);
        }
        if (!two) out[1] = out[0];
        auto result = [&]() -> PyObject * {
            if (!two) return THPVariable_Wrap(out[0]);
            PyObject *x = THPVariable_Wrap(out[0]), *y = THPVariable_Wrap(out[1]);
            PyObject *both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
            Py_XDECREF(x);
            Py_XDECREF(y);
            return both;
        };
        if (N == 0 && B > 0 && q.size(1) > 0 && k.size(1) > 0) return result();
        const bool dense = q.is_contiguous() && k.is_contiguous() && out[0].is_contiguous() && out[1].is_contiguous();
        const blin_rope_layouts lay{layout(q), layout(out[0]), layout(k), layout(out[1])};
        const blin_status rc =
            blin_rope(q.const_data_ptr(), out[0].data_ptr(), (int)q.size(1), two ? k.const_data_ptr() : nullptr,
                      two ? out[1].data_ptr() : nullptr, two ? (int)k.size(1) : 0, dt, (int)B, (int)N, (int)d, &g,
                      (int)integer(a[4], "t0"), pos, shared, inverse, dense ? nullptr : &lay, on.stream());
        if (rc != BLIN_OK) return PyLong_FromLong(rc);
        for (int i = 0; i < outs && a[8] != Py_None; ++i) written(out[i]);
        return result();
    });
}

PyMethodDef methods[] = {
    {"decay_prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decay_prefill)), METH_FASTCALL, nullptr},
    {"decay_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decay_step)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_blin_torch", "Tensor-side marshalling of libblin calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__blin_torch() {
    PyObject *m = PyModule_Create(&module);
    // what it was built with: its calls into torch and Python hold for these versions only
    const std::string built = std::string("torch ") + TORCH_VERSION + ", Python " + std::to_string(PY_MAJOR_VERSION) + "." +
                              std::to_string(PY_MINOR_VERSION);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", built.c_str()) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
