// marshal.cpp -- tensors to argument structs, for the operators that a decode
// loop calls once per token and layer (the Python module _marshal).
//
// Each function takes a helper's arguments in order and returns the bytes of
// the C struct, or None when anything is not as the common case has it (a
// tensor on another device, of another type or shape, not dense where it has
// to be, not a tensor at all): the Python helper then looks at the tensors one
// by one and either says what is wrong or fills the struct itself.  Looking at
// a tensor from Python costs about a microsecond, from here some ten
// nanoseconds; a call of these operators on a few rows takes two microseconds
// on the GPU.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "hm.h"

namespace {

struct No {};             // not the common case

using Args = PyObject *const *;

// a tensor, or nullptr for None
const at::Tensor *opt(PyObject *o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw No();
    return &THPVariable_Unpack(o);
}
const at::Tensor &need(PyObject *o) {
    const at::Tensor *t = opt(o);
    if (!t) throw No();
    return *t;
}
long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw No();
    return v;
}
double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw No();
    return v;
}

// What the rows of one call share: type, shape, the current device.
struct Common {
    at::IntArrayRef shape;
    at::ScalarType type;
    c10::Device dev;

    explicit Common(const at::Tensor &x) : shape(x.sizes()), type(x.scalar_type()), dev(x.device()) {
        if (!x.is_cuda() || dev.index() != c10::cuda::current_device()) throw No();
        if (type != at::kBFloat16 && type != at::kFloat) throw No();
    }
    hm_dtype code() const { return type == at::kBFloat16 ? HM_BF16 : HM_F32; }
    void *rows(const at::Tensor *t, at::IntArrayRef sh) const {
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->device() != dev || t->sizes() != sh || t->stride(-1) != 1) throw No();
        return t->data_ptr();
    }
    void *rows(const at::Tensor *t) const { return rows(t, shape); }
    void *dense(const at::Tensor *t, at::IntArrayRef sh, at::ScalarType ty = at::kFloat) const {
        if (!t) return nullptr;
        if (t->scalar_type() != ty || t->device() != dev || t->sizes() != sh || !t->is_contiguous()) throw No();
        return t->data_ptr();
    }
    float *f32(PyObject *o, at::IntArrayRef sh) const { return (float *)dense(opt(o), sh); }
    // a byte buffer of any type; dense, so that its size is that of the memory behind it
    void *buffer(PyObject *o, size_t &bytes) const {
        bytes = 0;
        const at::Tensor *t = opt(o);
        if (!t) return nullptr;
        if (t->device() != dev || !t->is_contiguous()) throw No();
        bytes = (size_t)t->numel() * t->element_size();
        return t->data_ptr();
    }
};

template <typename S>
PyObject *bytes_of(const S &s) {
    return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&s), sizeof(S));
}

// f(args), or None where it gives up
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// x, dt, y, A_log, dt_bias, h0, h_out, lengths, states, input_scale
PyObject *gated_scan(PyObject *, Args o, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &x = need(o[0]), &dt = need(o[1]), *y = opt(o[2]);
        const Common c(x);
        if (c.shape.size() != 3) throw No();
        const int64_t B = c.shape[0], D = c.shape[2];
        hm_gated_scan_args a{};
        a.B = B, a.L = c.shape[1], a.D = D;
        a.io_dtype = c.code();
        a.x = c.rows(&x), a.dt = c.rows(&dt), a.y = c.rows(y);
        a.x_stride_b = x.stride(0), a.x_stride_t = x.stride(1);
        a.dt_stride_b = dt.stride(0), a.dt_stride_t = dt.stride(1);
        if (y) a.y_stride_b = y->stride(0), a.y_stride_t = y->stride(1);
        a.A_log = c.f32(o[3], {D}), a.dt_bias = c.f32(o[4], {D});
        a.h0 = c.f32(o[5], {B, D}), a.h_out = c.f32(o[6], {B, D});
        a.lengths = (const int32_t *)c.dense(opt(o[7]), {B}, at::kInt);
        a.states = c.buffer(o[8], a.states_bytes);
        a.input_scale = (int)integer(o[9]);
        return bytes_of(a);
    });
}

// x, dt, dy, dx, ddt, A_log, dA_log, states, dt_bias, d_dt_bias, dh_out, dh0, lengths, input_scale, workspace
PyObject *gated_scan_bwd(PyObject *, Args o, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const at::Tensor &x = need(o[0]), &dt = need(o[1]), &dy = need(o[2]), &dx = need(o[3]), &ddt = need(o[4]);
        const Common c(x);
        if (c.shape.size() != 3) throw No();
        const int64_t B = c.shape[0], D = c.shape[2];
        hm_gated_scan_bwd_args a{};
        a.B = B, a.L = c.shape[1], a.D = D;
        a.io_dtype = c.code();
        a.x = c.rows(&x), a.dt = c.rows(&dt), a.dy = c.rows(&dy), a.dx = c.rows(&dx), a.ddt = c.rows(&ddt);
        a.x_stride_b = x.stride(0), a.x_stride_t = x.stride(1);
        a.dt_stride_b = dt.stride(0), a.dt_stride_t = dt.stride(1);
        a.dy_stride_b = dy.stride(0), a.dy_stride_t = dy.stride(1);
        a.dx_stride_b = dx.stride(0), a.dx_stride_t = dx.stride(1);
        a.ddt_stride_b = ddt.stride(0), a.ddt_stride_t = ddt.stride(1);
        a.A_log = c.f32(o[5], {D}), a.dA_log = c.f32(o[6], {D});
        a.states = c.buffer(o[7], a.states_bytes);
        a.dt_bias = c.f32(o[8], {D}), a.d_dt_bias = c.f32(o[9], {D});
        a.dh_out = c.f32(o[10], {B, D}), a.dh0 = c.f32(o[11], {B, D});
        a.lengths = (const int32_t *)c.dense(opt(o[12]), {B}, at::kInt);
        a.input_scale = (int)integer(o[13]);
        a.workspace = c.buffer(o[14], a.workspace_bytes);
        return bytes_of(a);
    });
}

// x, dt, y, h, h_out, A_log, dt_bias, input_scale
PyObject *gated_step(PyObject *, Args o, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        const at::Tensor &x = need(o[0]), &dt = need(o[1]), &y = need(o[2]);
        const Common c(x);
        if (c.shape.size() != 2) throw No();
        const int64_t D = c.shape[1];
        hm_gated_step_args a{};
        a.B = c.shape[0], a.D = D;
        a.io_dtype = c.code();
        a.x = c.rows(&x), a.dt = c.rows(&dt), a.y = c.rows(&y);
        a.x_stride = x.stride(0), a.dt_stride = dt.stride(0), a.y_stride = y.stride(0);
        a.h = c.f32(o[3], c.shape), a.h_out = c.f32(o[4], c.shape);
        a.A_log = c.f32(o[5], {D}), a.dt_bias = c.f32(o[6], {D});
        a.input_scale = (int)integer(o[7]);
        return bytes_of(a);
    });
}

// elements between the rows of a [.., D] array: two axes, or dense
int64_t row_stride(const at::Tensor *t) {
    if (!t) return 0;
    if (t->dim() == 2) return t->stride(0);
    if (!t->is_contiguous()) throw No();
    return t->size(-1);
}
int64_t row_count(const Common &c) {
    if (c.shape.size() < 2 || c.shape.back() == 0) throw No();
    int64_t n = 1;
    for (size_t i = 0; i + 1 < c.shape.size(); ++i) n *= c.shape[i];
    return n;
}

// y, r, r_out, xn, gate, norm, post, eps, alpha, scale, post_w, post_b, pre_w, pre_b
PyObject *norm_gate(PyObject *, Args o, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const at::Tensor &y = need(o[0]), *r = opt(o[1]), *r_out = opt(o[2]), *xn = opt(o[3]), *gate = opt(o[4]);
        const Common c(y);
        hm_norm_gate_args a{};
        a.rows = row_count(c), a.D = c.shape.back();
        a.io_dtype = c.code();
        a.norm = (int)integer(o[5]), a.post = (int)integer(o[6]);
        a.eps = (float)real(o[7]), a.alpha = (float)real(o[8]);
        a.y = c.rows(&y), a.gate = c.rows(gate), a.r = c.rows(r), a.r_out = c.rows(r_out), a.xn = c.rows(xn);
        a.y_stride = row_stride(&y), a.gate_stride = row_stride(gate), a.r_stride = row_stride(r);
        a.r_out_stride = row_stride(r_out), a.xn_stride = row_stride(xn);
        a.scale = c.f32(o[9], {a.D});
        a.post_w = c.f32(o[10], {a.D}), a.post_b = c.f32(o[11], {a.D});
        a.pre_w = c.f32(o[12], {a.D}), a.pre_b = c.f32(o[13], {a.D});
        return bytes_of(a);
    });
}

// y, r_out, dr_out, dxn, dy, dr, gate, dgate, norm, post, eps, alpha, scale, post_w, post_b, pre_w, dscale, dpost_w,
// dpost_b, dpre_w, dpre_b, workspace
PyObject *norm_gate_bwd(PyObject *, Args o, Py_ssize_t n) {
    return guarded(n, 22, [&] {
        const at::Tensor &y = need(o[0]), *r_out = opt(o[1]), *dr_out = opt(o[2]), *dxn = opt(o[3]), *dy = opt(o[4]),
                         *dr = opt(o[5]), *gate = opt(o[6]), *dgate = opt(o[7]);
        const Common c(y);
        hm_norm_gate_bwd_args a{};
        a.rows = row_count(c), a.D = c.shape.back();
        a.io_dtype = c.code();
        a.y = c.rows(&y), a.r_out = c.rows(r_out), a.dr_out = c.rows(dr_out), a.dxn = c.rows(dxn);
        a.dy = c.rows(dy), a.dr = c.rows(dr), a.gate = c.rows(gate), a.dgate = c.rows(dgate);
        a.norm = (int)integer(o[8]), a.post = (int)integer(o[9]);
        a.eps = (float)real(o[10]), a.alpha = (float)real(o[11]);
        a.y_stride = row_stride(&y), a.r_out_stride = row_stride(r_out), a.dr_out_stride = row_stride(dr_out);
        a.dxn_stride = row_stride(dxn), a.dy_stride = row_stride(dy), a.dr_stride = row_stride(dr);
        a.gate_stride = row_stride(gate), a.dgate_stride = row_stride(dgate);
        a.scale = c.f32(o[12], {a.D}), a.post_w = c.f32(o[13], {a.D}), a.post_b = c.f32(o[14], {a.D});
        a.pre_w = c.f32(o[15], {a.D}), a.dscale = c.f32(o[16], {a.D}), a.dpost_w = c.f32(o[17], {a.D});
        a.dpost_b = c.f32(o[18], {a.D}), a.dpre_w = c.f32(o[19], {a.D}), a.dpre_b = c.f32(o[20], {a.D});
        a.workspace = c.buffer(o[21], a.workspace_bytes);
        return bytes_of(a);
    });
}

// q, k, q_out, k_out, rot, base, layout, scaling, factor, orig_len, beta_slow, beta_fast, mscale, transpose,
// positions, pos0
PyObject *rotary(PyObject *, Args o, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const at::Tensor &q = need(o[0]), *k = opt(o[1]), &qo = need(o[2]), *ko = opt(o[3]), *pos = opt(o[14]);
        const Common c(q);
        if (c.shape.size() != 4 || !k != !ko) throw No();
        hm_rotary_args a{};
        a.B = c.shape[0], a.L = c.shape[1], a.Hq = (int)c.shape[2], a.d = (int)c.shape[3];
        a.io_dtype = c.code();
        const int64_t rot = integer(o[4]);
        if (c.shape[2] > (1 << 20) || c.shape[3] > (1 << 20) || rot < 0 || rot > (1 << 20)) throw No();
        a.rot = rot ? (int)rot : a.d;
        a.q = c.rows(&q), a.q_out = c.rows(&qo);
        a.q_stride_b = q.stride(0), a.q_stride_t = q.stride(1), a.q_stride_h = q.stride(2);
        a.q_out_stride_b = qo.stride(0), a.q_out_stride_t = qo.stride(1), a.q_out_stride_h = qo.stride(2);
        if (k) {
            if (k->dim() != 4 || k->size(2) > (1 << 20)) throw No();
            const int64_t sh[4] = {a.B, a.L, k->size(2), a.d};
            a.Hk = (int)k->size(2);
            a.k = c.rows(k, sh), a.k_out = c.rows(ko, sh);
            a.k_stride_b = k->stride(0), a.k_stride_t = k->stride(1), a.k_stride_h = k->stride(2);
            a.k_out_stride_b = ko->stride(0), a.k_out_stride_t = ko->stride(1), a.k_out_stride_h = ko->stride(2);
        }
        if (pos) {
            if (pos->scalar_type() != at::kLong || pos->device() != c.dev || pos->dim() != 2 ||
                (pos->size(0) != 1 && pos->size(0) != a.B) || (pos->size(1) != 1 && pos->size(1) != a.L))
                throw No();
            a.positions = (const int64_t *)pos->data_ptr();
            a.pos_stride_b = pos->size(0) == 1 ? 0 : pos->stride(0);
            a.pos_stride_t = pos->size(1) == 1 ? 0 : pos->stride(1);
        }
        a.base = real(o[5]);
        a.layout = (int)integer(o[6]), a.scaling = (int)integer(o[7]);
        a.factor = real(o[8]), a.orig_len = real(o[9]), a.beta_slow = real(o[10]), a.beta_fast = real(o[11]);
        a.mscale = real(o[12]);
        a.transpose = (int)integer(o[13]);
        a.pos0 = integer(o[15]);
        return bytes_of(a);
    });
}

// a byte buffer on the current device, or None where it is not 256-byte aligned
PyObject *alloc(PyObject *, Args o, Py_ssize_t n) {
    return guarded(n, 1, [&] {
        const long long bytes = integer(o[0]);
        at::Tensor t = at::empty({bytes > 1 ? bytes : 1},
                                 at::TensorOptions().dtype(at::kByte).device(at::kCUDA, c10::cuda::current_device()));
        if ((uintptr_t)t.data_ptr() % 256 != 0) throw No();
        return THPVariable_Wrap(std::move(t));
    });
}

#define FN(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(gated_scan), FN(gated_scan_bwd), FN(gated_step), FN(norm_gate), FN(norm_gate_bwd),
                         FN(rotary),     FN(alloc),          {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and Python whose objects this build knows (the binding compares)
PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", HM_MARSHAL_TAG) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
