// bind.cpp -- CPython module _cq_bind: the operand checks, output allocation and
// C calls of the operators between two LUT linears.
//
// A decode call of one of them runs for 2 to 4 us on the GPU and is enqueued in
// about 3.5 us; checking its 6 to 10 tensors and finding the stream in Python
// took another 8 to 10 us, which set the pace of an eager decode loop.  Here they
// take well under one.  What is computed, and every check of values, is
// behind include/cq.h; this file checks what the C interface cannot see: types,
// shapes, strides and devices of tensors.
#include <Python.h>

#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/cq.h"

namespace {

PyObject *g_error = nullptr;  // CQError(status, where)

struct Refused {
    cq_status status;
    std::string what;
};

struct PyFailed {};  // a Python exception is set

using at::Tensor;
using Shape = at::IntArrayRef;

std::string shape_text(Shape s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

// One call: its name, the operands' device, its stream.
struct Call {
    const char *name;
    c10::DeviceIndex dev = -1;

    [[noreturn]] void refuse(const std::string &why,
                             cq_status st = CQ_ERR_INVALID_ARGUMENT) const {
        throw Refused{st, std::string(name) + ": " + why};
    }
    void need(bool ok, const char *why) const {
        if (!ok) refuse(why);
    }
    const Tensor &tensor(PyObject *o, const char *what) const {
        if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor");
        return THPVariable_Unpack(o);
    }
    // the operand that fixes the device
    const Tensor &first(PyObject *o, const char *what, int64_t dim) {
        const Tensor &t = tensor(o, what);
        if (!t.is_cuda()) refuse(std::string(what) + " must be a CUDA tensor");
        if (t.dim() != dim) refuse(std::string(what) + " must have " + std::to_string(dim) + " dimensions");
        dev = t.device().index();
        return t;
    }
    void *dense(const Tensor &t, const char *what, at::ScalarType ty, Shape shape) const {
        if (t.scalar_type() != ty || t.sizes() != shape || !t.is_cuda() ||
            t.device().index() != dev || !t.is_contiguous())
            refuse(std::string(what) + " must be a contiguous " + c10::toString(ty) +
                   " tensor of shape " + shape_text(shape) + " on cuda:" + std::to_string(dev) +
                   ", got " + c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()) + " on " +
                   t.device().str());
        return t.data_ptr();
    }
    void *dense(PyObject *o, const char *what, at::ScalarType ty, Shape shape) const {
        return dense(tensor(o, what), what, ty, shape);
    }
    void *optional(PyObject *o, const char *what, at::ScalarType ty, Shape shape) const {
        return o == Py_None ? nullptr : dense(o, what, ty, shape);
    }
    at::TensorOptions options(at::ScalarType ty) const {
        return at::TensorOptions().dtype(ty).device(at::Device(at::kCUDA, dev));
    }
    void check(cq_status st) const {
        if (st != CQ_OK) throw Refused{st, name};
    }
};

// The call's stream: None (the device's current one), an object with
// cuda_stream, or its address.  While it lives, outputs and workspaces are
// allocated for that stream and the device is the operands'.
struct OnStream {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard guard;
    cudaStream_t st;
    OnStream(PyObject *o, c10::DeviceIndex dev) : device(dev) {
        if (o == Py_None) {
            st = c10::cuda::getCurrentCUDAStream(dev).stream();
            return;
        }
        PyObject *v = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!v) throw PyFailed{};
        st = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
        Py_DECREF(v);
        if (PyErr_Occurred()) throw PyFailed{};
        guard.reset_stream(st == c10::cuda::getDefaultCUDAStream(dev).stream()
                               ? c10::cuda::getDefaultCUDAStream(dev)
                               : c10::cuda::getStreamFromExternal(st, dev));
    }
    cq_stream_t raw() const { return reinterpret_cast<cq_stream_t>(st); }
};

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyFailed{};
    return v;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyFailed{};
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PyFailed{};
    return v != 0;
}

PyObject *given(PyObject *o) { return Py_NewRef(o); }
PyObject *made(const Tensor &t) {
    PyObject *o = THPVariable_Wrap(t);
    if (!o) throw PyFailed{};
    return o;
}

// residual_norm(resid, y, norm, eps, pre_weight, pre_bias, post_norm, post_weight,
//               post_bias, gate, resid_scale, block_scale, had_block, act_bits,
//               resid_out, x_out, q_out, s_out, stream)
PyObject *residual_norm(PyObject *const *a) {
    Call c{"cq_residual_norm"};
    const Tensor &r = c.first(a[0], "resid", 2);
    const auto ty = r.scalar_type();
    c.need(ty == at::kHalf || ty == at::kFloat, "resid must be fp16 or fp32");
    const int64_t T = r.size(0), H = r.size(1);
    const int64_t full[2] = {T, H}, per_row[2] = {T, 1}, vec[1] = {H}, rows[1] = {T};
    cq_norm_desc d{};
    d.H = H;
    d.norm = (int32_t)integer(a[2]);
    d.eps = number(a[3]);
    d.post_norm = truth(a[6]);
    d.resid_scale = number(a[10]);
    d.block_scale = number(a[11]);
    const int64_t had = integer(a[12]), bits = integer(a[13]);
    c.need(bits == 0 || bits == 4 || bits == 8, "act_bits must be 0, 4 or 8");
    c.need(had >= 0 && had <= (1 << 30), "had_block is out of range");
    d.had_block = (int32_t)had;
    d.act_bits = (int32_t)bits;
    d.resid_bits = ty == at::kHalf ? 16 : 32;
    const void *p_r = c.dense(r, "resid", ty, full);
    const void *p_pw = c.optional(a[4], "pre_weight", at::kHalf, vec);
    const void *p_pb = c.optional(a[5], "pre_bias", at::kHalf, vec);
    const void *p_qw = c.optional(a[7], "post_weight", at::kHalf, vec);
    const void *p_qb = c.optional(a[8], "post_bias", at::kHalf, vec);
    const bool block = a[1] != Py_None;
    const void *p_y = block ? c.dense(a[1], "y", at::kFloat, full) : nullptr;
    c.need(block || a[14] == Py_None, "resid_out without y");
    const void *p_g = nullptr;
    if (a[9] != Py_None) {
        const Tensor &g = c.tensor(a[9], "gate");
        if (g.dim() == 1) {
            d.gate_mode = CQ_GATE_CHANNEL;
            p_g = c.dense(g, "gate", at::kHalf, vec);
        } else if (g.dim() == 2 && g.size(1) == 1) {
            d.gate_mode = CQ_GATE_TOKEN;
            p_g = c.dense(g, "gate", at::kHalf, per_row);
        } else {
            d.gate_mode = CQ_GATE_ELEMENT;
            p_g = c.dense(g, "gate", at::kHalf, full);
        }
    }
    c.need(bits || (a[16] == Py_None && a[17] == Py_None), "q_out / s_out without act_bits");

    OnStream on(a[18], c.dev);
    Tensor t_r, t_x, t_q, t_s;  // what this call allocates
    void *p_ro = nullptr, *p_x, *p_q = nullptr;
    float *p_s = nullptr;
    if (block) {
        if (a[14] == Py_None) {
            t_r = at::empty(full, c.options(ty));
            p_ro = t_r.data_ptr();
        } else {
            p_ro = c.dense(a[14], "resid_out", ty, full);
        }
    }
    if (a[15] == Py_None) {
        t_x = at::empty(full, c.options(at::kHalf));
        p_x = t_x.data_ptr();
    } else {
        p_x = c.dense(a[15], "x_out", at::kHalf, full);
    }
    if (bits) {
        const auto qt = bits == 4 ? at::kByte : at::kChar;
        const int64_t codes[2] = {T, bits == 4 ? H / 2 : H};
        if (a[16] == Py_None) {
            t_q = at::empty(codes, c.options(qt));
            p_q = t_q.data_ptr();
        } else {
            p_q = c.dense(a[16], "q_out", qt, codes);
        }
        if (a[17] == Py_None) {
            t_s = at::empty(rows, c.options(at::kFloat));
            p_s = t_s.data_ptr<float>();
        } else {
            p_s = static_cast<float *>(c.dense(a[17], "s_out", at::kFloat, rows));
        }
    }
    c.check(cq_residual_norm(&d, T, static_cast<const float *>(p_y), p_g, p_qw, p_qb, p_r, p_ro,
                             p_pw, p_pb, p_x, p_q, p_s, on.raw()));
    PyObject *o = PyTuple_New(bits ? 4 : 2);
    if (!o) throw PyFailed{};
    PyTuple_SET_ITEM(o, 0, !block ? given(a[0]) : t_r.defined() ? made(t_r) : given(a[14]));
    PyTuple_SET_ITEM(o, 1, t_x.defined() ? made(t_x) : given(a[15]));
    if (bits) {
        PyTuple_SET_ITEM(o, 2, t_q.defined() ? made(t_q) : given(a[16]));
        PyTuple_SET_ITEM(o, 3, t_s.defined() ? made(t_s) : given(a[17]));
    }
    return o;
}

// An fp32 [M, N] operand whose rows may be slices of wider ones.
float *sliced(const Call &c, const Tensor &t, const char *what, int64_t M, int64_t N, int64_t &ld) {
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != M || t.size(1) != N ||
        !t.is_cuda() || t.device().index() != c.dev || (N > 1 && t.stride(1) != 1))
        c.refuse(std::string(what) + " must be fp32 [" + std::to_string(M) + ", " +
                 std::to_string(N) + "] on cuda:" + std::to_string(c.dev) + " with contiguous rows");
    ld = M > 1 ? t.stride(0) : N;
    return t.data_ptr<float>();
}

// lora_add(x, ids, a, b, y, scale, ranks, out, workspace, stream)
PyObject *lora_add(PyObject *const *a) {
    Call c{"cq_lora_add"};
    const Tensor &x = c.first(a[0], "x", 2);
    const Tensor &A = c.tensor(a[2], "a"), &B = c.tensor(a[3], "b");
    c.need(A.dim() == 3 && B.dim() == 3, "a must be [n, r, K] and b [n, N, r]");
    const int64_t M = x.size(0), K = x.size(1), n = A.size(0), r = A.size(1), N = B.size(1);
    const int64_t s_x[2] = {M, K}, s_i[1] = {M}, s_a[3] = {n, r, K}, s_b[3] = {n, N, r}, s_n[1] = {n};
    const void *p_x = c.dense(x, "x", at::kHalf, s_x);
    const void *p_i = c.dense(a[1], "ids", at::kInt, s_i);
    const void *p_a = c.dense(A, "a", at::kHalf, s_a), *p_b = c.dense(B, "b", at::kHalf, s_b);
    const void *p_s = c.optional(a[5], "scale", at::kFloat, s_n);
    const void *p_r = c.optional(a[6], "ranks", at::kInt, s_n);
    int64_t ldy = 0, ldo = 0;
    float *p_y = sliced(c, c.tensor(a[4], "y"), "y", M, N, ldy), *p_o = p_y;
    PyObject *out = a[7] == Py_None ? a[4] : a[7];
    if (a[7] == Py_None)
        ldo = ldy;
    else
        p_o = sliced(c, c.tensor(a[7], "out"), "out", M, N, ldo);

    OnStream on(a[9], c.dev);
    Tensor ws;
    size_t bytes = cq_lora_add_workspace_size(M, n, r);
    void *p_w = nullptr;
    if (a[8] != Py_None) {
        const Tensor &w = c.tensor(a[8], "workspace");
        c.need(w.is_cuda() && w.device().index() == c.dev && w.is_contiguous(),
               "workspace must be contiguous and on x's device");
        p_w = w.data_ptr();
        bytes = w.nbytes();
    } else if (bytes) {
        ws = at::empty({(int64_t)bytes}, c.options(at::kByte));
        p_w = ws.data_ptr();
    }
    c.check(cq_lora_add(p_x, static_cast<const int32_t *>(p_i), M, K, p_a, p_b,
                        static_cast<const float *>(p_s), static_cast<const int32_t *>(p_r), n, r, p_y,
                        ldy, p_o, ldo, N, p_w, bytes, on.raw()));
    return given(out);
}

// rope_qkv(qkv, positions, inv_freq, n_q, n_kv, head_dim, interleaved, attn_scale,
//          q_weight, k_weight, eps, q_out, k_out, v_out, slots, stream)
PyObject *rope_qkv(PyObject *const *a) {
    Call c{"cq_rope_qkv"};
    const Tensor &x = c.first(a[0], "qkv", 2);
    cq_rope_desc d{};
    d.n_q = integer(a[3]);
    d.n_kv = integer(a[4]);
    d.head_dim = integer(a[5]);
    constexpr int64_t kMax = 1 << 20;
    c.need(d.n_q > 0 && d.n_kv > 0 && d.head_dim > 0 && d.n_q < kMax && d.n_kv < kMax &&
               d.head_dim < kMax,
           "n_q, n_kv and head_dim must be positive");
    d.interleaved = truth(a[6]);
    d.attn_scale = (float)number(a[7]);
    d.eps = (float)number(a[10]);
    const int64_t M = x.size(0), nq = d.n_q, nkv = d.n_kv, D = d.head_dim;
    const int64_t s_x[2] = {M, (nq + 2 * nkv) * D}, s_m[1] = {M}, s_d[1] = {D}, s_q[3] = {M, nq, D},
                  s_k[3] = {M, nkv, D};
    const void *p_x = c.dense(x, "qkv", at::kFloat, s_x);
    const void *p_p = c.dense(a[1], "positions", at::kInt, s_m);
    const void *p_f = nullptr;
    if (a[2] != Py_None) {
        const Tensor &f = c.tensor(a[2], "inv_freq");
        c.need(f.dim() == 1 && f.size(0) > 0, "inv_freq must be [rot_dim / 2]");
        d.rot_dim = 2 * f.size(0);
        const int64_t s_f[1] = {f.size(0)};
        p_f = c.dense(f, "inv_freq", at::kFloat, s_f);
    }
    const void *p_qw = c.optional(a[8], "q_weight", at::kHalf, s_d);
    const void *p_kw = c.optional(a[9], "k_weight", at::kHalf, s_d);
    const void *p_sl = c.optional(a[14], "slots", at::kLong, s_m);
    c.need((a[12] == Py_None) == (a[13] == Py_None), "k_out and v_out come together");
    c.need(a[12] != Py_None || a[14] == Py_None, "slots need k_out and v_out");

    OnStream on(a[15], c.dev);
    Tensor t_q, t_k, t_v;
    void *p_q, *p_k, *p_v;
    if (a[11] == Py_None) {
        t_q = at::empty(s_q, c.options(at::kHalf));
        p_q = t_q.data_ptr();
    } else {
        p_q = c.dense(a[11], "q_out", at::kHalf, s_q);
    }
    if (a[12] == Py_None) {
        t_k = at::empty(s_k, c.options(at::kHalf));
        t_v = at::empty(s_k, c.options(at::kHalf));
        p_k = t_k.data_ptr();
        p_v = t_v.data_ptr();
        d.kv_token_stride = nkv * D;
        d.kv_head_stride = D;
        d.n_slots = M;
    } else {
        const Tensor &k = c.tensor(a[12], "k_out"), &v = c.tensor(a[13], "v_out");
        c.need(k.scalar_type() == at::kHalf && v.scalar_type() == at::kHalf && k.dim() == 3 &&
                   k.sizes() == v.sizes() && k.strides() == v.strides() && k.is_cuda() &&
                   v.is_cuda() && k.device().index() == c.dev && v.device().index() == c.dev,
               "k_out and v_out must be fp16 on qkv's device, alike in shape and strides");
        c.need(k.size(1) == nkv && k.size(2) == D && k.stride(2) == 1,
               "k_out must be [rows, n_kv, head_dim] with contiguous channels");
        c.need(a[14] != Py_None || k.size(0) >= M, "k_out has fewer rows than qkv");
        p_k = k.data_ptr();
        p_v = v.data_ptr();
        d.kv_token_stride = k.stride(0);
        d.kv_head_stride = k.stride(1);
        d.n_slots = k.size(0);
    }
    c.check(cq_rope_qkv(&d, M, static_cast<const float *>(p_x), static_cast<const int32_t *>(p_p),
                        static_cast<const float *>(p_f), p_qw, p_kw, p_q, p_k, p_v,
                        static_cast<const int64_t *>(p_sl), on.raw()));
    PyObject *o = PyTuple_New(3);
    if (!o) throw PyFailed{};
    PyTuple_SET_ITEM(o, 0, t_q.defined() ? made(t_q) : given(a[11]));
    PyTuple_SET_ITEM(o, 1, t_k.defined() ? made(t_k) : given(a[12]));
    PyTuple_SET_ITEM(o, 2, t_v.defined() ? made(t_v) : given(a[13]));
    return o;
}

// Runs one of them with its N arguments; refusals become CQError(status, where).
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return F(a);
    } catch (const Refused &r) {
        PyObject *e = PyObject_CallFunction(g_error, "is", (int)r.status, r.what.c_str());
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    } catch (const PyFailed &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_XSETREF(g_error, Py_NewRef(type));
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"residual_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<residual_norm, 19>)),
     METH_FASTCALL, nullptr},
    {"lora_add", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<lora_add, 10>)),
     METH_FASTCALL, nullptr},
    {"rope_qkv", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<rope_qkv, 16>)),
     METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, "the exception class of refusals"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cq_bind", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the torch whose headers this was built with
PyMODINIT_FUNC PyInit__cq_bind(void) {
    PyObject *m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "torch_version", CQ_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
