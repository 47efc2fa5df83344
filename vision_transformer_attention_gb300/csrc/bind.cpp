// bind.cpp -- the calls on tokens as functions of a CPython extension module,
// for the speed of small calls: api.py reads a torch tensor's type, strides and
// address in Python (20 us for a rotation of one decoding step, whose kernel
// takes 2), this reads them from the tensor object. Every function makes the
// call of include/rpe_attn.h that api.py would make, or returns None where
// anything is out of the ordinary (an argument of another type or shape,
// another device than the current one, a call that fails); api.py then goes
// its own way, with its checks and errors.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "rpe_attn.h"

namespace {

using at::Tensor;

// The tensor behind an argument; nullptr for anything else.
const Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int dtype_code(at::ScalarType t) {
    return t == at::kBFloat16 ? RPE_DTYPE_BF16
           : t == at::kHalf   ? RPE_DTYPE_F16
           : t == at::kFloat  ? RPE_DTYPE_F32
                              : -1;
}

// rpe_view of a [tokens, heads, d] or [batch, tokens, heads, d] tensor on
// `device` with contiguous channels.
bool view(const Tensor &t, at::ScalarType dtype, at::Device device, rpe_view *v) {
    const int64_t n = t.dim();
    if (t.scalar_type() != dtype || t.device() != device || (n != 3 && n != 4) ||
        t.layout() != at::kStrided)
        return false;
    const auto s = t.strides();
    if (t.size(n - 1) > 1 && s[n - 1] != 1) return false;
    v->data = t.data_ptr();
    v->batch_stride = n == 4 ? s[0] : 0;
    v->token_stride = s[n - 3];
    v->head_stride = s[n - 2];
    return true;
}

bool plain(const Tensor &t, at::ScalarType dtype, at::Device device) {
    return t.scalar_type() == dtype && t.device() == device && t.is_contiguous();
}

// An output: the caller's, or a new one of x's shape.
bool output(PyObject *o, const Tensor &x, Tensor *out) {
    if (o == Py_None) {
        *out = at::empty(x.sizes(), x.options().requires_grad(false));
        return true;
    }
    const Tensor *t = tensor(o);
    if (t == nullptr || t->sizes() != x.sizes()) return false;
    *out = *t;
    return true;
}

// q's device is the current one: its stream, else false.
bool here(const Tensor &q, void **stream) {
    if (!q.is_cuda() || q.device().index() != c10::cuda::current_device()) return false;
    *stream = c10::cuda::getCurrentCUDAStream(q.device().index()).stream();
    return true;
}

// rope(q, k, q_out, k_out, positions, phases, flags, magnitude, norm, eps, q_gain, k_gain);
// norm < 0: rope_fwd, else qk_norm_rope_fwd
PyObject *rope_call(PyObject *const *a) {
    const Tensor *q = tensor(a[0]);
    const bool has_k = a[1] != Py_None;
    const Tensor *k = has_k ? tensor(a[1]) : nullptr;
    void *stream;
    if (q == nullptr || (has_k && k == nullptr) || !here(*q, &stream)) return nullptr;
    const at::ScalarType dtype = q->scalar_type();
    const at::Device device = q->device();
    const int code = dtype_code(dtype);
    const int64_t n = q->dim();
    rpe_view vq, vk, oq, ok;
    if (code < 0 || !view(*q, dtype, device, &vq)) return nullptr;
    if (has_k) {
        if (!view(*k, dtype, device, &vk) || k->dim() != n) return nullptr;
        for (int64_t i = 0; i < n; ++i)
            if (i != n - 2 && k->size(i) != q->size(i)) return nullptr;
    }
    const int64_t batch = n == 4 ? q->size(0) : 1, tokens = q->size(n - 3);
    const long norm = PyLong_AsLong(a[8]);
    unsigned flags = static_cast<unsigned>(PyLong_AsUnsignedLong(a[6]));
    int axes = 1, rotary = 0;
    const int32_t *positions = nullptr;
    const uint64_t *phases = nullptr;
    if (a[5] != Py_None) {
        const Tensor *ph = tensor(a[5]), *pos = tensor(a[4]);
        if (ph == nullptr || pos == nullptr || !plain(*ph, at::kLong, device) ||
            !plain(*pos, at::kInt, device))
            return nullptr;
        const auto s = pos->sizes();
        if (s.size() == 3 && n == 4 && s[0] == batch && s[1] == tokens && s[2] <= 2) {
            axes = static_cast<int>(s[2]);
            flags |= RPE_ROPE_BATCH_POSITIONS;
        } else if (s.size() == 2 && s[0] == tokens && s[1] <= 2) {
            axes = static_cast<int>(s[1]);
        } else if (!(s.size() == 1 && s[0] == tokens)) {
            return nullptr;
        }
        if (ph->numel() > 128) return nullptr;
        rotary = 2 * static_cast<int>(ph->numel());
        positions = pos->data_ptr<int32_t>();
        phases = reinterpret_cast<const uint64_t *>(ph->data_ptr<int64_t>());
    } else if (norm < 0) {
        return nullptr;
    }
    const void *gains[2] = {nullptr, nullptr};
    int gain_code = code;
    if (norm >= 0) {
        at::ScalarType gain_type = dtype;
        for (int i = 0, seen = 0; i < 2; ++i) {
            if (a[10 + i] == Py_None) continue;
            const Tensor *g = tensor(a[10 + i]);
            if (g == nullptr) return nullptr;
            if (!seen++) gain_type = g->scalar_type() == at::kFloat ? at::kFloat : dtype;
            if (!plain(*g, gain_type, device) || g->dim() != 1 || g->size(0) != q->size(n - 1))
                return nullptr;
            gains[i] = g->data_ptr();
        }
        gain_code = dtype_code(gain_type);
    }
    if (q->size(n - 2) > 65536 || (has_k && k->size(n - 2) > 65536) || q->size(n - 1) > 256) return nullptr;
    const float magnitude = static_cast<float>(PyFloat_AsDouble(a[7]));
    const float eps = static_cast<float>(PyFloat_AsDouble(a[9]));
    if (PyErr_Occurred()) return nullptr;
    Tensor tq, tk;
    if (!output(a[2], *q, &tq) || !view(tq, dtype, device, &oq)) return nullptr;
    if (has_k && (!output(a[3], *k, &tk) || !view(tk, dtype, device, &ok))) return nullptr;
    const int hq = static_cast<int>(q->size(n - 2)), hk = has_k ? static_cast<int>(k->size(n - 2)) : 0;
    const int d = static_cast<int>(q->size(n - 1));
    const rpe_view *pk = has_k ? &vk : nullptr, *po = has_k ? &ok : nullptr;
    const int rc =
        norm < 0 ? rope_fwd(&vq, pk, &oq, po, positions, axes, phases, rotary, magnitude, flags, batch,
                            tokens, hq, hk, d, code, stream)
                 : qk_norm_rope_fwd(&vq, pk, &oq, po, static_cast<int>(norm), eps, gains[0], gains[1],
                                    gain_code, positions, axes, phases, rotary, magnitude, flags, batch,
                                    tokens, hq, hk, d, code, stream);
    if (rc != RPE_OK) return nullptr;
    PyObject *r0 = a[2] != Py_None ? Py_NewRef(a[2]) : THPVariable_Wrap(std::move(tq));
    PyObject *r1 = !has_k              ? Py_NewRef(Py_None)
                   : a[3] != Py_None ? Py_NewRef(a[3])
                                     : THPVariable_Wrap(std::move(tk));
    PyObject *both = r0 != nullptr && r1 != nullptr ? PyTuple_Pack(2, r0, r1) : nullptr;
    Py_XDECREF(r0);
    Py_XDECREF(r1);
    return both;
}

// attn(q, k, v, cu_q, cu_k, k_lens, causal, scale, out, return_lse, workspace); scale None: 1 / sqrt(d)
PyObject *attn_call(PyObject *const *a) {
    const Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *cu_q = tensor(a[3]);
    const Tensor *cu_k = a[4] == Py_None ? cu_q : tensor(a[4]);
    const bool lens = a[5] != Py_None, own_ws = a[10] == Py_None;
    const Tensor *k_lens = lens ? tensor(a[5]) : nullptr, *ws = own_ws ? nullptr : tensor(a[10]);
    void *stream;
    if (q == nullptr || k == nullptr || v == nullptr || cu_q == nullptr || cu_k == nullptr ||
        (lens && k_lens == nullptr) || (!own_ws && ws == nullptr) || !here(*q, &stream))
        return nullptr;
    const at::ScalarType dtype = q->scalar_type();
    const at::Device device = q->device();
    const int code = dtype_code(dtype);
    rpe_view vq, vk, vv, vo;
    if (code < 0 || q->dim() != 3 || k->dim() != 3 || k->sizes() != v->sizes() ||
        k->size(2) != q->size(2) || !view(*q, dtype, device, &vq) || !view(*k, dtype, device, &vk) ||
        !view(*v, dtype, device, &vv))
        return nullptr;
    const int64_t total_q = q->size(0), total_k = k->size(0), heads_q = q->size(1), heads_kv = k->size(1);
    const int64_t batch = cu_q->numel() - 1, d = q->size(2);
    if (!plain(*cu_q, at::kInt, device) || batch < 0 || !plain(*cu_k, at::kInt, device) ||
        cu_k->dim() != 1 || cu_k->size(0) != batch + 1 || batch > (1 << 24) || heads_q > 65536 ||
        heads_kv > 65536 || heads_kv < 1 || d > 256 || d < 1)
        return nullptr;
    if (lens && (!plain(*k_lens, at::kInt, device) || k_lens->dim() != 1 || k_lens->size(0) != batch))
        return nullptr;
    const int causal = PyObject_IsTrue(a[6]), want_lse = PyObject_IsTrue(a[9]);
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return nullptr;
    size_t bytes = 0;
    if (packed_attn_workspace(total_q, total_k, static_cast<int>(batch), static_cast<int>(heads_q),
                              static_cast<int>(heads_kv), static_cast<int>(d), code, &bytes) != RPE_OK)
        return nullptr;
    Tensor out, lse, space;
    if (!output(a[8], *q, &out) || !view(out, dtype, device, &vo)) return nullptr;
    if (want_lse) lse = at::empty({total_q, heads_q}, q->options().dtype(at::kFloat).requires_grad(false));
    if (own_ws && bytes > 0)
        space = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte).requires_grad(false));
    else if (!own_ws && !plain(*ws, at::kByte, device))
        return nullptr;
    void *ws_ptr = own_ws ? (bytes > 0 ? space.data_ptr() : nullptr) : ws->data_ptr();
    const size_t ws_bytes = own_ws ? bytes : static_cast<size_t>(ws->numel());
    const int rc = packed_attn_fwd(
        &vq, &vk, &vv, &vo, want_lse ? lse.data_ptr<float>() : nullptr, cu_q->data_ptr<int32_t>(),
        cu_k->data_ptr<int32_t>(), lens ? k_lens->data_ptr<int32_t>() : nullptr, static_cast<int>(batch),
        total_q, total_k, static_cast<int>(heads_q), static_cast<int>(heads_kv), static_cast<int>(d),
        static_cast<float>(scale), causal ? RPE_ATTN_CAUSAL : 0u, code, ws_ptr, ws_bytes, stream);
    if (rc != RPE_OK) return nullptr;
    PyObject *r0 = a[8] != Py_None ? Py_NewRef(a[8]) : THPVariable_Wrap(std::move(out));
    if (!want_lse || r0 == nullptr) return r0;
    PyObject *r1 = THPVariable_Wrap(std::move(lse));
    PyObject *both = r1 != nullptr ? PyTuple_Pack(2, r0, r1) : nullptr;
    Py_DECREF(r0);
    Py_XDECREF(r1);
    return both;
}

// No C++ exception leaves the module; what was not done here is None.
template <PyObject *(*call)(PyObject *const *), Py_ssize_t N>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
    PyObject *r = nullptr;
    if (n == N) {
        try {
            r = call(args);
        } catch (...) {
            r = nullptr;
        }
    }
    if (r != nullptr) return r;
    PyErr_Clear();
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<rope_call, 12>)),
     METH_FASTCALL, "rope_fwd or qk_norm_rope_fwd; None: not done"},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<attn_call, 11>)),
     METH_FASTCALL, "packed_attn_fwd; None: not done"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "vta_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_vta_bind(void) { return PyModule_Create(&module); }
