// py_mla.cpp -- the Python calls of the latent-attention operators and of those for
// drafted tokens in their common form: exact torch tensors on the current device, on
// its current stream.
//
// A decode step's kernels take about 10 us.  Interpreted checks, three
// allocations through Python's argument parser and a call with 18 converted
// arguments took 25 us in front of them; the same here takes 8 us (11 with
// at::empty), and 5 where the caller gives the outputs and the workspace.  An
// append (2 us on the GPU) went from 15 to 4 us.
//
// Whatever is not of the common form (another type, shape, device or stream, an
// argument that is wrong) gives NotImplemented before anything is launched: the
// caller in _binding.py then goes its own way, which ends in a message or in the
// same call.  Sizes and pointers are checked again behind the C entry points.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <initializer_list>
#include <limits>

#include "kda.h"

namespace {

constexpr int64_t LATENT = 512, ROPE = 64, ROW = LATENT + ROPE, NOPE = 128, DQK = NOPE + ROPE, DV = 128;
constexpr double SCALE = 0.07216878364870322;       // 192 ** -0.5

decltype(&kda_mla_append) append_fn;
decltype(&kda_mla_prefill) prefill_fn;
decltype(&kda_mla_prefill_workspace_size) prefill_ws_fn;
decltype(&kda_mla_decode) decode_fn;
decltype(&kda_mla_decode_workspace_size) decode_ws_fn;
decltype(&kda_mla_tree_decode) tree_decode_fn;
decltype(&kda_mla_tree_decode_workspace_size) tree_decode_ws_fn;
decltype(&kda_tree_step) step_fn[2];                // KDA, Gated DeltaNet
decltype(&kda_tree_commit) commit_fn[2];
decltype(&kda_tree_verify) verify_fn;
PyObject *error_class;                              // KdaError(function, status)

// The arguments of one call; `ok` turns false at the first that does not fit.
struct Call {
    bool ok = true;
    c10::DeviceIndex dev = -1;
    at::ScalarType type = at::kFloat;

    const at::Tensor *first(PyObject *o, int64_t dims) {
        if (!THPVariable_CheckExact(o)) { ok = false; return nullptr; }
        const at::Tensor &t = THPVariable_Unpack(o);
        type = t.scalar_type();
        dev = t.device().index();
        ok = t.is_cuda() && t.dim() == dims && (type == at::kBFloat16 || type == at::kFloat) &&
             dev == c10::cuda::current_device();
        return ok ? &t : nullptr;
    }
    // The tensor if it is of this type and shape, contiguous (`rows`: along its
    // last dimension) and on the call's device.  A dimension of -1 is any.
    const at::Tensor *need(PyObject *o, at::ScalarType of, std::initializer_list<int64_t> shape, bool rows = false) {
        if (!ok || !THPVariable_CheckExact(o)) { ok = false; return nullptr; }
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.is_cuda() && t.device().index() == dev && t.scalar_type() == of && t.dim() == (int64_t)shape.size();
        int64_t d = 0;
        for (const int64_t n : shape) {
            if (!ok) return nullptr;
            const int64_t have = t.size(d++);
            ok = (n < 0 || have == n) && have <= std::numeric_limits<int32_t>::max();
        }
        ok = ok && (t.is_contiguous() || (rows && t.stride(-1) == 1));
        return ok ? &t : nullptr;
    }
    at::Tensor make(at::ScalarType of, std::initializer_list<int64_t> shape) const {
        return at::Tensor(at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), of,
                                                 at::Device(at::kCUDA, dev), std::nullopt));
    }
    // An output: the caller's, or a new one.
    at::Tensor out(PyObject *o, at::ScalarType of, std::initializer_list<int64_t> shape) {
        if (o == Py_None) return ok ? make(of, shape) : at::Tensor();
        const at::Tensor *t = need(o, of, shape);
        return t ? *t : at::Tensor();
    }
    float scale(PyObject *o) {
        if (o == Py_None) return (float)SCALE;
        ok = ok && PyFloat_CheckExact(o);
        return ok ? (float)PyFloat_AS_DOUBLE(o) : 0.f;
    }
    int32_t code() const { return type == at::kBFloat16 ? KDA_BF16 : KDA_FP32; }
    void *stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

PyObject *not_handled() { Py_RETURN_NOTIMPLEMENTED; }

PyObject *failed(const char *name, kda_status st) {
    PyObject *e = PyObject_CallFunction(error_class, "si", name, (int)st);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return nullptr;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *x = THPVariable_Wrap(a), *y = x ? THPVariable_Wrap(b) : nullptr;
    PyObject *t = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// The workspace: the caller's, or one of `need` bytes until the call returns (the
// allocator hands it out again in the stream's order).
struct Scratch {
    c10::DataPtr own;
    void *data = nullptr;
    uint64_t bytes = 0;
    void get(Call &c, PyObject *o, uint64_t need) {
        if (!c.ok) return;
        if (o == Py_None) {
            if (!need) return;
            own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
            data = own.get();
            bytes = need;
        } else if (const at::Tensor *w = c.need(o, at::kByte, {-1})) {
            data = w->data_ptr();
            bytes = (uint64_t)w->numel();
        }
    }
};

// prefill(q, kv, k_r, cu_q, cu_k, scale, causal, o, lse, workspace)
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) return not_handled();
    Call c;
    const at::Tensor *q = c.first(a[0], 3);
    if (!q) return not_handled();
    const int64_t Tq = q->size(0), H = q->size(1);
    c.need(a[0], c.type, {Tq, H, DQK});
    const at::Tensor *kv = c.need(a[1], c.type, {-1, H, NOPE + DV});
    const int64_t Tk = kv ? kv->size(0) : 0;
    const at::Tensor *kr = c.need(a[2], c.type, {Tk, ROPE});
    const at::Tensor *cq = c.need(a[3], at::kInt, {-1});
    if (!c.ok || cq->size(0) < 1) return not_handled();
    const int64_t N = cq->size(0) - 1;
    const at::Tensor *ck = c.need(a[4], at::kInt, {N + 1});
    const float scale = c.scale(a[5]);
    const int causal = c.ok ? PyObject_IsTrue(a[6]) : 0;
    if (causal < 0) return nullptr;
    const at::Tensor o = c.out(a[7], c.type, {Tq, H, DV});
    const at::Tensor lse = c.out(a[8], at::kFloat, {Tq, H});
    Scratch w;
    w.get(c, a[9], c.ok ? prefill_ws_fn((int32_t)N, Tq, (int32_t)H, c.code()) : 0);
    if (!c.ok) return not_handled();
    kda_status st;
    void *stream = c.stream();
    Py_BEGIN_ALLOW_THREADS
    st = prefill_fn(q->data_ptr(), kv->data_ptr(), kr->data_ptr(), cq->data_ptr<int32_t>(),
                    ck->data_ptr<int32_t>(), (int32_t)N, Tq, Tk, (int32_t)H, NOPE, ROPE, DV, c.code(), scale,
                    causal, o.data_ptr(), lse.data_ptr<float>(), w.data, w.bytes, stream);
    Py_END_ALLOW_THREADS
    return st == KDA_OK ? pair(o, lse) : failed("kda_mla_prefill", st);
    END_HANDLE_TH_ERRORS
}

// decode(q, cache, table, seq_lens, scale, o, lse, workspace)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) return not_handled();
    Call c;
    const at::Tensor *q = c.first(a[0], 3);
    if (!q) return not_handled();
    const int64_t B = q->size(0), H = q->size(1);
    c.need(a[0], c.type, {B, H, ROW});
    const at::Tensor *cache = c.need(a[1], c.type, {-1, -1, ROW});
    const at::Tensor *table = c.need(a[2], at::kInt, {B, -1});
    const at::Tensor *lens = c.need(a[3], at::kInt, {B});
    const float scale = c.scale(a[4]);
    const at::Tensor o = c.out(a[5], c.type, {B, H, LATENT});
    const at::Tensor lse = c.out(a[6], at::kFloat, {B, H});
    Scratch w;
    w.get(c, a[7], c.ok ? decode_ws_fn((int32_t)B, (int32_t)H, c.code()) : 0);
    if (!c.ok) return not_handled();
    kda_status st;
    void *stream = c.stream();
    Py_BEGIN_ALLOW_THREADS
    st = decode_fn(q->data_ptr(), cache->data_ptr(), table->data_ptr<int32_t>(), lens->data_ptr<int32_t>(),
                   (int32_t)B, (int32_t)H, (int32_t)cache->size(0), (int32_t)cache->size(1),
                   (int32_t)table->size(1), LATENT, ROPE, c.code(), scale, o.data_ptr(),
                   lse.data_ptr<float>(), w.data, w.bytes, stream);
    Py_END_ALLOW_THREADS
    return st == KDA_OK ? pair(o, lse) : failed("kda_mla_decode", st);
    END_HANDLE_TH_ERRORS
}

// append(c, k_r, slots, cache, positions, rope, interleaved, k_out, q_r, q_out)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) return not_handled();
    Call c;
    const at::Tensor *lat = c.first(a[0], 2);
    if (!lat) return not_handled();
    const int64_t T = lat->size(0);
    c.need(a[0], c.type, {T, LATENT}, true);
    const at::Tensor *kr = c.need(a[1], c.type, {T, ROPE}, true);
    const at::Tensor *slots = c.need(a[2], at::kInt, {T});
    const at::Tensor *cache = c.need(a[3], c.type, {-1, -1, ROW});
    const at::Tensor *pos = nullptr, *rope = nullptr, *ko = nullptr, *qr = nullptr;
    if ((a[4] == Py_None) != (a[5] == Py_None) || (a[8] == Py_None && a[9] != Py_None)) return not_handled();
    if (a[5] != Py_None) {
        pos = c.need(a[4], at::kInt, {T});
        rope = c.need(a[5], at::kFloat, {-1, ROPE});
    }
    const int pairs = PyObject_IsTrue(a[6]);
    if (pairs < 0) return nullptr;
    if (a[7] != Py_None) ko = c.need(a[7], c.type, {T, ROPE}, true);
    at::Tensor qo;
    if (a[8] != Py_None) {
        qr = c.need(a[8], c.type, {T, -1, ROPE}, true);
        if (qr && a[9] == Py_None) qo = c.make(c.type, {T, qr->size(1), ROPE});
        else if (const at::Tensor *t = qr ? c.need(a[9], c.type, {T, qr->size(1), ROPE}, true) : nullptr) qo = *t;
    }
    if (!c.ok) return not_handled();
    kda_status st;
    void *stream = c.stream();
    Py_BEGIN_ALLOW_THREADS
    st = append_fn(lat->data_ptr(), lat->stride(0), kr->data_ptr(), kr->stride(0), slots->data_ptr<int32_t>(),
                   pos ? pos->data_ptr<int32_t>() : nullptr, rope ? rope->data_ptr<float>() : nullptr,
                   rope ? (int32_t)rope->size(0) : 0, pairs, T, cache->data_ptr(), (int32_t)cache->size(0),
                   (int32_t)cache->size(1), LATENT, ROPE, c.code(), ko ? ko->data_ptr() : nullptr,
                   ko ? ko->stride(0) : 0, qr ? qr->data_ptr() : nullptr, qr ? qr->stride(0) : 0,
                   qr ? qr->stride(1) : 0, qr ? (int32_t)qr->size(1) : 0, qr ? qo.data_ptr() : nullptr,
                   qr ? qo.stride(0) : 0, qr ? qo.stride(1) : 0, stream);
    Py_END_ALLOW_THREADS
    if (st != KDA_OK) return failed("kda_mla_append", st);
    if (!qr) Py_RETURN_NONE;
    if (a[9] != Py_None) { Py_INCREF(a[9]); return a[9]; }
    return THPVariable_Wrap(qo);
    END_HANDLE_TH_ERRORS
}

// tree_decode(q, cache, table, ctx_lens, parents, scale, o, lse, workspace)
PyObject *tree_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return not_handled();
    Call c;
    const at::Tensor *q = c.first(a[0], 4);
    if (!q) return not_handled();
    const int64_t B = q->size(0), T = q->size(1), H = q->size(2);
    c.need(a[0], c.type, {B, T, H, ROW});
    const at::Tensor *cache = c.need(a[1], c.type, {-1, -1, ROW});
    const at::Tensor *table = c.need(a[2], at::kInt, {B, -1});
    const at::Tensor *lens = c.need(a[3], at::kInt, {B});
    const at::Tensor *parents = c.need(a[4], at::kInt, {B, T});
    const float scale = c.scale(a[5]);
    const at::Tensor o = c.out(a[6], c.type, {B, T, H, LATENT});
    const at::Tensor lse = c.out(a[7], at::kFloat, {B, T, H});
    Scratch w;
    w.get(c, a[8], c.ok ? tree_decode_ws_fn((int32_t)B, (int32_t)T, (int32_t)H, c.code()) : 0);
    if (!c.ok) return not_handled();
    kda_status st;
    void *stream = c.stream();
    Py_BEGIN_ALLOW_THREADS
    st = tree_decode_fn(q->data_ptr(), cache->data_ptr(), table->data_ptr<int32_t>(), lens->data_ptr<int32_t>(),
                        parents->data_ptr<int32_t>(), (int32_t)B, (int32_t)T, (int32_t)H, (int32_t)cache->size(0),
                        (int32_t)cache->size(1), (int32_t)table->size(1), LATENT, ROPE, c.code(), scale,
                        o.data_ptr(), lse.data_ptr<float>(), w.data, w.bytes, stream);
    Py_END_ALLOW_THREADS
    return st == KDA_OK ? pair(o, lse) : failed("kda_mla_tree_decode", st);
    END_HANDLE_TH_ERRORS
}

// What a step and a commit over a tree share.
struct Tree {
    const at::Tensor *k = nullptr, *v = nullptr, *g = nullptr, *beta = nullptr, *S = nullptr, *slots = nullptr;
    int64_t B = 0, T = 0, H = 0, dk = 0, dv = 0, P = 0;
    bool get(Call &c, bool scalar, PyObject *k_, PyObject *v_, PyObject *g_, PyObject *beta_, PyObject *S_, PyObject *slots_) {
        k = c.first(k_, 4);
        if (!k) return false;
        B = k->size(0); T = k->size(1); H = k->size(2); dk = k->size(3);
        c.need(k_, c.type, {B, T, H, dk});
        v = c.need(v_, c.type, {B, T, H, -1});
        if (!c.ok) return false;
        dv = v->size(3);
        g = scalar ? c.need(g_, at::kFloat, {B, T, H}) : c.need(g_, at::kFloat, {B, T, H, dk});
        beta = c.need(beta_, at::kFloat, {B, T, H});
        P = B;
        if (slots_ != Py_None) {
            slots = c.need(slots_, at::kInt, {B});
            P = -1;
        }
        S = c.need(S_, at::kFloat, {P, H, dk, dv});
        if (c.ok) P = S->size(0);
        return c.ok;
    }
    const int32_t *slot_ptr() const { return slots ? slots->data_ptr<int32_t>() : nullptr; }
};

// tree_step(scalar gate, q, k, v, g, beta, S, parents, slots, o)
PyObject *tree_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) return not_handled();
    const bool scalar = a[0] == Py_True;
    Call c;
    Tree t;
    if (!t.get(c, scalar, a[2], a[3], a[4], a[5], a[6], a[8])) return not_handled();
    const at::Tensor *q = c.need(a[1], c.type, {t.B, t.T, t.H, t.dk});
    const at::Tensor *parents = c.need(a[7], at::kInt, {t.B, t.T});
    const at::Tensor o = c.out(a[9], c.type, {t.B, t.T, t.H, t.dv});
    if (!c.ok) return not_handled();
    kda_status st;
    void *stream = c.stream();
    Py_BEGIN_ALLOW_THREADS
    st = step_fn[scalar](q->data_ptr(), t.k->data_ptr(), t.v->data_ptr(), t.g->data_ptr<float>(),
                         t.beta->data_ptr<float>(), t.S->data_ptr<float>(), t.slot_ptr(), (int32_t)t.P,
                         parents->data_ptr<int32_t>(), (int32_t)t.B, (int32_t)t.T, (int32_t)t.H, (int32_t)t.dk,
                         (int32_t)t.dv, c.code(), o.data_ptr(), stream);
    Py_END_ALLOW_THREADS
    if (st != KDA_OK) return failed(scalar ? "kda_gdn_tree_step" : "kda_tree_step", st);
    if (a[9] != Py_None) { Py_INCREF(a[9]); return a[9]; }
    return THPVariable_Wrap(o);
    END_HANDLE_TH_ERRORS
}

// tree_commit(scalar gate, k, v, g, beta, S, path, slots)
PyObject *tree_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) return not_handled();
    const bool scalar = a[0] == Py_True;
    Call c;
    Tree t;
    if (!t.get(c, scalar, a[1], a[2], a[3], a[4], a[5], a[7])) return not_handled();
    const at::Tensor *path = c.need(a[6], at::kInt, {t.B, t.T});
    if (!c.ok) return not_handled();
    kda_status st;
    void *stream = c.stream();
    Py_BEGIN_ALLOW_THREADS
    st = commit_fn[scalar](t.k->data_ptr(), t.v->data_ptr(), t.g->data_ptr<float>(), t.beta->data_ptr<float>(),
                           t.S->data_ptr<float>(), t.slot_ptr(), (int32_t)t.P, path->data_ptr<int32_t>(),
                           (int32_t)t.B, (int32_t)t.T, (int32_t)t.H, (int32_t)t.dk, (int32_t)t.dv, c.code(), stream);
    Py_END_ALLOW_THREADS
    if (st != KDA_OK) return failed(scalar ? "kda_gdn_tree_commit" : "kda_tree_commit", st);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// tree_verify(target, tokens, parents, uniform, draft, path, count, next_token)
PyObject *tree_verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) return not_handled();
    Call c;
    const at::Tensor *target = c.first(a[0], 3);
    if (!target) return not_handled();
    const int64_t B = target->size(0), T = target->size(1), V = target->size(2);
    c.need(a[0], c.type, {B, T, V});                // rows of another stride go the other way
    const at::Tensor *draft = a[4] == Py_None ? nullptr : c.need(a[4], c.type, {B, T, V});
    const at::Tensor *tokens = c.need(a[1], at::kInt, {B, T});
    const at::Tensor *parents = c.need(a[2], at::kInt, {B, T});
    const at::Tensor *uniform = c.need(a[3], at::kFloat, {B, T});
    const at::Tensor out[3] = {c.out(a[5], at::kInt, {B, T}), c.out(a[6], at::kInt, {B}), c.out(a[7], at::kInt, {B})};
    if (!c.ok) return not_handled();
    kda_status st;
    void *stream = c.stream();
    Py_BEGIN_ALLOW_THREADS
    st = verify_fn(target->data_ptr(), V, draft ? draft->data_ptr() : nullptr, V, tokens->data_ptr<int32_t>(),
                   parents->data_ptr<int32_t>(), uniform->data_ptr<float>(), (int32_t)B, (int32_t)T, (int32_t)V,
                   c.code(), out[0].data_ptr<int32_t>(), out[1].data_ptr<int32_t>(), out[2].data_ptr<int32_t>(), stream);
    Py_END_ALLOW_THREADS
    if (st != KDA_OK) return failed("kda_tree_verify", st);
    PyObject *t = PyTuple_New(3);
    for (int i = 0; t && i < 3; ++i) {
        PyObject *x = THPVariable_Wrap(out[i]);
        if (!x) { Py_DECREF(t); return nullptr; }
        PyTuple_SET_ITEM(t, i, x);
    }
    return t;
    END_HANDLE_TH_ERRORS
}

// bind((addresses of the C entry points, in the order below), KdaError)
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *f, *e;
    if (!PyArg_ParseTuple(args, "O!O", &PyTuple_Type, &f, &e)) return nullptr;
    void *at[12];
    if (PyTuple_GET_SIZE(f) != 12) {
        PyErr_SetString(PyExc_ValueError, "bind takes 12 addresses");
        return nullptr;
    }
    for (int i = 0; i < 12; ++i) {
        at[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(f, i));
        if (!at[i]) return nullptr;
    }
    append_fn = reinterpret_cast<decltype(append_fn)>(at[0]);
    prefill_fn = reinterpret_cast<decltype(prefill_fn)>(at[1]);
    prefill_ws_fn = reinterpret_cast<decltype(prefill_ws_fn)>(at[2]);
    decode_fn = reinterpret_cast<decltype(decode_fn)>(at[3]);
    decode_ws_fn = reinterpret_cast<decltype(decode_ws_fn)>(at[4]);
    tree_decode_fn = reinterpret_cast<decltype(tree_decode_fn)>(at[5]);
    tree_decode_ws_fn = reinterpret_cast<decltype(tree_decode_ws_fn)>(at[6]);
    for (int i = 0; i < 2; ++i) {
        step_fn[i] = reinterpret_cast<decltype(&kda_tree_step)>(at[7 + i]);
        commit_fn[i] = reinterpret_cast<decltype(&kda_tree_commit)>(at[9 + i]);
    }
    verify_fn = reinterpret_cast<decltype(verify_fn)>(at[11]);
    Py_INCREF(e);
    Py_XDECREF(error_class);
    error_class = e;
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(F));
}
PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"append", fast<append>(), METH_FASTCALL, nullptr},
    {"prefill", fast<prefill>(), METH_FASTCALL, nullptr},
    {"decode", fast<decode>(), METH_FASTCALL, nullptr},
    {"tree_decode", fast<tree_decode>(), METH_FASTCALL, nullptr},
    {"tree_step", fast<tree_step>(), METH_FASTCALL, nullptr},
    {"tree_commit", fast<tree_commit>(), METH_FASTCALL, nullptr},
    {"tree_verify", fast<tree_verify>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_torch() { return PyModule_Create(&module); }
