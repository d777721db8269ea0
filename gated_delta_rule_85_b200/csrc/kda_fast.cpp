// The binding's short way for the linear-attention and group-norm calls: a small call takes
// less time on the GPU than its checks take in Python.  Each function here makes the checks of its
// Python wrapper on tensors of the current device, allocates what was not given, and calls the C
// ABI; it returns None without having done anything where a check does not hold, and the wrapper
// then goes its own way (refusals, tensors of other devices).  An int is the C ABI's error code.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/kda.h"

namespace {

using at::Tensor;

// The tensor of an argument; null for None, and `ok` false for anything else.
const Tensor *arg(PyObject *o, bool &ok) {
    if (o == Py_None) return nullptr;
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    ok = false;
    return nullptr;
}

bool sized(const Tensor &t, std::initializer_list<int64_t> s) { return t.sizes().equals(at::IntArrayRef(s)); }

// Contiguous, on CUDA device `dev`, of this type.
bool placed(const Tensor *t, int dev, at::ScalarType type) {
    return !t || (t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->is_contiguous());
}

const void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
float *fptr(const Tensor *t) { return t ? static_cast<float *>(t->data_ptr()) : nullptr; }
const int32_t *iptr(const Tensor *t) { return t ? static_cast<const int32_t *>(t->data_ptr()) : nullptr; }

void *stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

Tensor empty_of(const Tensor &like, at::IntArrayRef sizes, at::ScalarType type) {
    return at::empty(sizes, like.options().dtype(type));
}

bool fits(std::initializer_list<int64_t> sizes) {   // each an int of the C ABI
    for (const int64_t s : sizes)
        if (s < 0 || s > 0x7fffffff) return false;
    return true;
}

bool code_of(const Tensor &t, int &dt) {
    if (t.scalar_type() == at::kBFloat16) dt = KDA_BF16;
    else if (t.scalar_type() == at::kFloat) dt = KDA_F32;
    else return false;
    return true;
}

PyObject *none() { Py_RETURN_NONE; }
PyObject *code(int rc) { return PyLong_FromLong(rc); }

// Borrowed when it was given, else the new tensor.
PyObject *give(PyObject *given, const Tensor &made) {
    if (given && given != Py_None && given != Py_True) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(made);
}

constexpr at::ScalarType F32 = at::kFloat, I32 = at::kInt;

// ------------------------------------------------------------------ linear attention

// q, k, v, log_decay, state | pool, slots | None, o | None
PyObject *la_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7) return none();
    bool ok = true;
    const Tensor *q = arg(a[0], ok), *k = arg(a[1], ok), *v = arg(a[2], ok), *lg = arg(a[3], ok), *st = arg(a[4], ok),
                 *slots = arg(a[5], ok), *o = arg(a[6], ok);
    int dt;
    if (!ok || !q || !k || !v || !lg || !st || !q->is_cuda() || q->dim() != 3 || v->dim() != 3 ||
        st->dim() != 4 || !code_of(*q, dt))
        return none();
    const int dev = c10::cuda::current_device();
    const at::ScalarType type = q->scalar_type();
    const int64_t N = q->size(0), H = q->size(1), dk = q->size(2), dv = v->size(2);
    if (!placed(q, dev, type) || !placed(k, dev, type) || !placed(v, dev, type) || !placed(lg, dev, F32) ||
        !placed(st, dev, F32) || !placed(slots, dev, I32) || !placed(o, dev, type) || !sized(*k, {N, H, dk}) ||
        !sized(*v, {N, H, dv}) || !sized(*lg, {H}) || (o && !sized(*o, {N, H, dv})) || (slots && !sized(*slots, {N})) ||
        !sized(*st, {slots ? st->size(0) : N, H, dk, dv}) || !fits({N, H, dk, dv, st->size(0)}))
        return none();
    Tensor made;
    if (!o) made = empty_of(*v, v->sizes(), type);
    const Tensor &out = o ? *o : made;
    const int rc =
        slots ? kda_la_recurrent_step_slots(ptr(q), ptr(k), ptr(v), fptr(lg), fptr(st), iptr(slots), out.data_ptr(), (int)N,
                                            (int)H, (int)dk, (int)dv, (int)st->size(0), dt, stream(dev))
              : kda_la_recurrent_step(ptr(q), ptr(k), ptr(v), fptr(lg), fptr(st), out.data_ptr(), (int)N, (int)H, (int)dk,
                                      (int)dv, dt, stream(dev));
    return rc ? code(rc) : give(a[6], made);
    END_HANDLE_TH_ERRORS
}

// What the prefill calls check alike.
struct Prefill {
    const Tensor *q, *k, *v, *lg, *cu;
    int dev, dt;
    int64_t B, T, H, dk, dv, N;
    at::ScalarType type;
    bool good() {
        if (!q || !k || !v || !lg || !q->is_cuda() || q->dim() != 4 || v->dim() != 4 || !code_of(*q, dt)) return false;
        dev = c10::cuda::current_device();
        type = q->scalar_type();
        B = q->size(0), T = q->size(1), H = q->size(2), dk = q->size(3), dv = v->size(3);
        if (cu && cu->dim() != 1) return false;
        N = cu ? cu->size(0) - 1 : B;
        return N >= 0 && placed(q, dev, type) && placed(k, dev, type) && placed(v, dev, type) && placed(lg, dev, F32) &&
               placed(cu, dev, I32) && sized(*k, {B, T, H, dk}) && sized(*v, {B, T, H, dv}) && sized(*lg, {H}) &&
               fits({B, T, H, dk, dv, N});
    }
    bool state(const Tensor *s) const { return !s || (placed(s, dev, F32) && sized(*s, {N, H, dk, dv})); }
    // The workspace's address and bytes: the given one's, or a new one's.
    bool workspace(const Tensor *given, size_t need, Tensor &made, void *&p, size_t &bytes) const {
        p = nullptr;
        bytes = 0;
        if (given) {
            if (!given->is_cuda() || given->get_device() != dev || !given->is_contiguous()) return false;
            p = given->data_ptr();
            bytes = (size_t)given->numel() * given->element_size();
        } else if (need) {
            made = empty_of(*q, {(int64_t)need}, at::kByte);
            p = made.data_ptr();
            bytes = need;
        }
        return true;
    }
};

// q, k, v, log_decay, init | None, cu | None, o | None, final (bool or tensor), workspace | None
PyObject *la_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return none();
    bool ok = true;
    const bool final_bool = PyBool_Check(a[7]);
    const Tensor *init = arg(a[4], ok), *o = arg(a[6], ok), *last = final_bool ? nullptr : arg(a[7], ok),
                 *ws = arg(a[8], ok);
    Prefill p{arg(a[0], ok), arg(a[1], ok), arg(a[2], ok), arg(a[3], ok), arg(a[5], ok)};
    if (!ok || (!final_bool && !last) || !p.good() || !p.state(init) || !p.state(last) ||
        (o && (!placed(o, p.dev, p.type) || !sized(*o, {p.B, p.T, p.H, p.dv}))))
        return none();
    Tensor made_o, made_last, made_ws;
    void *wp;
    size_t nb;
    const size_t need = kda_la_chunk_forward_workspace_size((int)p.B, (int)p.T, (int)p.H, (int)p.dk, (int)p.dv, (int)p.N,
                                                            p.dt, 0);
    if (!p.workspace(ws, need, made_ws, wp, nb)) return none();
    if (!o) made_o = empty_of(*p.v, p.v->sizes(), p.type);
    if (a[7] == Py_True) made_last = empty_of(*p.q, {p.N, p.H, p.dk, p.dv}, F32);
    const bool want = a[7] != Py_False;
    const int rc = kda_la_chunk_forward(ptr(p.q), ptr(p.k), ptr(p.v), fptr(p.lg), fptr(init),
                                        o ? o->data_ptr() : made_o.data_ptr(),
                                        want ? (last ? fptr(last) : fptr(&made_last)) : nullptr, iptr(p.cu), (int)p.B,
                                        (int)p.T, (int)p.H, (int)p.dk, (int)p.dv, (int)p.N, p.dt, wp, nb, stream(p.dev));
    if (rc) return code(rc);
    PyObject *first = give(a[6], made_o), *second = want ? give(a[7], made_last) : none();
    PyObject *both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
    END_HANDLE_TH_ERRORS
}

// q, k, v, log_decay, pool, slots, cu | None, o | None, workspace | None
PyObject *la_forward_slots(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) return none();
    bool ok = true;
    const Tensor *pool = arg(a[4], ok), *slots = arg(a[5], ok), *o = arg(a[7], ok), *ws = arg(a[8], ok);
    Prefill p{arg(a[0], ok), arg(a[1], ok), arg(a[2], ok), arg(a[3], ok), arg(a[6], ok)};
    if (!ok || !pool || !slots || !p.good() || pool->dim() != 4 || !placed(pool, p.dev, F32) ||
        !sized(*pool, {pool->size(0), p.H, p.dk, p.dv}) || !fits({pool->size(0)}) || !placed(slots, p.dev, I32) ||
        !sized(*slots, {p.N}) || (o && (!placed(o, p.dev, p.type) || !sized(*o, {p.B, p.T, p.H, p.dv}))))
        return none();
    Tensor made_o, made_ws;
    void *wp;
    size_t nb;
    const size_t need = kda_la_chunk_forward_workspace_size((int)p.B, (int)p.T, (int)p.H, (int)p.dk, (int)p.dv, (int)p.N,
                                                            p.dt, 1);
    if (!p.workspace(ws, need, made_ws, wp, nb)) return none();
    if (!o) made_o = empty_of(*p.v, p.v->sizes(), p.type);
    const int rc = kda_la_chunk_forward_slots(ptr(p.q), ptr(p.k), ptr(p.v), fptr(p.lg), fptr(pool), iptr(slots),
                                              o ? o->data_ptr() : made_o.data_ptr(), iptr(p.cu), (int)p.B, (int)p.T,
                                              (int)p.H, (int)p.dk, (int)p.dv, (int)p.N, (int)pool->size(0), p.dt, wp, nb,
                                              stream(p.dev));
    return rc ? code(rc) : give(a[7], made_o);
    END_HANDLE_TH_ERRORS
}

// A dict of new tensors
bool put(PyObject *dict, const char *name, const Tensor &t) {
    PyObject *o = t.defined() ? THPVariable_Wrap(t) : none();
    const bool done = o && PyDict_SetItemString(dict, name, o) == 0;
    Py_XDECREF(o);
    return done;
}

// q, k, v, log_decay, d_o, init | None, dfinal | None, cu | None, dinit (bool), workspace | None
PyObject *la_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10 || !PyBool_Check(a[8])) return none();
    bool ok = true;
    const Tensor *d_o = arg(a[4], ok), *init = arg(a[5], ok), *dlast = arg(a[6], ok), *ws = arg(a[9], ok);
    Prefill p{arg(a[0], ok), arg(a[1], ok), arg(a[2], ok), arg(a[3], ok), arg(a[7], ok)};
    if (!ok || !d_o || !p.good() || !p.state(init) || !p.state(dlast) || !placed(d_o, p.dev, p.type) ||
        !sized(*d_o, {p.B, p.T, p.H, p.dv}))
        return none();
    Tensor dinit, made_ws;
    void *wp;
    size_t nb;
    const size_t need = kda_la_chunk_backward_workspace_size((int)p.B, (int)p.T, (int)p.H, (int)p.dk, (int)p.dv, (int)p.N,
                                                             p.dt);
    if (!p.workspace(ws, need, made_ws, wp, nb)) return none();
    const Tensor dq = empty_of(*p.q, p.q->sizes(), p.type), dk = empty_of(*p.q, p.q->sizes(), p.type),
                 dv = empty_of(*p.q, p.v->sizes(), p.type);
    if (a[8] == Py_True) dinit = empty_of(*p.q, {p.N, p.H, p.dk, p.dv}, F32);
    const int rc = kda_la_chunk_backward(ptr(p.q), ptr(p.k), ptr(p.v), fptr(p.lg), fptr(init), ptr(d_o), fptr(dlast),
                                         dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                         dinit.defined() ? fptr(&dinit) : nullptr, iptr(p.cu), (int)p.B, (int)p.T, (int)p.H,
                                         (int)p.dk, (int)p.dv, (int)p.N, p.dt, wp, nb, stream(p.dev));
    if (rc) return code(rc);
    PyObject *g = PyDict_New();
    if (g && !(put(g, "dq", dq) && put(g, "dk", dk) && put(g, "dv", dv) && put(g, "dinit_state", dinit))) Py_CLEAR(g);
    return g;
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ group norm

struct Norm {
    const Tensor *x, *w, *b, *gate;
    int dev, dt, act;
    int64_t N, L, C, G;
    at::ScalarType type;
    bool good(PyObject *groups, PyObject *activation) {
        if (!x || !x->is_cuda() || x->dim() < 2 || !code_of(*x, dt) || !PyLong_Check(groups) || !PyLong_Check(activation)) return false;
        int over = 0;
        G = PyLong_AsLongLongAndOverflow(groups, &over);
        act = (int)PyLong_AsLong(activation);
        dev = c10::cuda::current_device();
        type = x->scalar_type();
        N = x->size(0), C = x->size(-1), L = 1;
        for (int64_t i = 1; i + 1 < x->dim(); ++i) L *= x->size(i);
        return !over && G >= 1 && L >= 1 && C >= 1 && C % G == 0 && fits({L, C, G}) && placed(x, dev, type) &&
               placed(gate, dev, type) && placed(w, dev, F32) && placed(b, dev, F32) && (!w || sized(*w, {C})) &&
               (!b || sized(*b, {C})) && (!gate || gate->sizes().equals(x->sizes()));
    }
    bool workspace(const Tensor *given, bool backward, Tensor &made, void *&p, size_t &bytes) const {
        Prefill at{x};
        at.dev = dev;
        const size_t need = given ? 0 : kda_group_norm_workspace_size(N, (int)L, (int)C, (int)G, dt, backward);
        return at.workspace(given, need, made, p, bytes);
    }
};

// x, groups, weight | None, bias | None, gate | None, eps, activation code, y | None, workspace | None
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9 || !PyFloat_Check(a[5])) return none();
    bool ok = true;
    Norm m{arg(a[0], ok), arg(a[2], ok), arg(a[3], ok), arg(a[4], ok)};
    const Tensor *y = arg(a[7], ok), *ws = arg(a[8], ok);
    const double eps = PyFloat_AS_DOUBLE(a[5]);
    if (!ok || !m.good(a[1], a[6]) || !(eps > 0) || !placed(y, m.dev, m.type) || (y && !y->sizes().equals(m.x->sizes())))
        return none();
    Tensor made_y, made_ws;
    void *wp;
    size_t nb;
    if (!m.workspace(ws, false, made_ws, wp, nb)) return none();
    if (!y) made_y = empty_of(*m.x, m.x->sizes(), m.type);
    const Tensor mean = empty_of(*m.x, {m.N, m.G}, F32), rstd = empty_of(*m.x, {m.N, m.G}, F32);
    const int rc = kda_group_norm_forward(ptr(m.x), fptr(m.w), fptr(m.b), ptr(m.gate), y ? y->data_ptr() : made_y.data_ptr(),
                                          fptr(&mean), fptr(&rstd), m.N, (int)m.L, (int)m.C, (int)m.G, (float)eps, m.act,
                                          m.dt, wp, nb, stream(m.dev));
    if (rc) return code(rc);
    PyObject *out[3] = {give(a[7], made_y), THPVariable_Wrap(mean), THPVariable_Wrap(rstd)};
    PyObject *all = out[0] && out[1] && out[2] ? PyTuple_Pack(3, out[0], out[1], out[2]) : nullptr;
    for (PyObject *o : out) Py_XDECREF(o);
    return all;
    END_HANDLE_TH_ERRORS
}

// dy, x, mean, rstd, groups, weight | None, bias | None, gate | None, activation code, workspace | None
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) return none();
    bool ok = true;
    const Tensor *dy = arg(a[0], ok), *mean = arg(a[2], ok), *rstd = arg(a[3], ok), *ws = arg(a[9], ok);
    Norm m{arg(a[1], ok), arg(a[5], ok), arg(a[6], ok), arg(a[7], ok)};
    if (!ok || !dy || !mean || !rstd || !m.good(a[4], a[8]) || !placed(dy, m.dev, m.type) ||
        !dy->sizes().equals(m.x->sizes()) || !placed(mean, m.dev, F32) || !placed(rstd, m.dev, F32) ||
        !sized(*mean, {m.N, m.G}) || !sized(*rstd, {m.N, m.G}))
        return none();
    Tensor dx, dgate, dw, db, made_ws;
    void *wp;
    size_t nb;
    if (!m.workspace(ws, true, made_ws, wp, nb)) return none();
    dx = empty_of(*m.x, m.x->sizes(), m.type);
    if (m.gate) dgate = empty_of(*m.x, m.x->sizes(), m.type);
    if (m.w) dw = empty_of(*m.x, {m.C}, F32);
    if (m.b) db = empty_of(*m.x, {m.C}, F32);
    const int rc = kda_group_norm_backward(ptr(dy), ptr(m.x), fptr(mean), fptr(rstd), fptr(m.w), fptr(m.b), ptr(m.gate),
                                           dx.data_ptr(), m.gate ? dgate.data_ptr() : nullptr, m.w ? fptr(&dw) : nullptr,
                                           m.b ? fptr(&db) : nullptr, m.N, (int)m.L, (int)m.C, (int)m.G, m.act, m.dt, wp,
                                           nb, stream(m.dev));
    if (rc) return code(rc);
    PyObject *g = PyDict_New();
    if (g && !(put(g, "dx", dx) && (!m.gate || put(g, "dgate", dgate)) && (!m.w || put(g, "dweight", dw)) &&
               (!m.b || put(g, "dbias", db))))
        Py_CLEAR(g);
    return g;
    END_HANDLE_TH_ERRORS
}

#define KDA_FAST(name) {#name, (PyCFunction)(void (*)())name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_FAST(la_step), KDA_FAST(la_forward), KDA_FAST(la_forward_slots), KDA_FAST(la_backward),
                         KDA_FAST(norm), KDA_FAST(norm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// KDA_BUILT_FOR: the torch and Python whose headers this was compiled with; the binding uses it with no others.
PyMODINIT_FUNC PyInit__kda_fast() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", KDA_BUILT_FOR) != 0) Py_CLEAR(m);
    return m;
}
