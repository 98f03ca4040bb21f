// gdn_bind.cpp -- the host side of the calls that a decode step makes one after the other and
// whose time is the host's: the paged cache's (gdn_attn.h) and beam search's (gdn_beam.h).
//
// Each function takes the address of the library's entry point and the arguments of the Python
// function of that name (attention.py, beams.py).  Where everything about them is as it has to
// be, it makes the call on the tensors' device and its current stream and returns the results;
// otherwise NotImplemented, and the Python function goes on, which refuses with its message,
// switches devices, or takes what is rarer (sequences that are no tuple, say).  So every check
// here is one that Python makes too, and nothing is read or written before all have passed.
// Looking at a tensor costs 50 to 100 ns from Python and next to nothing here: a token's append
// and its reading back, two calls, take 36 us of the host from Python and 14 from here, a small
// selection 20 and 11, a reordering 21 and 7, a token's attention 14 and 7.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <vector>

#include "gdn_attn.h"
#include "gdn_beam.h"

namespace {

PyObject *g_error = nullptr;      // GdnError

PyObject *other() { Py_RETURN_NOTIMPLEMENTED; }

// ------------------------------------------------------------------ arguments

bool none(PyObject *o) { return o == Py_None; }

// A plain tensor (subclasses have ways of their own).
const at::Tensor *tensor(PyObject *o) {
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}
// The same on GPU `at`.
const at::Tensor *on(PyObject *o, int at) {
    const at::Tensor *t = tensor(o);
    return t && t->is_cuda() && t->get_device() == at && t->layout() == at::kStrided ? t : nullptr;
}
// The call's device: that of t, which has to be the current one.
bool device_of(const at::Tensor *t, int *at) {
    if (!t || !t->is_cuda() || t->layout() != at::kStrided) return false;
    *at = t->get_device();
    return c10::cuda::current_device() == *at;
}
bool whole(PyObject *o, int64_t *x) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    *x = PyLong_AsLongLongAndOverflow(o, &over);
    return over == 0;
}
bool fits(int64_t x, int *to) {
    if (x < INT_MIN || x > INT_MAX) return false;
    *to = (int)x;
    return true;
}
// A bound: what is larger than any int means the same as the largest.
bool bound(PyObject *o, int *to) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    const int64_t x = PyLong_AsLongLongAndOverflow(o, &over);
    if (over < 0 || x < INT_MIN) return false;
    *to = over > 0 || x > INT_MAX ? INT_MAX : (int)x;
    return true;
}
bool dtype_of(const at::Tensor &t, gdn_dtype *dt) {
    if (t.scalar_type() == at::kBFloat16) *dt = GDN_BF16;
    else if (t.scalar_type() == at::kFloat) *dt = GDN_F32;
    else return false;
    return true;
}
template <typename T>
T *data(const at::Tensor &t) { return static_cast<T *>(t.data_ptr()); }

// int32 of `dims` dimensions, the last one contiguous.
const at::Tensor *int32(PyObject *o, int64_t dims, int at) {
    const at::Tensor *t = on(o, at);
    if (!t || t->dim() != dims || t->scalar_type() != at::kInt) return nullptr;
    return t->size(dims - 1) > 1 && t->stride(dims - 1) != 1 ? nullptr : t;
}
// [B, W] of that type, contiguous.
const at::Tensor *grid(PyObject *o, int64_t B, int64_t W, at::ScalarType type, int at) {
    const at::Tensor *t = on(o, at);
    return t && t->dim() == 2 && t->size(0) == B && t->size(1) == W && t->scalar_type() == type &&
                   t->is_contiguous()
               ? t
               : nullptr;
}
// [tokens, heads, d] rows.
bool rows(const at::Tensor *t, int64_t heads, int64_t n, int64_t d, at::ScalarType type,
          gdn_rows *r) {
    if (!t || t->dim() != 3 || t->size(0) != n || t->size(1) != heads || t->size(2) != d ||
        t->stride(2) != 1 || t->scalar_type() != type)
        return false;
    *r = gdn_rows{t->data_ptr(), 0, heads > 1 ? t->stride(1) : 0, n > 1 ? t->stride(0) : 0, 0};
    return fits(heads, &r->heads);
}

int64_t page_size_of(int bits, int64_t size, int64_t d) {
    if (d < 1) return 0;
    if (bits == 4) {
        const int64_t n = size * 8 / (9 * d);
        return n * d * 9 == size * 8 ? n : 0;
    }
    int64_t n = (size - 16) / (2 * d);
    if (n > 128) n = (size - 32) / (2 * d);
    return n > 0 && 2 * n * d + 16 * (n < 128 ? 1 : n / 128) == size ? n : 0;
}

// The cache and the tokens of a call.
bool cache(int bits, PyObject *pages, PyObject *table, PyObject *len, PyObject *cu, PyObject *scale,
           int64_t n, int64_t d, int at, gdn_kv *kv) {
    const at::Tensor *p = on(pages, at), *t = int32(table, 2, at), *l = int32(len, 1, at);
    if (!p || !t || !l || p->dim() != 3 || p->scalar_type() != at::kByte || !p->is_contiguous())
        return false;
    const int64_t N = l->size(0), page = page_size_of(bits, p->size(2), d);
    if (page < 1 || t->size(0) != N) return false;
    const int32_t *offsets = nullptr;
    if (!none(cu)) {
        const at::Tensor *c = int32(cu, 1, at);
        if (!c || c->size(0) != N + 1) return false;
        offsets = data<int32_t>(*c);
    } else if (n < 0 || (n > 0 && (N == 0 || n % N != 0))) {
        return false;
    }
    const float *factors = nullptr;
    if (!none(scale)) {
        const at::Tensor *s = grid(scale, 2, p->size(1), at::kFloat, at);
        if (!s) return false;
        factors = data<float>(*s);
    }
    *kv = gdn_kv{};
    kv->pages = p->data_ptr();
    kv->head_scale = factors;
    kv->page_table = data<int32_t>(*t);
    kv->kv_len = data<int32_t>(*l);
    kv->cu_seqlens = offsets;
    kv->table_stride = t->stride(0);
    return fits(p->size(0), &kv->n_pages) && fits(page, &kv->page_size) &&
           fits(p->size(1), &kv->heads) && fits(d, &kv->d) && fits(N, &kv->N) &&
           fits(t->size(1), &kv->max_pages) && fits(n, &kv->n_tokens);
}

// The axis of each of n pairs: the bytes themselves, or numbers put into `kept`.
const uint8_t *axis_numbers(PyObject *o, int64_t n, std::vector<uint8_t> *kept) {
    if (PyBytes_CheckExact(o))
        return PyBytes_GET_SIZE(o) == n ? reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(o)) : nullptr;
    const bool list = PyList_CheckExact(o);
    if ((!list && !PyTuple_CheckExact(o)) || n < 1) return nullptr;
    if ((list ? PyList_GET_SIZE(o) : PyTuple_GET_SIZE(o)) != n) return nullptr;
    kept->resize(n);
    for (int64_t i = 0; i < n; ++i) {
        int64_t x;
        if (!whole(list ? PyList_GET_ITEM(o, i) : PyTuple_GET_ITEM(o, i), &x) || x < 0 || x > 255)
            return nullptr;
        (*kept)[i] = (uint8_t)x;
    }
    return kept->data();
}

// The rotation of packed tokens.
bool rotary(PyObject *cos, PyObject *sin, PyObject *pos, PyObject *axes, bool adjacent, int64_t n,
            int at, gdn_rotary *r, std::vector<uint8_t> *kept) {
    const at::Tensor *c = on(cos, at), *s = on(sin, at);
    if (!c || !s || c->dim() != 2 || s->dim() != 2 || c->size(0) != s->size(0) ||
        c->size(1) != s->size(1) || c->scalar_type() != at::kFloat ||
        s->scalar_type() != at::kFloat || !c->is_contiguous() || !s->is_contiguous())
        return false;
    const int lead = none(axes) ? 0 : 1;
    const at::Tensor *p = int32(pos, lead + 1, at);
    if (!p || p->size(lead) != n) return false;
    *r = gdn_rotary{};
    if (lead) {
        if (!(r->axes = axis_numbers(axes, c->size(1), kept))) return false;
        r->stride_axis = p->stride(0);
    }
    r->cos = data<float>(*c);
    r->sin = data<float>(*s);
    r->pos = data<int32_t>(*p);
    r->flags = adjacent ? GDN_ROPE_ADJACENT : 0;
    return fits(c->size(0), &r->table_len) && fits(2 * c->size(1), &r->d_rot) &&
           fits(lead ? p->size(0) : 1, &r->n_axes);
}

// fn(args..., stream) on the current stream of GPU `at`; false with the exception set if it
// answers with an error.
template <typename F, typename... A>
bool call(PyObject *address, PyObject *name, int at, A... args) {
    F *fn = reinterpret_cast<F *>(PyLong_AsVoidPtr(address));
    if (!fn) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no entry point");
        return false;
    }
    void *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)at).stream();
    gdn_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(args..., stream);
    Py_END_ALLOW_THREADS
    if (rc == GDN_OK) return true;
    PyObject *e = PyObject_CallFunction(g_error, "iO", (int)rc, name);
    if (e) PyErr_SetObject(g_error, e);
    Py_XDECREF(e);
    return false;
}

// What follows allocates: an exception of PyTorch's becomes one of Python's.
template <typename F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}
PyObject *wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
// A tuple of the given references, which it takes over.
PyObject *tuple(std::initializer_list<PyObject *> of) {
    PyObject *r = PyTuple_New((Py_ssize_t)of.size());
    Py_ssize_t i = 0;
    for (PyObject *o : of) {
        if (!o || !r) {
            Py_XDECREF(o);
            Py_CLEAR(r);
        } else {
            PyTuple_SET_ITEM(r, i++, o);
        }
    }
    return r;
}
PyObject *ref(PyObject *o) {
    Py_INCREF(o);
    return o;
}
// Entry i of the tuple `o` of n; nullptr if it is none.
PyObject *item(PyObject *o, Py_ssize_t n, Py_ssize_t i) {
    return PyTuple_CheckExact(o) && PyTuple_GET_SIZE(o) == n ? PyTuple_GET_ITEM(o, i) : nullptr;
}

// ---------------------------------------------------------------------- cache

// (address, name, bits, pages, k, v, page_table, kv_len, q, cu_seqlens, kv_scale, cos, sin, pos,
// axes, adjacent, out)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 17) return other();
    return guarded([&]() -> PyObject * {
        int64_t bits;
        int at;
        gdn_dtype dt;
        const at::Tensor *k = tensor(a[4]);
        if (!whole(a[2], &bits) || !device_of(k, &at) || k->dim() != 3 || !dtype_of(*k, &dt))
            return other();
        const int64_t n = k->size(0), d = k->size(2);
        const at::ScalarType type = k->scalar_type();
        gdn_kv kv;
        gdn_rows rk, rv, rq, rqo;
        gdn_rotary rot;
        std::vector<uint8_t> axes;
        if (!cache((int)bits, a[3], a[6], a[7], a[9], a[10], n, d, at, &kv) ||
            !rows(k, kv.heads, n, d, type, &rk) || !rows(on(a[5], at), kv.heads, n, d, type, &rv))
            return other();
        const int adjacent = PyObject_IsTrue(a[15]);
        const bool turned = !none(a[11]);
        if (adjacent < 0) return nullptr;
        if (turned != !none(a[12]) || turned != !none(a[13]) ||
            (!turned && (adjacent || !none(a[14]))))
            return other();
        if (turned && !rotary(a[11], a[12], a[13], a[14], adjacent != 0, n, at, &rot, &axes))
            return other();
        at::Tensor made;
        const at::Tensor *q = nullptr, *out = nullptr;
        if (none(a[8])) {
            if (!none(a[16])) return other();
        } else {
            q = on(a[8], at);
            if (!q || q->dim() != 3 || !rows(q, q->size(1), n, d, type, &rq)) return other();
            if (none(a[16])) {
                made = at::empty_like(*q);
                out = &made;
            } else {
                out = on(a[16], at);
            }
            if (!rows(out, q->size(1), n, d, type, &rqo)) return other();
        }
        if (!call<decltype(gdn_kv_append)>(a[0], a[1], at, &kv, &rk, &rv, q ? &rq : nullptr, q ? &rqo : nullptr,
                  turned ? &rot : nullptr, dt))
            return nullptr;
        if (!q) Py_RETURN_NONE;
        return made.defined() ? wrap(std::move(made)) : ref(a[16]);
    });
}

// (address, name, bits, pages, page_table, kv_len, n_tokens, d, cu_seqlens, kv_scale, dtype, out)
PyObject *read(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 12) return other();
    return guarded([&]() -> PyObject * {
        int64_t bits, n, d;
        int at;
        const at::Tensor *pages = tensor(a[3]);
        if (!whole(a[2], &bits) || !whole(a[6], &n) || !whole(a[7], &d) || !THPDtype_Check(a[10]) ||
            !device_of(pages, &at) || n < 0)
            return other();
        const at::ScalarType type = reinterpret_cast<THPDtype *>(a[10])->scalar_type;
        if (type != at::kBFloat16 && type != at::kFloat) return other();
        gdn_kv kv;
        gdn_rows rk, rv;
        if (!cache((int)bits, a[3], a[4], a[5], a[8], a[9], n, d, at, &kv)) return other();
        at::Tensor made[2];
        const at::Tensor *k = &made[0], *v = &made[1];
        if (none(a[11])) {
            for (at::Tensor &t : made) t = at::empty({n, kv.heads, d}, pages->options().dtype(type));
        } else {
            PyObject *first = item(a[11], 2, 0);
            if (!first) return other();
            k = on(first, at);
            v = on(item(a[11], 2, 1), at);
        }
        if (!rows(k, kv.heads, n, d, type, &rk) || !rows(v, kv.heads, n, d, type, &rv)) return other();
        if (!call<decltype(gdn_kv_read)>(a[0], a[1], at, &kv, &rk, &rv,
                  type == at::kFloat ? GDN_F32 : GDN_BF16))
            return nullptr;
        return made[0].defined() ? tuple({wrap(std::move(made[0])), wrap(std::move(made[1]))})
                                 : ref(a[11]);
    });
}

// (address, name, bits, q, pages, page_table, kv_len, cu_seqlens, kv_scale, max_len, max_new, scale,
// causal, window, out, return_lse)
PyObject *attn(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 16) return other();
    return guarded([&]() -> PyObject * {
        int64_t bits;
        int at, max_len, max_new, window;
        gdn_dtype dt;
        const at::Tensor *q = tensor(a[3]);
        if (!whole(a[2], &bits) || !device_of(q, &at) || q->dim() != 3 || !dtype_of(*q, &dt))
            return other();
        const int64_t n = q->size(0), Hq = q->size(1), d = q->size(2);
        const at::ScalarType type = q->scalar_type();
        gdn_kv kv;
        gdn_rows rq, ro;
        if (!cache((int)bits, a[4], a[5], a[6], a[7], a[8], n, d, at, &kv) ||
            !rows(q, Hq, n, d, type, &rq) || !bound(a[13], &window))
            return other();
        if (none(a[9])) {
            const int64_t most = (int64_t)kv.max_pages * kv.page_size;
            max_len = most > INT_MAX ? INT_MAX : (int)most;
        } else if (!bound(a[9], &max_len)) {
            return other();
        }
        if (none(a[10])) max_new = kv.cu_seqlens ? kv.n_tokens : kv.n_tokens / (kv.N > 1 ? kv.N : 1);
        else if (!bound(a[10], &max_new)) return other();
        float scale = 0;
        if (none(a[11])) scale = (float)std::pow((double)d, -0.5);
        else if (PyFloat_CheckExact(a[11])) scale = (float)PyFloat_AS_DOUBLE(a[11]);
        else return other();
        const int causal = PyObject_IsTrue(a[12]), want = PyObject_IsTrue(a[15]);
        if (causal < 0 || want < 0) return nullptr;
        at::Tensor made, lse;
        const at::Tensor *o = &made;
        if (none(a[14])) made = at::empty_like(*q);
        else o = on(a[14], at);
        if (!rows(o, Hq, n, d, type, &ro)) return other();
        if (want) lse = at::empty({n, Hq}, q->options().dtype(at::kFloat));
        if (!call<decltype(gdn_kv_attn)>(a[0], a[1], at, &kv, &rq, &ro, want ? data<float>(lse) : nullptr,
                  max_len, max_new, scale, window, causal ? (unsigned)GDN_ATTN_CAUSAL : 0u, dt))
            return nullptr;
        PyObject *r = made.defined() ? wrap(std::move(made)) : ref(a[14]);
        return want ? tuple({r, wrap(std::move(lse))}) : r;
    });
}

// ---------------------------------------------------------------------- beams

// (address, name, logits, scores, n, done, eos, out)
PyObject *select(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 8) return other();
    return guarded([&]() -> PyObject * {
        int at;
        gdn_dtype dt;
        const at::Tensor *x = tensor(a[2]);
        if (!device_of(x, &at) || !dtype_of(*x, &dt) || (x->dim() != 2 && x->dim() != 3)) return other();
        const at::Tensor *s = on(a[3], at);
        if (!s || s->dim() != 2) return other();
        const int64_t B = s->size(0), W = s->size(1), V = x->size(-1);
        int iB, iW, iV, iN;
        if (!fits(B, &iB) || !fits(W, &iW) || !fits(V, &iV) || !grid(a[3], B, W, at::kFloat, at))
            return other();
        if (x->dim() == 3 ? x->size(0) != B || x->size(1) != W : x->size(0) != B * W) return other();
        if (V > 1 && x->stride(-1) != 1) return other();
        const int64_t stride = W > 1 || x->dim() == 2 ? x->stride(-2) : x->stride(0);
        if (x->dim() == 3 && B > 1 && W > 1 && x->stride(0) != W * stride) return other();
        int64_t n = W, eos = 0;
        if (!none(a[4]) && !whole(a[4], &n)) return other();
        if (n < 1 || n > W * V || !fits(n, &iN)) return other();
        const uint8_t *done = nullptr;
        if (none(a[5]) != none(a[6])) return other();
        if (!none(a[5])) {
            const at::Tensor *t = grid(a[5], B, W, at::kBool, at);
            if (!t) t = grid(a[5], B, W, at::kByte, at);
            if (!t || !whole(a[6], &eos) || eos < 0 || eos >= V) return other();
            done = static_cast<const uint8_t *>(t->data_ptr());
        }
        at::Tensor made[3];
        void *to[3];
        for (int i = 0; i < 3; ++i) {
            const at::ScalarType type = i == 0 ? at::kFloat : at::kInt;
            const at::Tensor *t = &made[i];
            if (none(a[7])) {
                made[i] = at::empty({B, n}, x->options().dtype(type));
            } else {
                PyObject *o = item(a[7], 3, i);
                if (!o || !(t = grid(o, B, n, type, at))) return other();
            }
            to[i] = t->data_ptr();
        }
        if (!call<decltype(gdn_beam_select)>(a[0], a[1], at, (const void *)x->data_ptr(), stride,
                  (const float *)data<float>(*s), done, (int)eos, static_cast<float *>(to[0]),
                  static_cast<int32_t *>(to[1]), static_cast<int32_t *>(to[2]), iB, iW, iV, iN, dt))
            return nullptr;
        if (!made[0].defined()) return ref(a[7]);
        return tuple({wrap(std::move(made[0])), wrap(std::move(made[1])), wrap(std::move(made[2]))});
    });
}

// The pools of a list or tuple of tensors.
bool pools(PyObject *o, int at, std::vector<gdn_beam_pool> *to) {
    const bool list = PyList_CheckExact(o);
    if (!list && !PyTuple_CheckExact(o)) return false;
    const Py_ssize_t n = list ? PyList_GET_SIZE(o) : PyTuple_GET_SIZE(o);
    to->reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor *t = on(list ? PyList_GET_ITEM(o, i) : PyTuple_GET_ITEM(o, i), at);
        if (!t || t->dim() < 1 || !t->is_contiguous()) return false;
        gdn_beam_pool p{t->data_ptr(), 0, 0};
        if (!fits(t->size(0), &p.count)) return false;
        if (p.count) p.bytes = t->numel() / p.count * (int64_t)t->element_size();
        to->push_back(p);
    }
    return true;
}

// (address, name, parent, slots, states, caches, page_table, own_pages, kv_len, page_size, out)
PyObject *reorder(PyObject *, PyObject *const *a, Py_ssize_t na) {
    if (na != 11) return other();
    return guarded([&]() -> PyObject * {
        int at, iB, iW;
        const at::Tensor *parent = tensor(a[2]);
        if (!device_of(parent, &at) || parent->dim() != 2) return other();
        const int64_t B = parent->size(0), W = parent->size(1);
        const at::Tensor *slots = grid(a[3], B, W, at::kInt, at);
        if (!slots || !grid(a[2], B, W, at::kInt, at) || !fits(B, &iB) || !fits(W, &iW)) return other();
        std::vector<gdn_beam_pool> states, caches;
        if (!pools(a[4], at, &states) || !pools(a[5], at, &caches)) return other();
        const bool paged = !none(a[6]);
        for (int i = 7; i < 10; ++i)
            if (none(a[i]) == paged) return other();
        if ((!paged && !caches.empty()) || (!paged && states.empty())) return other();
        const at::Tensor *table = nullptr, *own = nullptr, *len = nullptr;
        int64_t page = 0;
        if (paged) {
            table = int32(a[6], 2, at);
            own = int32(a[7], 2, at);
            len = int32(a[8], 1, at);
            if (!table || !own || !len || !whole(a[9], &page) || table->size(0) != B * W ||
                len->size(0) != B * W || own->size(1) != table->size(1))
                return other();
        }
        int lanes;
        if (!fits(paged ? own->size(0) : states[0].count, &lanes)) return other();
        for (const gdn_beam_pool &p : states)
            if (p.count != lanes) return other();
        if (lanes < 1 && B * W > 0) return other();
        // results
        at::Tensor made[2];
        const at::Tensor *to = &made[0], *to_table = &made[1];
        if (none(a[10])) {
            made[0] = at::empty({B, W}, slots->options());
            if (paged) made[1] = at::empty({B * W, table->size(1)}, slots->options());
        } else {
            PyObject *first = paged ? item(a[10], 2, 0) : a[10];
            if (!first || !(to = grid(first, B, W, at::kInt, at))) return other();
            if (paged && (!(to_table = int32(item(a[10], 2, 1), 2, at)) ||
                          to_table->sizes() != table->sizes()))
                return other();
            for (const at::Tensor *t : {parent, slots, table, own, len})
                if (t && (t->data_ptr() == to->data_ptr() ||
                          (paged && t->data_ptr() == to_table->data_ptr())))
                    return other();
        }
        gdn_beam_tables tables{};
        if (paged) {
            tables.page_table = data<int32_t>(*table);
            tables.table_out = data<int32_t>(*to_table);
            tables.own_pages = data<int32_t>(*own);
            tables.kv_len = data<int32_t>(*len);
            tables.table_stride = table->stride(0);
            tables.out_stride = to_table->stride(0);
            tables.own_stride = own->stride(0);
            if (!fits(table->size(1), &tables.max_pages) || !fits(page, &tables.page_size))
                return other();
        }
        if (!call<decltype(gdn_beam_reorder)>(a[0], a[1], at, (const int32_t *)data<int32_t>(*parent),
                  (const int32_t *)data<int32_t>(*slots), data<int32_t>(*to), iB, iW,
                  lanes > 1 ? lanes : 1, (const gdn_beam_pool *)states.data(), (int)states.size(),
                  paged ? (const gdn_beam_tables *)&tables : nullptr,
                  (const gdn_beam_pool *)caches.data(), (int)caches.size()))
            return nullptr;
        if (!none(a[10])) return paged ? tuple({ref(item(a[10], 2, 0)), ref(item(a[10], 2, 1))}) : ref(a[10]);
        PyObject *r = wrap(std::move(made[0]));
        return paged ? tuple({r, wrap(std::move(made[1]))}) : r;
    });
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_XSETREF(g_error, ref(type));
    Py_RETURN_NONE;
}

// (a METH_FASTCALL function as the table wants it)
template <typename F>
PyCFunction fast(F *f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }
PyMethodDef methods[] = {
    {"append", fast(append), METH_FASTCALL, nullptr},
    {"read", fast(read), METH_FASTCALL, nullptr},
    {"attn", fast(attn), METH_FASTCALL, nullptr},
    {"select", fast(select), METH_FASTCALL, nullptr},
    {"reorder", fast(reorder), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
