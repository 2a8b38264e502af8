// Native argument marshalling of the entry points that a serving loop calls
// once per layer and token (paged cache, windowed prefill).  A kernel takes a
// few microseconds there; reading the same tensors' attributes from Python and
// converting two dozen arguments through ctypes took 10 to 20 per call, this
// module takes one or two.  It checks shapes, dtypes and devices, allocates
// outputs and calls the C ABI (include/libattn.h) on the current CUDA stream;
// the Python functions of the package name and document each call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>

#include <exception>
#include <string>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "libattn.h"

namespace {

PyObject *g_error = nullptr;                           // AttnError(status, where)

struct Fail : std::exception {
    PyObject *type;
    std::string msg;
    Fail(PyObject *t, std::string m) : type(t), msg(std::move(m)) {}
};
struct PyFail : std::exception {};                     // a Python error is set already

[[noreturn]] void value_error(const char *msg) { throw Fail(PyExc_ValueError, msg); }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Fail(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int to_int(int64_t x) {
    if (x < INT_MIN || x > INT_MAX) value_error("a size does not fit 32 bits");
    return int(x);
}

int integer(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw PyFail();
    return to_int(x);
}

// a token count of any size: beyond 2^31 it means all
int tokens(PyObject *o) {
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    if (x == -1 && !over && PyErr_Occurred()) throw PyFail();
    if (over > 0 || x > INT_MAX) return INT_MAX;
    if (over < 0 || x < INT_MIN) return INT_MIN;
    return int(x);
}

float scale_of(PyObject *o) {
    if (o == Py_None) return 0.f;
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw PyFail();
    return float(x);
}

// The current call's device and stream; every tensor it takes is checked here.
struct Call {
    c10::DeviceIndex index = -1;
    c10::cuda::OptionalCUDAGuard guard;

    const at::Tensor &on(const at::Tensor &t) {
        if (!t.is_cuda()) value_error("libattn tensors must be on a CUDA device");
        if (index < 0) {
            index = t.get_device();
            guard.set_index(index);
        } else if (t.get_device() != index) {
            value_error("all tensors must be on the same device");
        }
        return t;
    }
    const at::Tensor &take(PyObject *o, const char *name) { return on(tensor(o, name)); }
    // contiguous int32 of n entries (one axis)
    int32_t *ints(PyObject *o, const char *name, int64_t n) {
        const at::Tensor &t = take(o, name);
        if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
            throw Fail(PyExc_ValueError, std::string(name) + " must be a contiguous int32 tensor [" +
                                             std::to_string(n) + "]");
        return static_cast<int32_t *>(t.data_ptr());
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream(index).stream(); }
};

// The element strides of all axes but the last (null: contiguous).
struct Outer {
    int64_t st[4];
    const int64_t *p = nullptr;
    explicit Outer(const at::Tensor &t) {
        if (t.is_contiguous()) return;
        const int n = int(t.dim()) - 1;
        if (n > 4) value_error("a tensor has more axes than any argument");
        if (t.size(n) != 1 && t.stride(n) != 1) value_error("the last (D) dimension must be contiguous");
        for (int i = 0; i < n; ++i) st[i] = t.stride(i);
        p = st;
    }
};

attn_dtype_t dtype_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return ATTN_F32;
        case at::kBFloat16: return ATTN_BF16;
        case at::kHalf: return ATTN_F16;
        default: throw Fail(PyExc_TypeError, "unsupported dtype (float32, bfloat16 or float16)");
    }
}

struct Table {
    int32_t *p;
    int B, M;
    int64_t stride;
    Table(Call &c, PyObject *o) {
        const at::Tensor &t = c.take(o, "page_table");
        if (t.scalar_type() != at::kInt || t.dim() != 2) value_error("page_table must be int32 [B, max_pages]");
        B = to_int(t.size(0));
        M = to_int(t.size(1));
        if (M > 1 && t.stride(1) != 1) value_error("the rows of page_table must be contiguous");
        stride = B > 1 ? t.stride(0) : M;
        p = static_cast<int32_t *>(t.data_ptr());
    }
};

struct Workspace {
    at::Tensor t;
    Workspace(Call &c, PyObject *o, size_t need, bool zeroed, const at::Tensor &like) {
        if (o == Py_None) {
            const auto opt = like.options().dtype(at::kByte);
            const int64_t n = need > 256 ? int64_t(need) : 256;
            t = zeroed ? at::zeros({n}, opt) : at::empty({n}, opt);
        } else {
            t = c.take(o, "workspace");
            if (!t.is_contiguous()) value_error("the workspace must be contiguous");
        }
    }
    void *ptr() const { return t.data_ptr(); }
    size_t bytes() const { return t.nbytes(); }
};

PyObject *done(attn_status_t st, const char *where) {
    if (st == ATTN_OK) Py_RETURN_NONE;
    PyObject *e = g_error ? PyObject_CallFunction(g_error, "is", int(st), where) : nullptr;
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, where);
    }
    throw PyFail();
}

// n entries of a one-axis tensor from `at` on: an output of its own that shares
// an allocation (an allocation costs as much as a launch).
at::Tensor part(const at::Tensor &t, int64_t at, int64_t n) {
    at::Tensor x = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
    x.unsafeGetTensorImpl()->set_storage_offset(at);
    x.unsafeGetTensorImpl()->set_sizes_contiguous(n);
    return x;
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

// The output: the caller's (checked by the shape and dtype of `like`) or a new
// contiguous one.  *own: a new reference to return.
at::Tensor output(Call &c, PyObject *o, const at::Tensor &like) {
    if (o == Py_None) return at::empty(like.sizes(), like.options());
    const at::Tensor &t = c.take(o, "o");
    if (t.sizes() != like.sizes() || t.scalar_type() != like.scalar_type())
        value_error("o must have q's shape and dtype");
    return t;
}

PyObject *returned(PyObject *given, const at::Tensor &t) {
    if (given == Py_None) return wrap(t);
    Py_INCREF(given);
    return given;
}

// q, k, v, window, sinks, o, scale
PyObject *causal_gqa_window_fwd(PyObject *const *a) {
    Call c;
    const at::Tensor &q = c.take(a[0], "q"), &k = c.take(a[1], "k"), &v = c.take(a[2], "v");
    if (q.dim() != 4 || k.dim() != 4 || k.size(0) != q.size(0) || k.size(3) != q.size(3) ||
        v.sizes() != k.sizes() || k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        value_error("k/v must be [B, Hkv, Nkv, D] with q's dtype");
    const at::Tensor o = output(c, a[5], q);
    const Outer sq(q), sk(k), sv(v), so(o);
    done(attn_causal_gqa_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                    to_int(q.size(0)), to_int(q.size(1)), to_int(k.size(1)),
                                    to_int(q.size(2)), to_int(k.size(2)), to_int(q.size(3)), sq.p, sk.p,
                                    sv.p, so.p, tokens(a[3]), tokens(a[4]), dtype_of(q), scale_of(a[6]),
                                    c.stream()),
         "attn_causal_gqa_window_fwd");
    return returned(a[5], o);
}

// q, k_pages, v_pages, page_table, seq_len, o, scale, window, sinks, workspace
PyObject *decode_gqa_paged(PyObject *const *a) {
    Call c;
    const at::Tensor &q = c.take(a[0], "q"), &k = c.take(a[1], "k_pages"), &v = c.take(a[2], "v_pages");
    const Table t(c, a[3]);
    if (q.dim() != 3 || k.dim() != 4 || k.size(3) != q.size(2) || q.size(0) != t.B || v.sizes() != k.sizes() ||
        k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        value_error("q [B,Hq,D], pages [P,Hkv,S,D] of q's dtype and page_table [B,max_pages] required");
    const int32_t *sl = c.ints(a[4], "seq_len", t.B);
    const int Hq = to_int(q.size(1)), Hkv = to_int(k.size(1)), D = to_int(q.size(2));
    const at::Tensor o = output(c, a[5], q);
    const Workspace ws(c, a[9], attn_decode_gqa_paged_workspace_bytes(t.B, Hq, Hkv, D), true, q);
    const Outer sq(q), sk(k), sv(v), so(o);
    done(attn_decode_gqa_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), t.p, sl, o.data_ptr(), t.B, Hq, Hkv,
                               D, to_int(k.size(0)), to_int(k.size(2)), t.M, t.stride, sq.p, sk.p, sv.p, so.p,
                               tokens(a[7]), tokens(a[8]), dtype_of(q), scale_of(a[6]), ws.ptr(), ws.bytes(),
                               c.stream()),
         "attn_decode_gqa_paged");
    return returned(a[5], o);
}

// k_pages, v_pages, k_new, v_new, page_table, seq_len, new_len, advance
PyObject *kv_append_paged(PyObject *const *a) {
    Call c;
    const at::Tensor &k = c.take(a[0], "k_pages"), &v = c.take(a[1], "v_pages");
    at::Tensor kn = c.take(a[2], "k_new"), vn = c.take(a[3], "v_new");
    const Table t(c, a[4]);
    if (kn.dim() == 3 && vn.dim() == 3) {
        kn = kn.unsqueeze(2);
        vn = vn.unsqueeze(2);
    }
    if (k.dim() != 4 || kn.dim() != 4 || v.sizes() != k.sizes() || vn.sizes() != kn.sizes() ||
        kn.size(1) != k.size(1) || kn.size(3) != k.size(3) || kn.size(0) != t.B ||
        v.scalar_type() != k.scalar_type() || kn.scalar_type() != k.scalar_type() ||
        vn.scalar_type() != k.scalar_type())
        value_error("pages [P,Hkv,S,D], new rows [B,Hkv,T,D] of one dtype, page_table [B,max_pages] required");
    int32_t *sl = c.ints(a[5], "seq_len", t.B);
    const int32_t *nl = a[6] == Py_None ? nullptr : c.ints(a[6], "new_len", t.B);
    const int advance = PyObject_IsTrue(a[7]);
    if (advance < 0) throw PyFail();
    const Outer sk(k), sv(v), skn(kn), svn(vn);
    return done(attn_kv_append_paged(k.data_ptr(), v.data_ptr(), kn.data_ptr(), vn.data_ptr(), t.p, sl, nl, t.B,
                                     to_int(kn.size(2)), to_int(k.size(1)), to_int(k.size(3)),
                                     to_int(k.size(0)), to_int(k.size(2)), t.M, t.stride, sk.p, sv.p, skn.p,
                                     svn.p, dtype_of(k), advance, c.stream()),
                "attn_kv_append_paged");
}

// A table of rope_frequencies (None: no rotation).
struct Rotary {
    const uint64_t *freq = nullptr;
    int dim = 0;
    Rotary(Call &c, PyObject *o) {
        if (o == Py_None) return;
        const at::Tensor &t = c.take(o, "freq");
        if (t.scalar_type() != at::kLong || t.dim() != 1 || !t.is_contiguous())
            value_error("freq must be a contiguous int64 tensor [rotary_dim / 2] (rope_frequencies)");
        freq = static_cast<const uint64_t *>(t.data_ptr());
        dim = to_int(2 * t.size(0));
    }
};

int truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw PyFail();
    return x;
}

// x, freq, positions, interleaved, inverse, mscale, o
PyObject *rope_fwd(PyObject *const *a) {
    Call c;
    const at::Tensor &x = c.take(a[0], "x");
    const Rotary rot(c, a[1]);
    const at::Tensor &pos = c.take(a[2], "positions");
    if (x.dim() != 3 && x.dim() != 4) value_error("x must be [N, H, D] or [B, H, N, D]");
    const bool packed = x.dim() == 3;
    const int64_t B = packed ? 1 : x.size(0), H = x.size(1), N = packed ? x.size(0) : x.size(2);
    const bool rows = !packed && pos.dim() == 2;
    if (pos.scalar_type() != at::kInt || (rows ? pos.size(0) != B || pos.size(1) != N : pos.dim() != 1 || pos.size(0) != N) ||
        (N > 1 && pos.stride(pos.dim() - 1) != 1))
        value_error("positions must be int32 [N] (or [B, N] beside a 4-D x), rows contiguous");
    const at::Tensor o = output(c, a[6], x);
    const Outer sx(x), so(o);
    // (batch, head, token) of packed rows
    const int64_t D = x.size(x.dim() - 1);
    const int64_t px[3] = {D, x.stride(1), x.stride(0)}, po[3] = {D, o.stride(1), o.stride(0)};
    const float mscale = float(PyFloat_AsDouble(a[5]));
    if (PyErr_Occurred()) throw PyFail();
    done(attn_rope_fwd(x.data_ptr(), o.data_ptr(), rot.freq, static_cast<const int32_t *>(pos.data_ptr()),
                       rows ? (B > 1 ? pos.stride(0) : 0) : 0, to_int(B), to_int(H), to_int(N), to_int(D), rot.dim,
                       truth(a[3]), truth(a[4]), mscale, packed ? px : sx.p, packed ? po : so.p, dtype_of(x),
                       c.stream()),
         "attn_rope_fwd");
    return returned(a[6], o);
}

// New tokens' rows as the two appends of packed rows take them.
struct NewRows {
    const at::Tensor &kn, &vn;
    at::Tensor q, qo;
    const int32_t *cu;
    int64_t N, Hkv, D;
    Outer skn, svn;
    NewRows(Call &c, PyObject *k, PyObject *v, PyObject *q_, PyObject *qo_, PyObject *cu_, int B)
        : kn(c.take(k, "k_new")), vn(c.take(v, "v_new")), skn(kn), svn(vn) {
        if (kn.dim() != 3 || vn.sizes() != kn.sizes() || vn.scalar_type() != kn.scalar_type())
            value_error("k_new and v_new must be [N, Hkv, D] of one dtype");
        N = kn.size(0);
        Hkv = kn.size(1);
        D = kn.size(2);
        cu = cu_ == Py_None ? nullptr : c.ints(cu_, "cu_new", int64_t(B) + 1);
        if (!cu && N != B) value_error("without cu_new there is one new token per sequence");
        if (q_ != Py_None) {
            q = c.take(q_, "q");
            if (q.dim() != 3 || q.size(0) != N || q.size(2) != D || q.scalar_type() != kn.scalar_type())
                value_error("q must be [N, Hq, D] of k_new's dtype");
            if (qo_ == Py_None) {
                qo = at::empty(q.sizes(), q.options());
            } else {
                qo = c.take(qo_, "q_out");
                if (qo.sizes() != q.sizes() || qo.scalar_type() != q.scalar_type())
                    value_error("q_out must have q's shape and dtype");
            }
        } else if (qo_ != Py_None) {
            value_error("q_out without q");
        }
    }
    const void *q_ptr() const { return q.defined() ? q.data_ptr() : nullptr; }
    void *qo_ptr() const { return qo.defined() ? qo.data_ptr() : nullptr; }
    int Hq() const { return q.defined() ? to_int(q.size(1)) : 0; }
    PyObject *result(PyObject *qo_) const {
        if (!qo.defined()) Py_RETURN_NONE;
        return returned(qo_, qo);
    }
};

// k_pages, v_pages, k_new, v_new, page_table, seq_len, freq, cu_new, q, q_out, interleaved, mscale, advance
PyObject *kv_append_paged_rope(PyObject *const *a) {
    Call c;
    const at::Tensor &k = c.take(a[0], "k_pages"), &v = c.take(a[1], "v_pages");
    const Table t(c, a[4]);
    const NewRows n(c, a[2], a[3], a[8], a[9], a[7], t.B);
    if (k.dim() != 4 || v.sizes() != k.sizes() || n.Hkv != k.size(1) || n.D != k.size(3) ||
        v.scalar_type() != k.scalar_type() || n.kn.scalar_type() != k.scalar_type())
        value_error("pages [P,Hkv,S,D] and new rows [N,Hkv,D] of one dtype required");
    int32_t *sl = c.ints(a[5], "seq_len", t.B);
    const Rotary rot(c, a[6]);
    const Outer sk(k), sv(v), sq(n.q.defined() ? n.q : n.kn), sqo(n.qo.defined() ? n.qo : n.kn);
    const double mscale = PyFloat_AsDouble(a[11]);
    if (PyErr_Occurred()) throw PyFail();
    done(attn_kv_append_paged_rope(k.data_ptr(), v.data_ptr(), n.kn.data_ptr(), n.vn.data_ptr(), n.q_ptr(),
                                   n.qo_ptr(), t.p, sl, n.cu, rot.freq, t.B, to_int(n.N), n.Hq(), to_int(n.Hkv),
                                   to_int(n.D), rot.dim, truth(a[10]), float(mscale), to_int(k.size(0)),
                                   to_int(k.size(2)), t.M, t.stride, sk.p, sv.p, n.skn.p, n.svn.p, sq.p, sqo.p,
                                   dtype_of(k), truth(a[12]), c.stream()),
         "attn_kv_append_paged_rope");
    return n.result(a[9]);
}

// A cache held in 4 bits: uint8 [(layers,) P, Hkv, S, D + D / 8], the rows of a
// (page, head) contiguous.
struct PagesQ4 {
    const at::Tensor &t;
    int P, Hkv, S, D, layers = 1;
    int64_t st[3];                                     // of all axes but the last two
    const int64_t *p = nullptr;
    PagesQ4(Call &c, PyObject *o, bool with_layers = false) : t(c.take(o, "kv_pages")) {
        const int64_t n = t.dim();
        if (t.scalar_type() != at::kByte || (n != 4 && !(with_layers && n == 5)))
            value_error("kv_pages must be uint8 [P, Hkv, S, D + D / 8]");
        const int64_t row = t.size(n - 1);
        D = row == 72 ? 64 : row == 144 ? 128 : 0;
        if (D == 0) value_error("a row of kv_pages has D + D / 8 bytes, D 64 or 128");
        P = to_int(t.size(n - 4));
        Hkv = to_int(t.size(n - 3));
        S = to_int(t.size(n - 2));
        if (n == 5) layers = to_int(t.size(0));
        if (t.is_contiguous()) return;
        if (t.stride(n - 1) != 1 || (S > 1 && t.stride(n - 2) != row))
            value_error("the rows of a (page, head) of kv_pages must be contiguous");
        for (int i = 0; i < n - 2; ++i) st[i + (with_layers && n == 4)] = t.stride(i);
        if (with_layers && n == 4) st[0] = 16;         // one layer: not stepped along
        p = st;
    }
};

// kv_pages, k_new, v_new, page_table, seq_len, freq, cu_new, q, q_out, interleaved, mscale, advance
PyObject *kv_append_paged_q4(PyObject *const *a) {
    Call c;
    const PagesQ4 pg(c, a[0]);
    const Table t(c, a[3]);
    const NewRows n(c, a[1], a[2], a[7], a[8], a[6], t.B);
    if (n.Hkv != pg.Hkv || n.D != pg.D) value_error("new rows [N,Hkv,D] must have the pages' heads and channels");
    int32_t *sl = c.ints(a[4], "seq_len", t.B);
    const Rotary rot(c, a[5]);
    const Outer sq(n.q.defined() ? n.q : n.kn), sqo(n.qo.defined() ? n.qo : n.kn);
    const double mscale = PyFloat_AsDouble(a[10]);
    if (PyErr_Occurred()) throw PyFail();
    done(attn_kv_append_paged_q4(pg.t.data_ptr(), n.kn.data_ptr(), n.vn.data_ptr(), n.q_ptr(), n.qo_ptr(), t.p, sl,
                                 n.cu, rot.freq, t.B, to_int(n.N), n.Hq(), pg.Hkv, pg.D, rot.dim, truth(a[9]),
                                 float(mscale), pg.P, pg.S, t.M, t.stride, pg.p, n.skn.p, n.svn.p, sq.p, sqo.p,
                                 dtype_of(n.kn), truth(a[11]), c.stream()),
         "attn_kv_append_paged_q4");
    return n.result(a[8]);
}

// kv_pages, page_table, cu_len, k, v, start
PyObject *kv_gather_paged_q4(PyObject *const *a) {
    Call c;
    const PagesQ4 pg(c, a[0]);
    const Table t(c, a[1]);
    const int32_t *cu = c.ints(a[2], "cu_len", int64_t(t.B) + 1);
    const at::Tensor &k = c.take(a[3], "k"), &v = c.take(a[4], "v");
    const int32_t *start = a[5] == Py_None ? nullptr : c.ints(a[5], "start", t.B);
    if (k.dim() != 3 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || k.size(1) != pg.Hkv ||
        k.size(2) != pg.D)
        value_error("k and v must be [N, Hkv, D] of one dtype with the pages' heads and channels");
    const Outer sk(k), sv(v);
    done(attn_kv_gather_paged_q4(pg.t.data_ptr(), t.p, start, cu, k.data_ptr(), v.data_ptr(), t.B, to_int(k.size(0)),
                                 pg.Hkv, pg.D, pg.P, pg.S, t.M, t.stride, pg.p, sk.p, sv.p, dtype_of(k), c.stream()),
         "attn_kv_gather_paged_q4");
    Py_INCREF(a[3]);
    Py_INCREF(a[4]);
    return Py_BuildValue("(NN)", a[3], a[4]);
}

// kv_pages, copy_src, copy_dst, count
PyObject *kv_pages_copy_q4(PyObject *const *a) {
    Call c;
    const PagesQ4 pg(c, a[0], true);
    const int n = to_int(c.take(a[1], "copy_src").numel());
    const int32_t *src = c.ints(a[1], "copy_src", n), *dst = c.ints(a[2], "copy_dst", n);
    const int32_t *count = a[3] == Py_None ? nullptr : c.ints(a[3], "count", 1);
    if (n == 0) Py_RETURN_NONE;
    return done(attn_kv_pages_copy_q4(pg.t.data_ptr(), src, dst, n, count, pg.layers, pg.P, pg.Hkv, pg.S, pg.D, pg.p,
                                      c.stream()),
                "attn_kv_pages_copy_q4");
}

// q, kv_pages, page_table, seq_len, o, scale, window, sinks, workspace
PyObject *decode_gqa_paged_q4(PyObject *const *a) {
    Call c;
    const at::Tensor &q = c.take(a[0], "q");
    const PagesQ4 pg(c, a[1]);
    const Table t(c, a[2]);
    if (q.dim() != 3 || q.size(0) != t.B || q.size(2) != pg.D)
        value_error("q [B,Hq,D], kv_pages [P,Hkv,S,D + D / 8] and page_table [B,max_pages] required");
    const int32_t *sl = c.ints(a[3], "seq_len", t.B);
    const int Hq = to_int(q.size(1));
    const at::Tensor o = output(c, a[4], q);
    const Workspace ws(c, a[8], attn_decode_gqa_paged_q4_workspace_bytes(t.B, Hq, pg.Hkv, pg.D), true, q);
    const Outer sq(q), so(o);
    done(attn_decode_gqa_paged_q4(q.data_ptr(), pg.t.data_ptr(), t.p, sl, o.data_ptr(), t.B, Hq, pg.Hkv, pg.D, pg.P,
                                  pg.S, t.M, t.stride, sq.p, pg.p, so.p, tokens(a[6]), tokens(a[7]), dtype_of(q),
                                  scale_of(a[5]), ws.ptr(), ws.bytes(), c.stream()),
         "attn_decode_gqa_paged_q4");
    return returned(a[4], o);
}

// q, k, v, cu_q, cu_k, window, sinks, o, scale
PyObject *causal_gqa_varlen_fwd(PyObject *const *a) {
    Call c;
    const at::Tensor &q = c.take(a[0], "q"), &k = c.take(a[1], "k"), &v = c.take(a[2], "v");
    if (q.dim() != 3 || k.dim() != 3 || k.size(2) != q.size(2) || v.sizes() != k.sizes() ||
        k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        value_error("q must be [Nq, Hq, D], k and v [Nkv, Hkv, D] with q's dtype");
    const at::Tensor &cq = c.take(a[3], "cu_q");
    const int64_t n = cq.numel();
    if (n < 2) value_error("cu_q must be int32 [B + 1]");
    const int32_t *cu_q = c.ints(a[3], "cu_q", n);
    const int32_t *cu_k = a[4] == Py_None ? cu_q : c.ints(a[4], "cu_k", n);
    const at::Tensor o = output(c, a[7], q);
    const Outer sq(q), sk(k), sv(v), so(o);
    done(attn_causal_gqa_varlen_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), cu_q, cu_k,
                                    to_int(n - 1), to_int(q.size(0)), to_int(k.size(0)), to_int(q.size(1)),
                                    to_int(k.size(1)), to_int(q.size(2)), sq.p, sk.p, sv.p, so.p, tokens(a[5]),
                                    tokens(a[6]), dtype_of(q), scale_of(a[8]), c.stream()),
         "attn_causal_gqa_varlen_fwd");
    return returned(a[7], o);
}

// page_table, seq_len, add_len, page_refs, page_size, workspace
PyObject *kv_pages_reserve(PyObject *const *a) {
    Call c;
    const Table t(c, a[0]);
    const int32_t *sl = c.ints(a[1], "seq_len", t.B), *add = c.ints(a[2], "add_len", t.B);
    const at::Tensor &r = c.take(a[3], "page_refs");
    const int P = to_int(r.numel());
    int32_t *refs = c.ints(a[3], "page_refs", P);
    const Workspace ws(c, a[5], attn_kv_pages_workspace_bytes(P), false, r);
    return done(attn_kv_pages_reserve(t.p, sl, add, refs, t.B, P, integer(a[4]), t.M, t.stride, ws.ptr(),
                                      ws.bytes(), c.stream()),
                "attn_kv_pages_reserve");
}

// page_table, seq_len, page_refs, page_size, window, sinks
PyObject *kv_pages_free(PyObject *const *a) {
    Call c;
    const Table t(c, a[0]);
    const int32_t *sl = c.ints(a[1], "seq_len", t.B);
    const int P = to_int(c.take(a[2], "page_refs").numel());
    int32_t *refs = c.ints(a[2], "page_refs", P);
    return done(attn_kv_pages_free(t.p, sl, refs, t.B, P, integer(a[3]), t.M, t.stride, tokens(a[4]),
                                   tokens(a[5]), c.stream()),
                "attn_kv_pages_free");
}

// page_table, seq_len, page_refs, src, dst, page_size, workspace
PyObject *kv_pages_fork(PyObject *const *a) {
    Call c;
    const Table t(c, a[0]);
    int32_t *sl = c.ints(a[1], "seq_len", t.B);
    const at::Tensor &r = c.take(a[2], "page_refs");
    const int P = to_int(r.numel());
    int32_t *refs = c.ints(a[2], "page_refs", P);
    const int n = to_int(c.take(a[3], "src").numel());
    const int32_t *src = c.ints(a[3], "src", n), *dst = c.ints(a[4], "dst", n);
    const Workspace ws(c, a[6], attn_kv_pages_workspace_bytes(P), false, r);
    const at::Tensor lists = at::empty({2 * int64_t(n)}, r.options());
    const at::Tensor cs = part(lists, 0, n), cd = part(lists, n, n);
    if (n > 0)
        done(attn_kv_pages_fork(t.p, sl, refs, src, dst, n, static_cast<int32_t *>(cs.data_ptr()),
                                static_cast<int32_t *>(cd.data_ptr()), t.B, P, integer(a[5]), t.M, t.stride,
                                ws.ptr(), ws.bytes(), c.stream()),
             "attn_kv_pages_fork");
    return Py_BuildValue("(NN)", wrap(cs), wrap(cd));
}

// page_table, page_refs, new_table, new_refs, workspace
PyObject *kv_pages_compact(PyObject *const *a) {
    Call c;
    const Table t(c, a[0]);
    const Table nt(c, a[2] == Py_None ? a[0] : a[2]);
    if (nt.B != t.B || nt.M != t.M) value_error("new_table must be like page_table");
    const at::Tensor &r = c.take(a[1], "page_refs");
    const int P = to_int(r.numel());
    const int32_t *refs = c.ints(a[1], "page_refs", P);
    int32_t *nr = c.ints(a[3] == Py_None ? a[1] : a[3], "new_refs", P);
    const Workspace ws(c, a[4], attn_kv_pages_workspace_bytes(P), false, r);
    const int64_t cap = P / 2;
    const at::Tensor lists = at::empty({2 * cap + 1}, r.options());
    const at::Tensor cs = part(lists, 0, cap), cd = part(lists, cap, cap), n = part(lists, 2 * cap, 1);
    done(attn_kv_pages_compact(t.p, refs, nt.p, nr, static_cast<int32_t *>(cs.data_ptr()),
                               static_cast<int32_t *>(cd.data_ptr()), static_cast<int32_t *>(n.data_ptr()),
                               t.B, P, t.M, t.stride, nt.stride, ws.ptr(), ws.bytes(), c.stream()),
         "attn_kv_pages_compact");
    return Py_BuildValue("(NNN)", wrap(cs), wrap(cd), wrap(n));
}

// k_pages, v_pages, copy_src, copy_dst, count
PyObject *kv_pages_copy(PyObject *const *a) {
    Call c;
    at::Tensor k = c.take(a[0], "k_pages"), v = c.take(a[1], "v_pages");
    if (k.dim() == 4 && v.dim() == 4) {
        k = k.unsqueeze(0);
        v = v.unsqueeze(0);
    }
    if (k.dim() != 5 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
        value_error("pages [P,Hkv,S,D] or [layers,P,Hkv,S,D] of one dtype required");
    const int n = to_int(c.take(a[2], "copy_src").numel());
    const int32_t *src = c.ints(a[2], "copy_src", n), *dst = c.ints(a[3], "copy_dst", n);
    const int32_t *count = a[4] == Py_None ? nullptr : c.ints(a[4], "count", 1);
    if (n == 0) Py_RETURN_NONE;
    const Outer sk(k), sv(v);
    return done(attn_kv_pages_copy(k.data_ptr(), v.data_ptr(), src, dst, n, count, to_int(k.size(0)),
                                   to_int(k.size(1)), to_int(k.size(2)), to_int(k.size(3)), to_int(k.size(4)),
                                   sk.p, sv.p, dtype_of(k), c.stream()),
                "attn_kv_pages_copy");
}

// Python entry of one of the functions above with its argument count; no C++
// exception leaves it.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Fail &e) {
        PyErr_SetString(e.type, e.msg.c_str());
    } catch (const PyFail &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_XDECREF(g_error);
    Py_INCREF(cls);
    g_error = cls;
    Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void *)entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    ENTRY(causal_gqa_window_fwd, 7), ENTRY(decode_gqa_paged, 10), ENTRY(kv_append_paged, 8),
    ENTRY(kv_pages_reserve, 6),      ENTRY(kv_pages_free, 6),     ENTRY(kv_pages_fork, 7),
    ENTRY(kv_pages_compact, 5),      ENTRY(kv_pages_copy, 5),     ENTRY(rope_fwd, 7),
    ENTRY(kv_append_paged_rope, 13), ENTRY(kv_append_paged_q4, 12), ENTRY(kv_gather_paged_q4, 6),
    ENTRY(kv_pages_copy_q4, 4),      ENTRY(decode_gqa_paged_q4, 9), ENTRY(causal_gqa_varlen_fwd, 9),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr,
                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_native() { return PyModule_Create(&g_module); }
