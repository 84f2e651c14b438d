/*
 * Native side of the Python binding for the calls around the attention (step
 * tables, norm and rotation, cross attention, trees): checks the tensors and makes
 * the C ABI call in one step.  A decode step makes these calls once a layer on
 * kernels of a few microseconds, and the same checks cost more than the launch
 * when written in Python (12 tensors: 7.8 of 10.5 us) or through the tensors'
 * Python attributes (2.7 of 6.2); here they are reads of the tensor objects.
 *
 * A bad tensor raises ValueError before anything is launched; the call's
 * spec_attn_status is returned as an int.  The library itself does not depend
 * on torch, only this module does.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <vector>

#include "spec_attn.h"

static PyObject* n_cuda_stream;

enum { kMaxDims = 4 };
static constexpr at::ScalarType t_bf16 = at::kBFloat16, t_f32 = at::kFloat, t_i32 = at::kInt, t_i64 = at::kLong,
                                t_u8 = at::kByte;

/* A tensor as a call wants it; shape entries of -1 take the tensor's own size. */
typedef struct {
    const char* what;
    at::ScalarType dtype;
    int nd;
    int64_t shape[kMaxDims];
    const int64_t* strides;   /* elements; NULL: contiguous */
} want_t;

/* A checked tensor's address, as whatever pointer the call takes. */
struct Address {
    void* p = nullptr;
    template <class T>
    operator T*() const {
        return static_cast<T*>(p);
    }
};

static int check(const at::Tensor& t, want_t* w, long* dev, Address* out) {
    if (!t.is_cuda()) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", w->what);
        return -1;
    }
    if (*dev < 0) *dev = c10::cuda::current_device();
    const long at = t.get_device();
    if (at != *dev) {
        PyErr_Format(PyExc_ValueError, "%s must be on the current device, cuda:%ld, got cuda:%ld", w->what, *dev, at);
        return -1;
    }
    if (t.scalar_type() != w->dtype) {
        PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", w->what, c10::toString(w->dtype),
                     c10::toString(t.scalar_type()));
        return -1;
    }
    const at::IntArrayRef size = t.sizes(), step = t.strides();
    if (static_cast<int>(size.size()) != w->nd) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions, got %d", w->what, w->nd, static_cast<int>(size.size()));
        return -1;
    }
    for (int i = 0; i < w->nd; ++i) {
        if (w->shape[i] < 0) w->shape[i] = size[i];
        if (w->shape[i] != size[i]) {
            PyErr_Format(PyExc_ValueError, "%s must have %lld entries in dimension %d, got %lld", w->what,
                         static_cast<long long>(w->shape[i]), i, static_cast<long long>(size[i]));
            return -1;
        }
        if (w->strides && size[i] > 1 && step[i] != w->strides[i]) {
            PyErr_Format(PyExc_ValueError, "%s must have a stride of %lld elements in dimension %d, got %lld", w->what,
                         static_cast<long long>(w->strides[i]), i, static_cast<long long>(step[i]));
            return -1;
        }
    }
    if (!w->strides && !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", w->what);
        return -1;
    }
    out->p = t.mutable_data_ptr();
    return 0;
}

/* Address of `t` after its checks, NULL for None.  *dev is the current device, asked for with the first tensor. */
static int address(PyObject* t, want_t* w, long* dev, Address* out) {
    out->p = nullptr;
    if (t == Py_None) return 0;
    if (!THPVariable_Check(t)) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", w->what);
        return -1;
    }
    try {
        return check(THPVariable_Unpack(t), w, dev, out);
    } catch (const std::exception& e) {   /* (a tensor without storage, a failing driver) */
        PyErr_Format(PyExc_RuntimeError, "%s: %s", w->what, e.what());
        return -1;
    }
}

/* Handle of `stream` (a torch stream, or None: the current one of the device). */
static int stream_of(PyObject* stream, long dev, spec_attn_stream_t* out) {
    if (stream == Py_None) {
        try {
            if (dev < 0) dev = c10::cuda::current_device();
            *out = reinterpret_cast<spec_attn_stream_t>(
                c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
        } catch (const std::exception& e) {
            PyErr_SetString(PyExc_RuntimeError, e.what());
            return -1;
        }
        return 0;
    }
    PyObject* o = PyObject_GetAttr(stream, n_cuda_stream);
    if (!o) return -1;
    void* p = PyLong_AsVoidPtr(o);
    *out = reinterpret_cast<spec_attn_stream_t>(p);
    Py_DECREF(o);
    return (!p && PyErr_Occurred()) ? -1 : 0;
}

/* Integers of a tuple. */
static int ints(PyObject* tuple, int n, int64_t* out) {
    if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != n) {
        PyErr_SetString(PyExc_TypeError, "not a plan of this call");
        return -1;
    }
    for (int i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) return -1;
    }
    return 0;
}

static int count_args(const char* name, Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
    return -1;
}

/* The workspace, one-dimensional bytes. */
static int workspace_of(PyObject* t, long* dev, Address* out, int64_t* bytes) {
    want_t w = {"workspace", t_u8, 1, {-1}, NULL};
    if (address(t, &w, dev, out)) return -1;
    *bytes = out->p ? w.shape[0] : 0;
    return 0;
}

/* build_tables((page_size, max_w, max_seq_len), ctx_lens, window_lens, prev_seq_lens, prev_free_count, free_pages,
 * block_table, seq_lens, q_indptr, free_count, positions, slot_map, workspace, stream) */
static PyObject* build_tables(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    int64_t c[3], bytes;
    if (count_args("build_tables", n, 14) || ints(a[0], 3, c)) return NULL;
    long dev = -1;
    Address ctx, win, prev, count0, pages, table, seq, indptr, count, pos, slot, ws;
    want_t w = {"ctx_lens", t_i32, 1, {-1}, NULL};
    if (address(a[1], &w, &dev, &ctx)) return NULL;
    const int64_t P = w.shape[0];
#define ONE(arg, name, size, to)                          \
    {                                                     \
        want_t x = {name, t_i32, 1, {size}, NULL};        \
        if (address(a[arg], &x, &dev, &to)) return NULL;  \
    }
    ONE(2, "window_lens", P, win)
    ONE(3, "prev_seq_lens", P, prev)
    ONE(4, "prev_free_count", 1, count0)
    want_t f = {"free_pages", t_i32, 1, {-1}, NULL}, b = {"block_table", t_i32, 2, {P, -1}, NULL};
    want_t s = {"slot_map", t_i64, 1, {-1}, NULL};
    if (address(a[5], &f, &dev, &pages) || address(a[6], &b, &dev, &table)) return NULL;
    ONE(7, "seq_lens", P, seq)
    ONE(8, "q_indptr", P + 1, indptr)
    ONE(9, "free_count", 1, count)
    if (address(a[11], &s, &dev, &slot)) return NULL;
    ONE(10, "positions", s.shape[0], pos)
#undef ONE
    spec_attn_stream_t st;
    if (workspace_of(a[12], &dev, &ws, &bytes) || stream_of(a[13], dev, &st)) return NULL;
    if (P < 0 || f.shape[0] < 0 || b.shape[1] < 0 || s.shape[0] < 0) return PyLong_FromLong(SPEC_ATTN_E_INVALID_ARG);
    if (P > INT32_MAX || s.shape[0] > INT32_MAX || f.shape[0] > INT32_MAX || b.shape[1] > INT32_MAX ||
        c[0] > INT32_MAX || c[1] > INT32_MAX || c[0] < INT32_MIN || c[1] < INT32_MIN)
        return PyLong_FromLong(SPEC_ATTN_E_UNSUPPORTED);
    const spec_attn_tables_problem p = {(int32_t)P, (int32_t)s.shape[0], (int32_t)c[0], (int32_t)f.shape[0],
                                        (int32_t)b.shape[1], (int32_t)c[1], c[2]};
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_build_tables(&p, ctx, win, prev, count0, pages, table, seq, indptr, count, pos, slot, ws,
                                    (size_t)bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* What a norm_rope plan tells: handle, Hq, Hkv, d, axes, the five row strides (0: dense), KV dtype, page size,
 * pages, page strides in bytes (0: dense). */
enum { kHandle, kHq, kHkv, kD, kAxes, kQs, kKs, kVs, kQos, kKos, kKvDtype, kPageSize, kPages, kKvStride, kScStride, kNr };

/* Rows of heads, `stride` elements apart. */
static int rows_of(PyObject* t, const char* what, int64_t n, int64_t h, int64_t d, int64_t stride, long* dev, Address* out,
                   int64_t* got_n) {
    const int64_t strides[3] = {stride ? stride : h * d, d, 1};
    want_t w = {what, t_bf16, 3, {n, h, d}, strides};
    if (address(t, &w, dev, out)) return -1;
    if (got_n && t != Py_None) *got_n = w.shape[0];
    return 0;
}

typedef struct {
    int64_t c[kNr];
    int64_t n;
    long dev;
    Address q, k, qw, kw, pos;
} nr_call;

/* a: plan, q, k, q_weight, k_weight, positions */
static int nr_args(PyObject* plan, PyObject* q, PyObject* k, PyObject* qw, PyObject* kw, PyObject* pos, nr_call* r) {
    if (ints(plan, kNr, r->c)) return -1;
    const int64_t* c = r->c;
    r->dev = -1;
    r->n = -1;
    if (rows_of(q, "q", -1, c[kHq], c[kD], c[kQs], &r->dev, &r->q, &r->n) ||
        rows_of(k, "k", r->n, c[kHkv], c[kD], c[kKs], &r->dev, &r->k, &r->n))
        return -1;
    want_t a = {"q_weight", t_f32, 1, {c[kD]}, NULL}, b = {"k_weight", t_f32, 1, {c[kD]}, NULL};
    want_t p = {"positions", t_i32, 2, {c[kAxes], r->n}, NULL};
    if (address(qw, &a, &r->dev, &r->qw) || address(kw, &b, &r->dev, &r->kw) || address(pos, &p, &r->dev, &r->pos))
        return -1;
    if (r->n < 0 || r->n > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "q and k must give at most 2^31 - 1 rows");
        return -1;
    }
    return 0;
}

/* norm_rope(plan, q, k, q_weight, k_weight, positions, q_out, k_out, stream) */
static PyObject* norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    nr_call r;
    if (count_args("norm_rope", n, 9) || nr_args(a[0], a[1], a[2], a[3], a[4], a[5], &r)) return NULL;
    const int64_t* c = r.c;
    Address qo, ko;
    spec_attn_stream_t st;
    if (rows_of(a[6], "q_out", r.n, c[kHq], c[kD], c[kQos], &r.dev, &qo, NULL) ||
        rows_of(a[7], "k_out", r.n, c[kHkv], c[kD], c[kKos], &r.dev, &ko, NULL) || stream_of(a[8], r.dev, &st))
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_norm_rope((const spec_attn_norm_rope_plan*)(intptr_t)c[kHandle], (int32_t)r.n, r.q, r.k, r.qw, r.kw,
                                 r.pos, qo, ko, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* A pool of pages [pages, Hkv, page_size, row], pages `bytes` apart (0: dense). */
static int pool_of(PyObject* t, const char* what, const int64_t* c, int64_t row, int64_t bytes, int size, at::ScalarType dtype,
                   long* dev, Address* out) {
    const int64_t dense = c[kHkv] * c[kPageSize] * row;
    const int64_t strides[4] = {bytes ? bytes / size : dense, c[kPageSize] * row, row, 1};
    want_t w = {what, dtype, 4, {c[kPages], c[kHkv], c[kPageSize], row}, strides};
    return address(t, &w, dev, out);
}

/* norm_rope_append(plan, q, k, v, q_weight, k_weight, positions, slot_map, q_out, k_pool, v_pool, workspace, k_scales,
 * v_scales, k_gscale, v_gscale, stream) */
static PyObject* norm_rope_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    nr_call r;
    if (count_args("norm_rope_append", n, 17) || nr_args(a[0], a[1], a[2], a[4], a[5], a[6], &r)) return NULL;
    const int64_t* c = r.c;
    const int fp4 = c[kKvDtype] == SPEC_ATTN_KV_NVFP4;
    const int64_t row = fp4 ? c[kD] / 2 : c[kD];
    const at::ScalarType kind = fp4 ? t_u8 : t_bf16;
    Address v, slot, qo, kp, vp, ks, vs, ws;
    int64_t bytes;
    spec_attn_stream_t st;
    want_t s = {"slot_map", t_i64, 1, {r.n}, NULL};
    if (rows_of(a[3], "v", r.n, c[kHkv], c[kD], c[kVs], &r.dev, &v, NULL) || address(a[7], &s, &r.dev, &slot) ||
        rows_of(a[8], "q_out", r.n, c[kHq], c[kD], c[kQos], &r.dev, &qo, NULL) ||
        pool_of(a[9], "k_pool", c, row, c[kKvStride], fp4 ? 1 : 2, kind, &r.dev, &kp) ||
        pool_of(a[10], "v_pool", c, row, c[kKvStride], fp4 ? 1 : 2, kind, &r.dev, &vp) ||
        workspace_of(a[11], &r.dev, &ws, &bytes) ||
        pool_of(a[12], "k_scales", c, c[kD] / 16, c[kScStride], 1, t_u8, &r.dev, &ks) ||
        pool_of(a[13], "v_scales", c, c[kD] / 16, c[kScStride], 1, t_u8, &r.dev, &vs))
        return NULL;
    const double kg = PyFloat_AsDouble(a[14]), vg = PyFloat_AsDouble(a[15]);
    if (PyErr_Occurred() || stream_of(a[16], r.dev, &st)) return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_norm_rope_append((const spec_attn_norm_rope_plan*)(intptr_t)c[kHandle], (int32_t)r.n, r.q, r.k, v,
                                        r.qw, r.kw, r.pos, slot, qo, kp, vp, ks, vs, (float)kg, (float)vg, ws,
                                        (size_t)bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* run_cross((handle, P, query rows, Hq, Hkv, d, state rows, row stride), q, k, v, q_indptr, kv_start, kv_len, o, lse,
 * workspace, stream) */
static PyObject* run_cross(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    int64_t c[8], bytes;
    if (count_args("run_cross", n, 11) || ints(a[0], 8, c)) return NULL;
    const int64_t P = c[1], rows = c[2], hq = c[3], hkv = c[4], d = c[5];
    long dev = -1;
    Address q, k, v, indptr, start, len, o, lse, ws;
    spec_attn_stream_t st;
    want_t wq = {"q", t_bf16, 3, {rows, hq, d}, NULL}, wo = {"o", t_bf16, 3, {rows, hq, d}, NULL};
    want_t wl = {"lse", t_f32, 2, {rows, hq}, NULL}, wi = {"q_indptr", t_i32, 1, {P + 1}, NULL};
    want_t ws_ = {"kv_start", t_i32, 1, {P}, NULL}, wn = {"kv_len", t_i32, 1, {P}, NULL};
    if (address(a[1], &wq, &dev, &q) || rows_of(a[2], "k", c[6], hkv, d, c[7], &dev, &k, NULL) ||
        rows_of(a[3], "v", c[6], hkv, d, c[7], &dev, &v, NULL) || address(a[4], &wi, &dev, &indptr) ||
        address(a[5], &ws_, &dev, &start) || address(a[6], &wn, &dev, &len) || address(a[7], &wo, &dev, &o) ||
        address(a[8], &wl, &dev, &lse) || workspace_of(a[9], &dev, &ws, &bytes) || stream_of(a[10], dev, &st))
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_run_cross((const spec_attn_cross_plan*)(intptr_t)c[0], q, k, v, indptr, start, len, o, lse, ws,
                                 (size_t)bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* What a masked plan tells: handle, P, query rows, Hq, Hkv, d, pages, page size, table stride, KV dtype, page strides in
 * bytes (0: dense), whether the windows are trees, words of a mask row. */
enum { mHandle, mP, mRows, mHq, mHkv, mD, mPages, mPageSize, mTable, mKvDtype, mKvStride, mScStride, mTree, mWords, mN };

/* Pools and scales, with the layout pool_of reads. */
static int caches_of(PyObject* const* a, const int64_t* m, long* dev, Address* kp, Address* vp, Address* ks, Address* vs) {
    int64_t c[kNr] = {};
    c[kHkv] = m[mHkv];
    c[kPageSize] = m[mPageSize];
    c[kPages] = m[mPages];
    const int fp4 = m[mKvDtype] == SPEC_ATTN_KV_NVFP4;
    const int64_t row = fp4 ? m[mD] / 2 : m[mD];
    const at::ScalarType kind = fp4 ? t_u8 : t_bf16;
    return pool_of(a[0], "k_pool", c, row, m[mKvStride], fp4 ? 1 : 2, kind, dev, kp) ||
           pool_of(a[1], "v_pool", c, row, m[mKvStride], fp4 ? 1 : 2, kind, dev, vp) ||
           pool_of(a[2], "k_scales", c, m[mD] / 16, m[mScStride], 1, t_u8, dev, ks) ||
           pool_of(a[3], "v_scales", c, m[mD] / 16, m[mScStride], 1, t_u8, dev, vs);
}

/* run_masked(plan, q, k_pool, v_pool, k_scales, v_scales, k_gscale, v_gscale, block_table, seq_lens, q_indptr, row_mask,
 * positions, o, lse, workspace, stream) */
static PyObject* run_masked(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    int64_t m[mN], bytes;
    if (count_args("run_masked", n, 17) || ints(a[0], mN, m)) return NULL;
    long dev = -1;
    Address q, kp, vp, ks, vs, table, seq, indptr, mask, pos, o, lse, ws;
    spec_attn_stream_t st;
    want_t wq = {"q", t_bf16, 3, {m[mRows], m[mHq], m[mD]}, NULL}, wo = {"o", t_bf16, 3, {m[mRows], m[mHq], m[mD]}, NULL};
    want_t wl = {"lse", t_f32, 2, {m[mRows], m[mHq]}, NULL}, wt = {"block_table", t_i32, 2, {m[mP], m[mTable]}, NULL};
    want_t wn = {"seq_lens", t_i32, 1, {m[mP]}, NULL}, wi = {"q_indptr", t_i32, 1, {m[mP] + 1}, NULL};
    want_t wm = {"row_mask", t_i32, 2, {m[mRows], m[mWords]}, NULL}, wp = {"positions", t_i32, 1, {m[mRows]}, NULL};
    if (address(a[1], &wq, &dev, &q) || caches_of(a + 2, m, &dev, &kp, &vp, &ks, &vs)) return NULL;
    const double kg = PyFloat_AsDouble(a[6]), vg = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return NULL;
    if (address(a[8], &wt, &dev, &table) || address(a[9], &wn, &dev, &seq) || address(a[10], &wi, &dev, &indptr) ||
        address(a[11], &wm, &dev, &mask) || address(a[12], &wp, &dev, &pos) || address(a[13], &wo, &dev, &o) ||
        address(a[14], &wl, &dev, &lse) || workspace_of(a[15], &dev, &ws, &bytes) || stream_of(a[16], dev, &st))
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_run_masked((const spec_attn_masked_plan*)(intptr_t)m[mHandle], q, kp, vp, ks, vs, (float)kg,
                                  (float)vg, table, seq, indptr, mask, pos, o, lse, ws, (size_t)bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* The tensors both tree calls take: parents [rows], seq_lens [P], q_indptr [P + 1]. */
static int tree_of(PyObject* const* a, PyObject* seqs, PyObject* ptr, long* dev, Address* parents, Address* seq,
                   Address* indptr, int64_t* rows, int64_t* reqs) {
    want_t wp = {"parents", t_i32, 1, {-1}, NULL}, wn = {"seq_lens", t_i32, 1, {-1}, NULL};
    if (address(a[0], &wp, dev, parents) || address(seqs, &wn, dev, seq)) return -1;
    want_t wi = {"q_indptr", t_i32, 1, {wn.shape[0] + 1}, NULL};
    if (address(ptr, &wi, dev, indptr)) return -1;
    *rows = wp.shape[0];
    *reqs = wn.shape[0];
    return 0;
}

static int fits(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }

/* build_tree((max_w, window_left, sink_keys), parents, seq_lens, q_indptr, positions, row_mask, workspace, stream) */
static PyObject* build_tree(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    int64_t c[3], bytes, rows, P;
    if (count_args("build_tree", n, 8) || ints(a[0], 3, c)) return NULL;
    long dev = -1;
    Address parents, seq, indptr, pos, mask, ws;
    spec_attn_stream_t st;
    if (tree_of(a + 1, a[2], a[3], &dev, &parents, &seq, &indptr, &rows, &P)) return NULL;
    want_t wp = {"positions", t_i32, 1, {rows}, NULL}, wm = {"row_mask", t_i32, 2, {rows, -1}, NULL};
    if (address(a[4], &wp, &dev, &pos) || address(a[5], &wm, &dev, &mask) || workspace_of(a[6], &dev, &ws, &bytes) ||
        stream_of(a[7], dev, &st))
        return NULL;
    if (P < 0 || rows < 0 || wm.shape[1] < 1) return PyLong_FromLong(SPEC_ATTN_E_INVALID_ARG);
    if (!fits(P) || !fits(rows) || !fits(wm.shape[1]) || !fits(c[0]) || !fits(c[1]) || !fits(c[2]))
        return PyLong_FromLong(SPEC_ATTN_E_UNSUPPORTED);
    const spec_attn_tree_problem p = {(int32_t)P, (int32_t)rows, (int32_t)c[0], (int32_t)wm.shape[1], (int32_t)c[1],
                                      (int32_t)c[2], 1, 0};
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_build_tree(&p, parents, seq, indptr, pos, mask, ws, (size_t)bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* accept_tree((max_w,), parents, draft_tokens, target_tokens, seq_lens, q_indptr, path, accept_lens, next_tokens, ctx_lens,
 * workspace, stream) */
static PyObject* accept_tree(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    int64_t c[1], bytes, rows, P;
    if (count_args("accept_tree", n, 12) || ints(a[0], 1, c)) return NULL;
    long dev = -1;
    Address parents, draft, target, seq, indptr, path, accepted, next, ctx, ws;
    spec_attn_stream_t st;
    if (tree_of(a + 1, a[4], a[5], &dev, &parents, &seq, &indptr, &rows, &P)) return NULL;
    want_t wd = {"draft_tokens", t_i64, 1, {rows}, NULL}, wt = {"target_tokens", t_i64, 1, {rows}, NULL};
    want_t wp = {"path", t_i32, 2, {P, -1}, NULL}, wa = {"accept_lens", t_i32, 1, {P}, NULL};
    want_t wn = {"next_tokens", t_i64, 1, {P}, NULL}, wc = {"ctx_lens", t_i32, 1, {P}, NULL};
    if (address(a[2], &wd, &dev, &draft) || address(a[3], &wt, &dev, &target) || address(a[6], &wp, &dev, &path) ||
        address(a[7], &wa, &dev, &accepted) || address(a[8], &wn, &dev, &next) || address(a[9], &wc, &dev, &ctx) ||
        workspace_of(a[10], &dev, &ws, &bytes) || stream_of(a[11], dev, &st))
        return NULL;
    if (P < 0 || rows < 0 || wp.shape[1] < 1) return PyLong_FromLong(SPEC_ATTN_E_INVALID_ARG);
    if (!fits(P) || !fits(rows) || !fits(wp.shape[1]) || !fits(c[0])) return PyLong_FromLong(SPEC_ATTN_E_UNSUPPORTED);
    const spec_attn_tree_problem p = {(int32_t)P, (int32_t)rows, (int32_t)c[0], 0, 0, 0, (int32_t)wp.shape[1], 0};
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_accept_tree(&p, parents, draft, target, seq, indptr, path, accepted, next, ctx, ws, (size_t)bytes,
                                   st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* move_kv((max_seq_len,), k_pools, v_pools, k_scales, v_scales, block_table, seq_lens, q_indptr, path, accept_lens,
 * workspace, stream): pools are lists of tensors, the scales' None for bf16.  The first layer's pools give the shapes. */
static PyObject* move_kv(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    int64_t c[1], bytes;
    if (count_args("move_kv", n, 12) || ints(a[0], 1, c)) return NULL;
    for (int i = 1; i < 5; ++i)
        if (!(PyList_Check(a[i]) || (i > 2 && a[i] == Py_None))) {
            PyErr_SetString(PyExc_TypeError, "pools and scales are lists of tensors, one for each layer");
            return NULL;
        }
    const Py_ssize_t layers = PyList_GET_SIZE(a[1]);
    const int fp4 = a[3] != Py_None;
    for (int i = 2; i < (fp4 ? 5 : 3); ++i)
        if (!PyList_Check(a[i]) || PyList_GET_SIZE(a[i]) != layers) {
            PyErr_SetString(PyExc_ValueError, "pools and scales must have the same number of layers");
            return NULL;
        }
    if (!fp4 && a[4] != Py_None) {
        PyErr_SetString(PyExc_ValueError, "k_scales and v_scales go together");
        return NULL;
    }
    spec_attn_move_problem p = {};
    long dev = -1;
    Address table, seq, indptr, path, accepted, ws;
    spec_attn_stream_t st;
    want_t wn = {"seq_lens", t_i32, 1, {-1}, NULL};
    if (address(a[6], &wn, &dev, &seq)) return NULL;
    const int64_t P = wn.shape[0];
    want_t wi = {"q_indptr", t_i32, 1, {P + 1}, NULL}, wt = {"block_table", t_i32, 2, {P, -1}, NULL};
    want_t wp = {"path", t_i32, 2, {P, -1}, NULL}, wa = {"accept_lens", t_i32, 1, {P}, NULL};
    if (address(a[5], &wt, &dev, &table) || address(a[7], &wi, &dev, &indptr) || address(a[8], &wp, &dev, &path) ||
        address(a[9], &wa, &dev, &accepted) || workspace_of(a[10], &dev, &ws, &bytes) || stream_of(a[11], dev, &st))
        return NULL;
    int64_t m[mN] = {};
    m[mKvDtype] = fp4;
    if (layers > 0) {   /* shapes and strides of the first layer's K */
        PyObject* k0 = PyList_GET_ITEM(a[1], 0);
        PyObject* s0 = fp4 ? PyList_GET_ITEM(a[3], 0) : Py_None;
        if (!THPVariable_Check(k0) || THPVariable_Unpack(k0).dim() != 4 ||
            (fp4 && (!THPVariable_Check(s0) || THPVariable_Unpack(s0).dim() != 4))) {
            PyErr_SetString(PyExc_ValueError, "pools and scales must be CUDA tensors [pages, Hkv, page_size, row]");
            return NULL;
        }
        const at::Tensor& k = THPVariable_Unpack(k0);
        m[mPages] = k.size(0);
        m[mHkv] = k.size(1);
        m[mPageSize] = k.size(2);
        m[mD] = fp4 ? k.size(3) * 2 : k.size(3);
        if (k.size(0) > 1) m[mKvStride] = k.stride(0) * (fp4 ? 1 : 2);
        if (fp4 && k.size(0) > 1) m[mScStride] = THPVariable_Unpack(s0).stride(0);
    }
    std::vector<void*> at[4];
    try {
        for (auto& v : at) v.resize(static_cast<size_t>(layers));
    } catch (const std::exception&) {
        return PyErr_NoMemory();
    }
    for (Py_ssize_t l = 0; l < layers; ++l) {
        PyObject* const pools[4] = {PyList_GET_ITEM(a[1], l), PyList_GET_ITEM(a[2], l),
                                    fp4 ? PyList_GET_ITEM(a[3], l) : Py_None, fp4 ? PyList_GET_ITEM(a[4], l) : Py_None};
        Address x[4];
        if (caches_of(pools, m, &dev, &x[0], &x[1], &x[2], &x[3])) return NULL;
        for (int i = 0; i < 4; ++i) at[i][static_cast<size_t>(l)] = x[i].p;
    }
    if (P < 0 || wt.shape[1] < 0 || wp.shape[1] < 0) return PyLong_FromLong(SPEC_ATTN_E_INVALID_ARG);
    if (layers == 0) return PyLong_FromLong(SPEC_ATTN_OK);
    if (!fits(P) || !fits(layers) || !fits(m[mHkv]) || !fits(m[mD]) || !fits(m[mPageSize]) || !fits(m[mPages]) ||
        !fits(wt.shape[1]) || !fits(wp.shape[1]))
        return PyLong_FromLong(SPEC_ATTN_E_UNSUPPORTED);
    p.num_reqs = (int32_t)P;
    p.num_layers = (int32_t)layers;
    p.num_kv_heads = (int32_t)m[mHkv];
    p.head_dim = (int32_t)m[mD];
    p.page_size = (int32_t)m[mPageSize];
    p.num_pages = (int32_t)m[mPages];
    p.block_table_stride = (int32_t)wt.shape[1];
    p.kv_dtype = fp4;
    p.path_stride = (int32_t)wp.shape[1];
    p.max_seq_len = c[0];
    p.kv_page_stride = m[mKvStride];
    p.scale_page_stride = m[mScStride];
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = spec_attn_move_kv(&p, at[0].data(), at[1].data(), at[2].data(), at[3].data(), table, seq, indptr, path,
                               accepted, ws, (size_t)bytes, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(build_tables), FAST(norm_rope), FAST(norm_rope_append), FAST(run_cross),
                                FAST(run_masked), FAST(build_tree), FAST(accept_tree), FAST(move_kv),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "spec_attn_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_spec_attn_calls(void) {
    n_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!n_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
