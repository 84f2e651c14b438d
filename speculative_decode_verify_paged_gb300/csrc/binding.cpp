/*
 * Native side of the Python binding for the calls around the attention (step
 * tables, norm and rotation, cross attention): checks the tensors and makes
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

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(build_tables), FAST(norm_rope), FAST(norm_rope_append), FAST(run_cross),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "spec_attn_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_spec_attn_calls(void) {
    n_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!n_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
