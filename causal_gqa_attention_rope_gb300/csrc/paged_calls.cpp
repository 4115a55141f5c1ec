// paged_calls.cpp -- the Python calls of the paged cache, argument marshalling
// only.  A step of a few tokens runs for 3 .. 7 us on the GPU; read attribute by
// attribute from Python, the checks of its 9 .. 14 tensors took 8.6 .. 11.2 us of
// host time, more than the launch (3.4 us).
//
// Each function reads what its Python namesake was given, checks dtypes, shapes,
// contiguity and device as the Python checks do, and calls the C ABI.  It answers
// the call's status, or None for anything but the plain case, without having
// called: the Python checks then find the words for it, or another route.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "na.h"

namespace {

decltype(&na_rope_append_kv_paged) g_append;
decltype(&na_attn_prefill_chunk_paged) g_prefill;
decltype(&na_attn_decode_paged) g_decode;
PyTypeObject *g_cfg_type, *g_rope_type, *g_cache_type;  // owned

// One call's arguments on their way; `ok` falls with the first that is not plain.
struct Reader {
    bool ok = true;
    int device = -1;

    long long integer(PyObject *o, long long lo, long long hi)
    {
        long long x = 0;
        if (ok && PyLong_Check(o)) {
            int over;
            x = PyLong_AsLongLongAndOverflow(o, &over);
            ok = !over && x >= lo && x <= hi;
        } else {
            ok = false;
        }
        return x;
    }
    int32_t i32(PyObject *o) { return (int32_t)integer(o, INT32_MIN, INT32_MAX); }

    // A borrowed attribute: instances keep what they hold while the call runs.
    PyObject *attr(PyObject *o, PyObject *name)
    {
        PyObject *x = ok ? PyObject_GetAttr(o, name) : nullptr;
        if (!x) {
            ok = false;
            PyErr_Clear();
            return Py_None;
        }
        Py_DECREF(x);
        return x;
    }
    double real(PyObject *o)
    {
        double x = ok ? PyFloat_AsDouble(o) : 0;
        if (x == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return x;
    }
    bool truth(PyObject *o)
    {
        ok = ok && PyBool_Check(o);
        return o == Py_True;
    }

    // A contiguous tensor of the call's device; null when it is not one.
    const at::Tensor *tensor(PyObject *o)
    {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.is_cuda() && t.layout() == at::kStrided && t.get_device() == device &&
             t.is_contiguous();
        return ok ? &t : nullptr;
    }
    // The same with a dtype and shape; a size of -1 matches any, the first has to
    // be at least its.  None gives a null pointer where it may be left out.
    void *ptr(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape,
              bool optional = false)
    {
        if (optional && o == Py_None)
            return nullptr;
        const at::Tensor *t = tensor(o);
        if (!t)
            return nullptr;
        ok = t->scalar_type() == type && t->dim() == (int64_t)shape.size();
        int i = 0;
        for (int64_t want : shape) {
            if (!ok)
                return nullptr;
            const int64_t got = t->size(i);
            ok = want < 0 || (i == 0 ? got >= want : got == want);
            i++;
        }
        return ok ? t->data_ptr() : nullptr;
    }
};

#define NAMES(X)                                                                              \
    X(num_heads) X(num_kv_heads) X(head_dim) X(rotary_dim) X(sm_scale) X(rms_eps) X(qk_norm)  \
    X(qk_norm_zero_centered) X(v_norm) X(out_gate) X(softcap) X(window) X(ring_cache) X(base) \
    X(yarn) X(factor) X(orig_max_pos) X(beta_fast) X(beta_slow) X(attn_factor) X(k) X(v)      \
    X(page_table) X(k_scale) X(v_scale) X(cuda_stream)
#define DECLARE(n) PyObject *s_##n;
NAMES(DECLARE)
#undef DECLARE

void read_cfg(Reader &r, PyObject *o, na_attn_cfg &c)
{
    r.ok = r.ok && Py_TYPE(o) == g_cfg_type;
    c.num_heads = r.i32(r.attr(o, s_num_heads));
    c.num_kv_heads = r.i32(r.attr(o, s_num_kv_heads));
    c.head_dim = r.i32(r.attr(o, s_head_dim));
    PyObject *rd = r.attr(o, s_rotary_dim);
    c.rotary_dim = rd == Py_None ? c.head_dim : r.i32(rd);
    c.sm_scale = (float)r.real(r.attr(o, s_sm_scale));
    c.rms_eps = (float)r.real(r.attr(o, s_rms_eps));
    c.flags = (r.truth(r.attr(o, s_qk_norm)) ? NA_QK_NORM : 0u) |
              (r.truth(r.attr(o, s_qk_norm_zero_centered)) ? NA_QK_NORM_ZERO_CENTERED : 0u) |
              (r.truth(r.attr(o, s_v_norm)) ? NA_V_NORM : 0u) |
              (r.truth(r.attr(o, s_out_gate)) ? NA_OUT_GATE : 0u) |
              (r.truth(r.attr(o, s_ring_cache)) ? NA_RING_CACHE : 0u);
    c.softcap = (float)r.real(r.attr(o, s_softcap));
    c.window = r.i32(r.attr(o, s_window));
}

void read_rope(Reader &r, PyObject *o, na_rope_params &p)
{
    r.ok = r.ok && Py_TYPE(o) == g_rope_type;
    p.base = r.real(r.attr(o, s_base));
    p.yarn = r.truth(r.attr(o, s_yarn));
    p.factor = r.real(r.attr(o, s_factor));
    p.orig_max_pos = r.i32(r.attr(o, s_orig_max_pos));
    p.beta_fast = r.real(r.attr(o, s_beta_fast));
    p.beta_slow = r.real(r.attr(o, s_beta_slow));
    p.attn_factor = r.real(r.attr(o, s_attn_factor));
}

void read_cache(Reader &r, PyObject *o, const na_attn_cfg &cfg, int64_t batch, na_paged_kv_cache &c)
{
    r.ok = r.ok && Py_TYPE(o) == g_cache_type;
    PyObject *k = r.attr(o, s_k), *v = r.attr(o, s_v), *table = r.attr(o, s_page_table);
    PyObject *ks = r.attr(o, s_k_scale), *vs = r.attr(o, s_v_scale);
    const bool bf16 = ks == Py_None && vs == Py_None;
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat8_e4m3fn;
    c.k = r.ptr(k, type, {-1, cfg.num_kv_heads, -1, cfg.head_dim});
    const at::Tensor *tk = r.tensor(k);
    const int64_t pages = tk ? tk->size(0) : 0, page_size = tk ? tk->size(2) : 0;
    c.v = r.ptr(v, type, {pages, cfg.num_kv_heads, page_size, cfg.head_dim});
    c.page_table = (const int32_t *)r.ptr(table, at::kInt, {batch, -1});
    c.k_scale = c.v_scale = nullptr;
    if (!bf16) {
        c.k_scale = (uint8_t *)r.ptr(ks, at::kByte, {pages, cfg.num_kv_heads});
        c.v_scale = (uint8_t *)r.ptr(vs, at::kByte, {pages, cfg.num_kv_heads});
    }
    if (!r.ok)
        return;
    // the pools agree in their number of pages; sizes fit the struct
    const at::Tensor &tt = THPVariable_Unpack(table);
    r.ok = THPVariable_Unpack(v).size(0) == pages &&
           (bf16 || (THPVariable_Unpack(ks).size(0) == pages && THPVariable_Unpack(vs).size(0) == pages)) &&
           pages <= INT32_MAX && page_size <= INT32_MAX && tt.size(0) <= INT32_MAX &&
           tt.size(1) <= INT32_MAX;
    c.num_pages = (int32_t)pages;
    c.page_size = (int32_t)page_size;
    c.batch = (int32_t)tt.size(0);
    c.pages_per_seq = (int32_t)tt.size(1);
    c.dtype = bf16 ? NA_KV_BF16 : NA_KV_E4M3;
}

void *read_workspace(Reader &r, PyObject *o, size_t &bytes)
{
    bytes = 0;
    if (o == Py_None)
        return nullptr;
    const at::Tensor *t = r.tensor(o);
    if (!t)
        return nullptr;
    bytes = (size_t)t->nbytes();
    return t->data_ptr();
}

// The tokens a packed call reads, and the sequences of cu_seqlens.
void read_packing(Reader &r, PyObject *cu, PyObject *q, PyObject *total, int64_t &batch, int64_t &tokens)
{
    const at::Tensor *tc = r.tensor(cu), *tq = r.tensor(q);
    batch = tc ? tc->numel() - 1 : 0;
    tokens = 0;
    if (total != Py_None)
        tokens = r.i32(total);
    else if (tq && tq->dim() > 0)
        tokens = tq->size(0);
    r.ok = r.ok && batch <= INT32_MAX && tokens <= INT32_MAX;
}

void *read_stream(Reader &r, PyObject *o)
{
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)r.device).stream();
    PyObject *h = r.attr(o, s_cuda_stream);
    if (!r.ok || !PyLong_Check(h)) {
        r.ok = false;
        return nullptr;
    }
    void *s = PyLong_AsVoidPtr(h);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        r.ok = false;
    }
    return s;
}

// Only once a tensor says that CUDA is up: asking starts it.
void start(Reader &r, PyObject *q)
{
    r.ok = THPVariable_Check(q) && THPVariable_Unpack(q).is_cuda();
    if (r.ok)
        r.device = c10::cuda::current_device();
}

PyObject *declined()
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

template <class F>
PyObject *answer(const Reader &r, F call)
{
    if (!r.ok)
        Py_RETURN_NONE;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// (cfg, rope, cu_seqlens, cache_lens, q, k, v, q_out, cache, q_norm_w, k_norm_w, status,
//  total_tokens, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 14)
        Py_RETURN_NONE;
    try {
        Reader r;
        na_attn_cfg cfg;
        na_rope_params rope;
        na_paged_kv_cache cache;
        int64_t B, T;
        start(r, a[4]);
        read_cfg(r, a[0], cfg);
        read_rope(r, a[1], rope);
        read_packing(r, a[2], a[4], a[12], B, T);
        const int64_t H = cfg.num_heads, KV = cfg.num_kv_heads, d = cfg.head_dim;
        r.ok = r.ok && B >= 0 && T >= 0;
        auto cu = (const int32_t *)r.ptr(a[2], at::kInt, {-1});
        auto lens = (const int32_t *)r.ptr(a[3], at::kInt, {B});
        void *q = r.ptr(a[4], at::kBFloat16, {T, H, d});
        void *k = r.ptr(a[5], at::kBFloat16, {T, KV, d});
        void *v = r.ptr(a[6], at::kBFloat16, {T, KV, d});
        void *q_out = r.ptr(a[7], at::kBFloat16, {T, H, d});
        read_cache(r, a[8], cfg, B, cache);
        void *qw = r.ptr(a[9], at::kBFloat16, {d}, true);
        void *kw = r.ptr(a[10], at::kBFloat16, {d}, true);
        r.ok = r.ok && (!qw || THPVariable_Unpack(a[9]).size(0) == d) &&
               (!kw || THPVariable_Unpack(a[10]).size(0) == d);
        auto status = (int32_t *)r.ptr(a[11], at::kInt, {1}, true);
        void *stream = read_stream(r, a[13]);
        return answer(r, [&] {
            return g_append(&cfg, &rope, (int32_t)B, cu, lens, (int32_t)T, q, k, v, qw, kw, q_out,
                            &cache, status, stream);
        });
    } catch (...) {  // a tensor without storage: Python's checks say so
        return declined();
    }
}

// (cfg, cu_seqlens, cache_lens, max_new_len, max_total_len, q_rot, cache, out, gate, workspace,
//  status, total_tokens, stream)
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13)
        Py_RETURN_NONE;
    try {
        Reader r;
        na_attn_cfg cfg;
        na_paged_kv_cache cache;
        int64_t B, T;
        size_t ws_bytes;
        start(r, a[5]);
        read_cfg(r, a[0], cfg);
        read_packing(r, a[1], a[5], a[11], B, T);
        const int64_t H = cfg.num_heads, d = cfg.head_dim;
        r.ok = r.ok && B >= 0 && T >= 0;
        auto cu = (const int32_t *)r.ptr(a[1], at::kInt, {-1});
        auto lens = (const int32_t *)r.ptr(a[2], at::kInt, {B});
        const int32_t max_new = r.i32(a[3]), max_total = r.i32(a[4]);
        void *q = r.ptr(a[5], at::kBFloat16, {T, H, d});
        read_cache(r, a[6], cfg, B, cache);
        void *out = r.ptr(a[7], at::kBFloat16, {T, H, d});
        void *gate = r.ptr(a[8], at::kBFloat16, {T, H, d}, true);
        void *ws = read_workspace(r, a[9], ws_bytes);
        auto status = (int32_t *)r.ptr(a[10], at::kInt, {1}, true);
        void *stream = read_stream(r, a[12]);
        return answer(r, [&] {
            return g_prefill(&cfg, (int32_t)B, cu, lens, (int32_t)T, max_new, max_total, q, &cache,
                             gate, out, ws, ws_bytes, status, stream);
        });
    } catch (...) {
        return declined();
    }
}

// (cfg, q_rot, cache, kv_lens, max_kv_len, out, probs, gate, workspace, num_splits, status,
//  stream)
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 12)
        Py_RETURN_NONE;
    try {
        Reader r;
        na_attn_cfg cfg;
        na_paged_kv_cache cache;
        size_t ws_bytes;
        start(r, a[1]);
        read_cfg(r, a[0], cfg);
        const int64_t H = cfg.num_heads, d = cfg.head_dim;
        void *q = r.ptr(a[1], at::kBFloat16, {-1, H, d});
        const int64_t B = r.ok ? THPVariable_Unpack(a[1]).size(0) : 0;
        r.ok = r.ok && B <= INT32_MAX;
        read_cache(r, a[2], cfg, B, cache);
        auto lens = (const int32_t *)r.ptr(a[3], at::kInt, {B});
        const int32_t max_kv = r.i32(a[4]);
        void *out = r.ptr(a[5], at::kBFloat16, {B, H, d});
        auto probs = (float *)r.ptr(a[6], at::kFloat, {B, H, -1}, true);
        int64_t stride = 0;
        if (probs)
            stride = THPVariable_Unpack(a[6]).size(2);
        void *gate = r.ptr(a[7], at::kBFloat16, {B, H, d}, true);
        // rows of a decode call are as many as its queries
        for (int i : {5, 6, 7})
            r.ok = r.ok && (a[i] == Py_None || THPVariable_Unpack(a[i]).size(0) == B);
        r.ok = r.ok && stride <= INT32_MAX;
        void *ws = read_workspace(r, a[8], ws_bytes);
        const int32_t splits = r.i32(a[9]);
        auto status = (int32_t *)r.ptr(a[10], at::kInt, {1}, true);
        void *stream = read_stream(r, a[11]);
        return answer(r, [&] {
            return g_decode(&cfg, (int32_t)B, q, &cache, lens, max_kv, gate, out, probs,
                            (int32_t)stride, splits, ws, ws_bytes, status, stream);
        });
    } catch (...) {
        return declined();
    }
}

// (addresses of the three C entries, the classes AttnConfig, RopeConfig, PagedKVCache)
PyObject *bind(PyObject *, PyObject *args)
{
    PyObject *fa, *fp, *fd;
    PyTypeObject *c, *r, *k;
    if (!PyArg_ParseTuple(args, "OOOO!O!O!", &fa, &fp, &fd, &PyType_Type, &c, &PyType_Type, &r,
                          &PyType_Type, &k))
        return nullptr;
    void *pa = PyLong_AsVoidPtr(fa), *pp = PyLong_AsVoidPtr(fp), *pd = PyLong_AsVoidPtr(fd);
    if (PyErr_Occurred())
        return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(pa);
    g_prefill = reinterpret_cast<decltype(g_prefill)>(pp);
    g_decode = reinterpret_cast<decltype(g_decode)>(pd);
    g_cfg_type = (PyTypeObject *)Py_NewRef((PyObject *)c);
    g_rope_type = (PyTypeObject *)Py_NewRef((PyObject *)r);
    g_cache_type = (PyTypeObject *)Py_NewRef((PyObject *)k);
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"append", (PyCFunction)(void *)append, METH_FASTCALL, nullptr},
    {"prefill", (PyCFunction)(void *)prefill, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void *)decode, METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged_calls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_calls()
{
#define INTERN(n)                                   \
    if (!(s_##n = PyUnicode_InternFromString(#n)))  \
        return nullptr;
    NAMES(INTERN)
#undef INTERN
    PyObject *m = PyModule_Create(&kModule);
    // the torch it reads tensors of (NA_TORCH: version and commit, by the build)
    if (m && PyModule_AddStringConstant(m, "torch", NA_TORCH) < 0)
        Py_CLEAR(m);
    return m;
}
