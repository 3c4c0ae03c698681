// Argument marshalling of the rotary and windowed calls for Python.
//
// These calls may be a few microseconds of GPU work, less than the interpreter
// takes to check their tensors one attribute at a time and to hand them to
// ctypes (measured on the Grace host: 8.7 us a decode call in Python and
// ctypes, of which the launch is about 2).  Here the regular case (CUDA tensors
// on the current device, of the expected type and shape, dense) is checked and
// called directly.  Anything else returns None, and the package's Python
// function says what is wrong or does it the general way.  A tensor's type,
// device, shape, strides and address come from one call, its DLPack capsule (0.2
// us, against 0.35 for its Python methods one by one), whose layout is a
// published standard; the functions that make it and name the current device and
// stream are handed in (setup), so nothing here depends on a torch build.  The
// package does without this module where it is not built.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "kvattn.h"

namespace {

// Names and objects that are looked up once (setup()).
PyObject *s_desc, *s_pool, *s_k_pool;
PyObject *g_dlpack_fn, *g_device_fn, *g_stream_fn;

// The tensor description of a DLPack capsule (as the standard lays it out).
struct DlTensor {
    void* data;
    struct {
        int32_t type, id;
    } device;
    int32_t ndim;
    struct {
        uint8_t code, bits;
        uint16_t lanes;
    } dtype;
    int64_t* shape;
    int64_t* strides;  // in elements; null: dense
    uint64_t byte_offset;
};
constexpr int32_t kDlCuda = 2;

// An element type: its DLPack code and bits (bits 0: any type).
struct Type {
    uint8_t code, bits;
};
constexpr Type kAny{0, 0}, kInt32{0, 32}, kFloat32{2, 32}, kBfloat16{4, 16};

constexpr int kMaxDims = 4;

struct View {
    void* ptr;
    int ndim;
    int64_t dim[kMaxDims];
    int64_t stride[kMaxDims];
    int64_t nbytes;  // of a dense tensor
};

bool to_int(PyObject* o, int64_t* out)  // steals o
{
    if (!o) return false;
    const long long v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    if (v == -1 && PyErr_Occurred()) return false;
    *out = v;
    return true;
}

// A tensor of the type on the device; dense, unless its strides are asked for
// (they say nothing of a dimension of one element).
bool view(PyObject* t, Type type, int64_t device, bool strides, View* v)
{
    PyObject* cap = PyObject_CallOneArg(g_dlpack_fn, t);
    if (!cap) return false;
    const DlTensor* d = static_cast<const DlTensor*>(PyCapsule_GetPointer(cap, "dltensor"));
    bool ok = d && d->device.type == kDlCuda && d->device.id == device && d->ndim <= kMaxDims && d->dtype.lanes == 1 &&
              d->dtype.bits % 8 == 0 &&
              (type.bits == 0 || (d->dtype.code == type.code && d->dtype.bits == type.bits));
    if (ok) {
        v->ptr = static_cast<char*>(d->data) + d->byte_offset;
        v->ndim = d->ndim;
        int64_t dense = 1;  // the stride that a dense tensor has
        for (int i = d->ndim - 1; i >= 0; --i) {
            v->dim[i] = d->shape[i];
            v->stride[i] = d->strides ? d->strides[i] : dense;
            if (!strides && d->shape[i] > 1 && v->stride[i] != dense) ok = false;
            dense *= d->shape[i];
        }
        if (dense == 0) ok = true;  // without elements every tensor is dense
        v->nbytes = dense * (d->dtype.bits / 8);
    }
    Py_DECREF(cap);
    return ok;
}

bool has_shape(const View& v, int ndim, int64_t a, int64_t b = 0, int64_t c = 0)
{
    return v.ndim == ndim && v.dim[0] == a && (ndim < 2 || v.dim[1] == b) && (ndim < 3 || v.dim[2] == c);
}

// The bytes of a ctypes structure, held while this object lives.
template <typename T>
class Struct {
public:
    explicit Struct(PyObject* o)
    {
        held_ = o && PyObject_GetBuffer(o, &b_, PyBUF_SIMPLE) == 0;
    }
    ~Struct()
    {
        if (held_) PyBuffer_Release(&b_);
    }
    const T* get() const { return held_ && b_.len == (Py_ssize_t)sizeof(T) ? static_cast<const T*>(b_.buf) : nullptr; }

private:
    Py_buffer b_;
    bool held_;
};

Type type_of(const kvattn_config* cfg) { return cfg->dtype == KVATTN_BF16 ? kBfloat16 : kFloat32; }

// The current device and its current stream.
bool here(int64_t* device, void** stream)
{
    if (!g_device_fn) return false;
    PyObject* d = PyObject_CallNoArgs(g_device_fn);
    if (!d) return false;
    const long long v = PyLong_AsLongLong(d);
    PyObject* s = PyObject_CallOneArg(g_stream_fn, d);
    Py_DECREF(d);
    int64_t raw;
    if (!to_int(s, &raw) || (v == -1 && PyErr_Occurred())) return false;
    *device = v;
    *stream = reinterpret_cast<void*>(raw);
    return true;
}

// A Cache or CacheFP8 of the package that fits the config: its descriptor.
struct CacheArg {
    PyObject* desc = nullptr;
    ~CacheArg() { Py_XDECREF(desc); }
    bool get(PyObject* cache, bool fp8, const kvattn_config* cfg, int64_t device)
    {
        PyObject* pool = PyObject_GetAttr(cache, fp8 ? s_pool : s_k_pool);
        if (!pool) return false;
        View v;
        const bool ok = view(pool, fp8 ? kAny : type_of(cfg), device, false, &v) &&
                        v.ndim == 4 && v.dim[1] == cfg->num_kv_heads && (fp8 ? 128 : v.dim[3]) == cfg->head_dim;
        Py_DECREF(pool);
        return ok && (desc = PyObject_GetAttr(cache, s_desc)) != nullptr;
    }
};

bool as_i32(PyObject* o, int32_t* out)
{
    const long long v = PyLong_AsLongLong(o);
    if ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX) return false;
    *out = (int32_t)v;
    return true;
}

// None: not the regular case (an error that the checks met on the way, a
// missing attribute for one, is dropped: the Python function meets it again).
PyObject* irregular()
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

template <typename F>
PyObject* call(F&& f)
{
    kvattn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// setup(to_dlpack, current_device, current_raw_stream)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "setup takes 3 arguments");
        return nullptr;
    }
    PyObject** const to[3] = {&g_dlpack_fn, &g_device_fn, &g_stream_fn};
    for (int i = 0; i < 3; ++i) {
        Py_INCREF(args[i]);
        Py_XSETREF(*to[i], args[i]);
    }
    Py_RETURN_NONE;
}

// decode_window(fp8, cfg, cache, q, block_table, seq_lens, max_seq_len, window,
//               num_sinks, num_splits, out, workspace)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    int64_t device;
    void* stream;
    int32_t max_len, window, sinks, splits;
    if (n != 12 || !here(&device, &stream)) return irregular();
    const bool fp8 = a[0] == Py_True;
    const Struct<kvattn_config> cfg_s(a[1]);
    const kvattn_config* cfg = cfg_s.get();
    CacheArg cache;
    View q, table, lens, out, ws;
    if (!cfg || !cache.get(a[2], fp8, cfg, device) || !view(a[3], type_of(cfg), device, false, &q) ||
        !view(a[4], kInt32, device, false, &table) || !view(a[5], kInt32, device, false, &lens) ||
        !as_i32(a[6], &max_len) || !as_i32(a[7], &window) || !as_i32(a[8], &sinks) || !as_i32(a[9], &splits) ||
        !view(a[10], type_of(cfg), device, false, &out) || !view(a[11], kAny, device, false, &ws))
        return irregular();
    const int64_t B = q.dim[0];
    if (!has_shape(q, 3, B, cfg->num_q_heads, cfg->head_dim) || !has_shape(out, 3, B, cfg->num_q_heads, cfg->head_dim) ||
        !has_shape(lens, 1, B) || table.ndim != 2 || table.dim[0] < B || table.dim[1] > INT32_MAX || B > INT32_MAX)
        return irregular();
    if (fp8) {
        const Struct<kvattn_cache_fp8> d(cache.desc);
        if (!d.get()) return irregular();
        return call([&] {
            return kvattn_decode_window_fp8(cfg, d.get(), q.ptr, (const int32_t*)table.ptr, (int32_t)table.dim[1],
                                            (const int32_t*)lens.ptr, (int32_t)B, max_len, window, sinks, splits, out.ptr,
                                            ws.ptr, (size_t)ws.nbytes, stream);
        });
    }
    const Struct<kvattn_cache> d(cache.desc);
    if (!d.get()) return irregular();
    return call([&] {
        return kvattn_decode_window(cfg, d.get(), q.ptr, (const int32_t*)table.ptr, (int32_t)table.dim[1],
                                    (const int32_t*)lens.ptr, (int32_t)B, max_len, window, sinks, splits, out.ptr, ws.ptr,
                                    (size_t)ws.nbytes, stream);
    });
}

// prefill_window(fp8, cfg, cache, q, cu_q_lens, prefix_lens, block_table,
//                max_q_len, window, num_sinks, out, workspace or None)
PyObject* prefill_window(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    int64_t device;
    void* stream;
    int32_t max_q, window, sinks;
    if (n != 12 || !here(&device, &stream)) return irregular();
    const bool fp8 = a[0] == Py_True;
    const Struct<kvattn_config> cfg_s(a[1]);
    const kvattn_config* cfg = cfg_s.get();
    CacheArg cache;
    View q, cu, prefix, table, out, ws;
    if (!cfg || cfg->dtype != KVATTN_BF16 || !cache.get(a[2], fp8, cfg, device) ||
        !view(a[3], kBfloat16, device, false, &q) || !view(a[4], kInt32, device, false, &cu) ||
        !view(a[5], kInt32, device, false, &prefix) || !view(a[6], kInt32, device, false, &table) ||
        !as_i32(a[7], &max_q) || !as_i32(a[8], &window) || !as_i32(a[9], &sinks) ||
        !view(a[10], kBfloat16, device, false, &out))
        return irregular();
    if (fp8 && !view(a[11], kAny, device, false, &ws)) return irregular();
    const int64_t T = q.dim[0], C = prefix.dim[0];
    if (!has_shape(q, 3, T, cfg->num_q_heads, cfg->head_dim) || !has_shape(out, 3, T, cfg->num_q_heads, cfg->head_dim) ||
        !has_shape(prefix, 1, C) || !has_shape(cu, 1, C + 1) || table.ndim != 2 || table.dim[0] < C ||
        table.dim[1] > INT32_MAX || T > INT32_MAX || C > INT32_MAX)
        return irregular();
    if (fp8) {
        const Struct<kvattn_cache_fp8> d(cache.desc);
        if (!d.get()) return irregular();
        return call([&] {
            return kvattn_prefill_window_fp8(cfg, d.get(), q.ptr, (const int32_t*)cu.ptr, (const int32_t*)prefix.ptr,
                                             (const int32_t*)table.ptr, (int32_t)table.dim[1], (int32_t)C, max_q,
                                             (int32_t)T, window, sinks, out.ptr, ws.ptr, (size_t)ws.nbytes, stream);
        });
    }
    const Struct<kvattn_cache> d(cache.desc);
    if (!d.get()) return irregular();
    return call([&] {
        return kvattn_prefill_window(cfg, d.get(), q.ptr, (const int32_t*)cu.ptr, (const int32_t*)prefix.ptr,
                                     (const int32_t*)table.ptr, (int32_t)table.dim[1], (int32_t)C, max_q, (int32_t)T,
                                     window, sinks, out.ptr, stream);
    });
}

// A [T, heads, D] view whose rows are dense.
bool token_rows(PyObject* t, Type type, int64_t device, int64_t heads, int64_t d, View* v)
{
    if (!view(t, type, device, true, v) || v->ndim != 3 || v->dim[1] != heads || v->dim[2] != d) return false;
    if (v->stride[2] != 1 || (heads > 1 && v->stride[1] != d)) return false;
    if (v->dim[0] <= 1) v->stride[0] = heads * d;
    return true;
}

// rotary_append(fp8, cfg, rotary, cache, q, k, v, positions, seq_ids, block_table, q_out or None)
PyObject* rotary_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    int64_t device;
    void* stream;
    if (n != 11 || !here(&device, &stream)) return irregular();
    const bool fp8 = a[0] == Py_True;
    const Struct<kvattn_config> cfg_s(a[1]);
    const Struct<kvattn_rotary> rot(a[2]);
    const kvattn_config* cfg = cfg_s.get();
    CacheArg cache;
    View q, k, v, pos, ids, table, out;
    if (!cfg || !rot.get() || !cache.get(a[3], fp8, cfg, device)) return irregular();
    const Type dt = type_of(cfg);
    if (!token_rows(a[4], dt, device, cfg->num_q_heads, cfg->head_dim, &q) ||
        !token_rows(a[5], dt, device, cfg->num_kv_heads, cfg->head_dim, &k) ||
        !token_rows(a[6], dt, device, cfg->num_kv_heads, cfg->head_dim, &v) ||
        !view(a[7], kInt32, device, false, &pos) || !view(a[8], kInt32, device, false, &ids) ||
        !view(a[9], kInt32, device, false, &table))
        return irregular();
    const int64_t T = q.dim[0];
    out.ptr = nullptr;
    if (a[10] != Py_None && (!view(a[10], dt, device, false, &out) ||
                             !has_shape(out, 3, T, cfg->num_q_heads, cfg->head_dim)))
        return irregular();
    if (k.dim[0] != T || v.dim[0] != T || !has_shape(pos, 1, T) || !has_shape(ids, 1, T) || table.ndim != 2 ||
        table.dim[0] > INT32_MAX || table.dim[1] > INT32_MAX || T > INT32_MAX)
        return irregular();
    auto run = [&](auto fn, auto* desc) {
        return call([&] {
            return fn(cfg, rot.get(), desc, q.ptr, q.stride[0], k.ptr, k.stride[0], v.ptr, v.stride[0], out.ptr,
                      (const int32_t*)pos.ptr, (const int32_t*)ids.ptr, (const int32_t*)table.ptr, (int32_t)table.dim[0],
                      (int32_t)table.dim[1], (int32_t)T, stream);
        });
    };
    if (fp8) {
        const Struct<kvattn_cache_fp8> d(cache.desc);
        return d.get() ? run(kvattn_rotary_append_fp8, d.get()) : irregular();
    }
    const Struct<kvattn_cache> d(cache.desc);
    return d.get() ? run(kvattn_rotary_append, d.get()) : irregular();
}

#define KVATTN_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KVATTN_METHOD(setup), KVATTN_METHOD(decode_window), KVATTN_METHOD(prefill_window),
                         KVATTN_METHOD(rotary_append), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void)
{
    if (!(s_desc = PyUnicode_InternFromString("desc")) || !(s_pool = PyUnicode_InternFromString("pool")) ||
        !(s_k_pool = PyUnicode_InternFromString("k_pool")))
        return nullptr;
    return PyModule_Create(&module);
}
