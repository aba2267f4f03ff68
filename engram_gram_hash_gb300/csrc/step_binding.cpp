// The Python binding's marshalling for the calls of a decode step (block
// tables, head norm + rotation, cache append, paged attention): tensors to the plain structures of
// engram.h and back.  These calls run several times per layer and token on
// kernels of a few microseconds, so what a call costs the host decides how fast
// small steps go; reading the tensors here costs about a tenth of what it does
// through attribute lookups.  No arithmetic, no CUDA work of its own: the
// checks, torch::empty for outputs, one call of libengram each.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/engram.h"

namespace {

// libengram's entry points, set by bind()
decltype(&engram_qk_norm_rope) fn_qk = nullptr;
decltype(&engram_kv_append) fn_append = nullptr;
decltype(&engram_paged_attention) fn_attend = nullptr;
decltype(&engram_paged_attention_workspace_bytes) fn_bytes = nullptr;
decltype(&engram_kv_plan) fn_plan = nullptr;
decltype(&engram_kv_append_q8) fn_append8 = nullptr;
decltype(&engram_paged_attention_q8) fn_attend8 = nullptr;
decltype(&engram_paged_attention_q8_workspace_bytes) fn_bytes8 = nullptr;
PyObject *error_class = nullptr;  // EngramError(status, where)

// Thrown with the Python error set.
struct PyFailed {};

[[noreturn]] void fail(PyObject *type, const std::string &text) {
    PyErr_SetString(type, text.c_str());
    throw PyFailed();
}

const at::Tensor *tensor(PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

at::ScalarType type_of(const engram_attn_config *c) { return c->dtype == ENGRAM_BF16 ? at::kBFloat16 : at::kHalf; }

std::string sizes(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

void need_type(const at::Tensor &t, at::ScalarType type, const char *name) {
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, std::string(name) + " must be " + toString(type) + ", got " + toString(t.scalar_type()));
}

// On the call's device (its cache's or first tensor's; CUDA is checked before): pointers are handed on, and
// another device's would fault there.
[[noreturn, gnu::cold, gnu::noinline]] void wrong_device(const at::Tensor &t, at::Device dev, const char *name) {
    fail(PyExc_ValueError, std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
}
void need_device(const at::Tensor &t, at::Device dev, const char *name) {
    if (t.get_device() != dev.index()) wrong_device(t, dev, name);
}

// A contiguous CUDA tensor of the type on the device.
void need(const at::Tensor &t, at::ScalarType type, at::Device dev, const char *name) {
    need_type(t, type, name);
    if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
    if (!t.is_cuda()) fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    need_device(t, dev, name);
}

// A [tokens, heads, head_dim] tensor with contiguous heads.
engram_heads heads(const at::Tensor &t, const engram_attn_config *c, int64_t tokens, int64_t n, at::Device dev, const char *name) {
    need_type(t, type_of(c), name);
    const int64_t want[3] = {tokens, n, c->head_dim};
    if (t.sizes() != at::IntArrayRef(want, 3))
        fail(PyExc_ValueError, std::string(name) + " must be " + sizes({want, 3}) + ", got " + sizes(t.sizes()));
    if ((t.stride(2) != 1 && c->head_dim > 1) || !t.is_cuda())
        fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor with contiguous heads");
    need_device(t, dev, name);
    // the stride of a size of one is never used, and torch may give it any value
    return {t.data_ptr(), tokens > 1 ? t.stride(0) : 0, n > 1 ? t.stride(1) : 0};
}

at::Tensor new_heads(const at::Tensor &like, int64_t tokens, int64_t n, const engram_attn_config *c) {
    return at::empty({tokens, n, c->head_dim}, at::TensorOptions().dtype(type_of(c)).device(like.device()));
}

const void *weight(PyObject *o, const engram_attn_config *c, at::Device dev, const char *name) {
    const at::Tensor *w = tensor(o, name);
    if (!w) return nullptr;
    need(*w, type_of(c), dev, name);
    if (w->numel() != c->head_dim) fail(PyExc_ValueError, std::string(name) + " must have " + std::to_string(c->head_dim) + " values");
    return w->data_ptr();
}

const float *table(PyObject *o, const engram_attn_config *c, at::Device dev, int64_t &rows) {
    const at::Tensor *t = tensor(o, "table");
    rows = 0;
    if (!t) {
        if (c->rope_dim) fail(PyExc_ValueError, "table is needed: rope_dim is not 0");
        return nullptr;
    }
    need(*t, at::kFloat, dev, "table");
    if (t->dim() != 2 || t->size(1) != c->rope_dim)
        fail(PyExc_ValueError, "table must be [positions, " + std::to_string(c->rope_dim) + "]");
    rows = t->size(0);
    return t->data_ptr<float>();
}

template <typename T>
T *address(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PyFailed();
    return static_cast<T *>(p);
}

// One of engram.h's structures as its ctypes object's own memory (never a kept
// address: copies of the object would bring the first one's along).
template <typename T>
const T *structure(PyObject *o, const char *name) {
    Py_buffer view;
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) {
        PyErr_Clear();
        view.buf = nullptr;
        view.len = 0;
    } else {
        PyBuffer_Release(&view);  // the caller's argument keeps the memory
    }
    if (view.len != (Py_ssize_t)sizeof(T)) fail(PyExc_TypeError, std::string(name) + " must be its engram.h structure");
    return static_cast<const T *>(view.buf);
}

// The CUDA device of an index.
at::Device cache_device(PyObject *o) {
    const long i = PyLong_AsLong(o);
    if (i == -1 && PyErr_Occurred()) throw PyFailed();
    return at::Device(at::kCUDA, (c10::DeviceIndex)i);
}

// The device of the call's tensors and its stream (a torch.cuda.Stream, or None
// for the current one on that device), both current while this lives: what is
// allocated here belongs to the stream that uses it.
struct Where {
    c10::cuda::OptionalCUDAStreamGuard guard;
    c10::cuda::CUDAStream stream;

    static c10::cuda::CUDAStream named(PyObject *o, const at::Tensor &t) {
        if (!t.is_cuda()) fail(PyExc_ValueError, "the tensors must be CUDA tensors");
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(t.device().index());
        PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw PyFailed();
        void *p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred()) throw PyFailed();
        return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), t.device().index());
    }
    Where(PyObject *o, const at::Tensor &t) : stream(named(o, t)) {
        if (o != Py_None || c10::cuda::current_device() != t.device().index()) guard.reset_stream(stream);
    }
};

void check(engram_status s, const char *where) {
    if (s == ENGRAM_OK) return;
    PyObject *e = PyObject_CallFunction(error_class, "is", (int)s, where);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    throw PyFailed();
}

// What an output argument gives back: the caller's own tensor, or the new one.
PyObject *give(PyObject *given, const at::Tensor &made) {
    if (given == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, const F &body) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
        return nullptr;
    }
    try {
        return body();
    } catch (const PyFailed &) {
        return nullptr;
    } catch (const std::exception &e) {  // torch's own errors (out of memory)
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (cfg, q, k, positions, table, w_q, w_k, q_out, k_out, stream) -> (q_out, k_out)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const auto *c = structure<engram_attn_config>(a[0], "cfg");
        const at::Tensor *q = tensor(a[1], "q"), *k = tensor(a[2], "k"), *pos = tensor(a[3], "positions");
        const at::Tensor *some = q ? q : k;
        if (!some) fail(PyExc_ValueError, "q or k is needed");
        if (some->dim() != 3) fail(PyExc_ValueError, "q and k must be [tokens, heads, head_dim]");
        const int64_t T = some->size(0);
        const at::Device dev = some->device();
        engram_heads hq, hk, hqo, hko;
        at::Tensor made_q, made_k;
        if (q) hq = heads(*q, c, T, c->n_heads, dev, "q");
        if (k) hk = heads(*k, c, T, c->n_kv_heads, dev, "k");
        const Where where(a[9], *some);
        if (q) {
            if (a[7] == Py_None) made_q = new_heads(*q, T, c->n_heads, c);
            hqo = heads(a[7] == Py_None ? made_q : *tensor(a[7], "q_out"), c, T, c->n_heads, dev, "q_out");
        }
        if (k) {
            if (a[8] == Py_None) made_k = new_heads(*k, T, c->n_kv_heads, c);
            hko = heads(a[8] == Py_None ? made_k : *tensor(a[8], "k_out"), c, T, c->n_kv_heads, dev, "k_out");
        }
        if (pos) {
            need(*pos, at::kInt, dev, "positions");
            if (pos->numel() != T) fail(PyExc_ValueError, "positions must have " + std::to_string(T) + " entries");
        }
        int64_t rows;
        const float *tab = table(a[4], c, dev, rows);
        const void *wq = weight(a[5], c, dev, "w_q"), *wk = weight(a[6], c, dev, "w_k");
        check(fn_qk(c, T, q ? &hq : nullptr, k ? &hk : nullptr, pos ? pos->data_ptr<int32_t>() : nullptr, tab, rows, wq, wk,
                    q ? &hqo : nullptr, k ? &hko : nullptr, where.stream.stream()),
              "engram_qk_norm_rope");
        PyObject *x = q ? give(a[7], made_q) : Py_NewRef(a[7]), *y = k ? give(a[8], made_k) : Py_NewRef(a[8]);
        PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        return r;
    });
}

// (cfg, cache, batch, k, v, table, w_k, q, w_q, q_out, stream, the cache's device) -> q_out or None
template <typename Cache, typename F>
PyObject *append_into(const char *name, const F &fn, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject * {
        const auto *c = structure<engram_attn_config>(a[0], "cfg");
        const auto *cache = structure<Cache>(a[1], "cache");
        const auto *batch = structure<engram_kv_batch>(a[2], "batch");
        const at::Tensor *k = tensor(a[3], "k"), *v = tensor(a[4], "v"), *q = tensor(a[7], "q");
        if (!k || !v) fail(PyExc_ValueError, "k and v are needed");
        const int64_t T = batch->n_query;
        const at::Device dev = cache_device(a[11]);
        const engram_heads hk = heads(*k, c, T, c->n_kv_heads, dev, "k"), hv = heads(*v, c, T, c->n_kv_heads, dev, "v");
        engram_heads hq, ho;
        at::Tensor made;
        if (q) hq = heads(*q, c, T, c->n_heads, dev, "q");
        const Where where(a[10], *k);
        if (q) {
            if (a[9] == Py_None) made = new_heads(*q, T, c->n_heads, c);
            ho = heads(a[9] == Py_None ? made : *tensor(a[9], "q_out"), c, T, c->n_heads, dev, "q_out");
        }
        int64_t rows;
        const float *tab = table(a[5], c, dev, rows);
        const void *wk = weight(a[6], c, dev, "w_k"), *wq = weight(a[8], c, dev, "w_q");
        check(fn(c, cache, batch, &hk, &hv, wk, tab, rows, q ? &hq : nullptr, wq, q ? &ho : nullptr, where.stream.stream()),
              name);
        return q ? give(a[9], made) : Py_NewRef(Py_None);
    });
}

// (cfg, cache, batch, q, out, lse, workspace, stream, the cache's device) -> out
template <typename Cache, typename F, typename B>
PyObject *attention_over(const char *name, const F &fn, const B &fn_size, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const auto *c = structure<engram_attn_config>(a[0], "cfg");
        const auto *cache = structure<Cache>(a[1], "cache");
        const auto *batch = structure<engram_kv_batch>(a[2], "batch");
        const at::Tensor *q = tensor(a[3], "q"), *lse = tensor(a[5], "lse"), *ws = tensor(a[6], "workspace");
        if (!q) fail(PyExc_ValueError, "q is needed");
        const int64_t T = batch->n_query;
        const at::Device dev = cache_device(a[8]);
        const engram_heads hq = heads(*q, c, T, c->n_heads, dev, "q");
        const Where where(a[7], *q);
        at::Tensor made, made_ws;
        if (a[4] == Py_None) made = new_heads(*q, T, c->n_heads, c);
        const engram_heads ho = heads(a[4] == Py_None ? made : *tensor(a[4], "out"), c, T, c->n_heads, dev, "out");
        if (lse) {
            need(*lse, at::kFloat, dev, "lse");
            const int64_t want[2] = {T, c->n_heads};
            if (lse->sizes() != at::IntArrayRef(want, 2)) fail(PyExc_ValueError, "lse must be " + sizes({want, 2}));
        }
        size_t bytes = 0;
        void *room = nullptr;
        if (ws) {
            need(*ws, at::kByte, dev, "workspace");
            bytes = (size_t)ws->numel();
            room = ws->data_ptr();
        } else if ((bytes = fn_size(c, cache, batch)) > 0) {  // freed on return, to this stream's pool
            made_ws = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(q->device()));
            room = made_ws.data_ptr();
        }
        check(fn(c, cache, batch, &hq, &ho, lse ? lse->data_ptr<float>() : nullptr, room, bytes, where.stream.stream()),
              name);
        return give(a[4], made);
    });
}

PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return append_into<engram_kv_cache>("engram_kv_append", fn_append, a, n);
}
PyObject *kv_append_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return append_into<engram_kv_cache_q8>("engram_kv_append_q8", fn_append8, a, n);
}
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return attention_over<engram_kv_cache>("engram_paged_attention", fn_attend, fn_bytes, a, n);
}
PyObject *paged_attention_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return attention_over<engram_kv_cache_q8>("engram_paged_attention_q8", fn_attend8, fn_bytes8, a, n);
}

int64_t integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        fail(PyExc_TypeError, std::string(name) + " must be an integer");
    }
    return v;
}

// A contiguous tensor of the type and number of values on the device; nullptr for None.
template <typename T>
T *values(PyObject *o, at::ScalarType type, int64_t count, at::Device dev, const char *name) {
    const at::Tensor *t = tensor(o, name);
    if (!t) return nullptr;
    need(*t, type, dev, name);
    if (t->numel() != count) fail(PyExc_ValueError, std::string(name) + " must have " + std::to_string(count) + " values");
    return t->data_ptr<T>();
}

// (new_len, kv_len, block_table, free_pages, n_free, page_size, max_tokens, keep_len, kv_len_out, n_free_out, seq_offsets,
// positions, slots, counts, stream) -> (seq_offsets, kv_len_out, n_free_out, positions, slots, counts)
PyObject *kv_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const at::Tensor *fresh = tensor(a[0], "new_len"), *table = tensor(a[2], "block_table"), *stack = tensor(a[3], "free_pages");
        if (!fresh || !table || !stack) fail(PyExc_ValueError, "new_len, block_table and free_pages are needed");
        const at::Device dev = stack->device();
        engram_kv_plan_args p = {};
        p.n_seqs = fresh->numel();
        p.max_tokens = integer(a[6], "max_tokens");
        const int64_t size = integer(a[5], "page_size");
        if (size < 1 || size > INT32_MAX) fail(PyExc_ValueError, "page_size must be a multiple of 16, at most 65536");
        p.page_size = (int32_t)size;
        if (p.max_tokens < 0 || p.max_tokens > INT32_MAX) fail(PyExc_ValueError, "max_tokens must be from 0 to 2^31 - 1");
        need(*stack, at::kInt, dev, "free_pages");
        p.n_pages = stack->numel();
        p.free_pages = stack->data_ptr<int32_t>();
        p.new_len = values<int32_t>(a[0], at::kInt, p.n_seqs, dev, "new_len");
        p.kv_len = values<int32_t>(a[1], at::kInt, p.n_seqs, dev, "kv_len");
        if (!p.kv_len && p.n_seqs) fail(PyExc_ValueError, "kv_len is needed");
        p.keep_len = values<int32_t>(a[7], at::kInt, p.n_seqs, dev, "keep_len");
        p.n_free = values<int32_t>(a[4], at::kInt, 1, dev, "n_free");
        if (!p.n_free) fail(PyExc_ValueError, "n_free is needed");
        need_type(*table, at::kInt, "block_table");
        if (!table->is_cuda() || table->dim() != 2 || table->size(0) != p.n_seqs)
            fail(PyExc_ValueError, "block_table must be a CUDA tensor [" + std::to_string(p.n_seqs) + ", pages]");
        need_device(*table, dev, "block_table");
        p.table_width = table->size(1);
        if (p.n_seqs && ((p.table_width > 1 && table->stride(1) != 1) || (p.n_seqs > 1 && table->stride(0) < p.table_width)))
            fail(PyExc_ValueError, "block_table must have contiguous rows");
        p.table_stride = p.n_seqs > 1 ? table->stride(0) : p.table_width;
        p.block_table = table->data_ptr<int32_t>();
        const Where where(a[14], *stack);
        // what is not given is made: offsets, lengths, free pages, positions, slots, counts
        static const char *const names[6] = {"seq_offsets", "kv_len_out", "n_free_out", "positions", "slots", "counts"};
        const int from[6] = {10, 8, 9, 11, 12, 13};
        const int64_t counts[6] = {p.n_seqs + 1, p.n_seqs, 1, p.max_tokens, p.max_tokens, 4};
        // one allocation for all of them, a 16-byte boundary for each (six would cost the host more than the plan the GPU)
        int64_t at[6], bytes = 0;
        bool makes = false;
        for (int i = 0; i < 6; ++i) {
            at[i] = bytes;
            if (a[from[i]] != Py_None) continue;
            bytes += (counts[i] * (i == 0 || i == 4 ? 8 : 4) + 15) / 16 * 16;
            makes = true;
        }
        at::Tensor made[6];
        void *data[6];
        c10::Storage storage;
        if (makes) {  // also of no bytes: an output without values has a storage too
            c10::Allocator *const pool = c10::cuda::CUDACachingAllocator::get();
            storage = c10::Storage(c10::Storage::use_byte_size_t(), bytes, pool->allocate(bytes), pool, /*resizable=*/false);
        }
        for (int i = 0; i < 6; ++i) {
            const bool wide = i == 0 || i == 4;
            if (a[from[i]] == Py_None) {
                made[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                                   c10::scalarTypeToTypeMeta(wide ? at::kLong : at::kInt));
                c10::TensorImpl *const impl = made[i].unsafeGetTensorImpl();
                impl->set_sizes_contiguous(c10::IntArrayRef(&counts[i], 1));
                impl->set_storage_offset(at[i] / (wide ? 8 : 4));
                data[i] = static_cast<char *>(storage.mutable_data()) + at[i];
            } else {
                data[i] = wide ? (void *)values<int64_t>(a[from[i]], at::kLong, counts[i], dev, names[i])
                               : (void *)values<int32_t>(a[from[i]], at::kInt, counts[i], dev, names[i]);
            }
        }
        p.seq_offsets = static_cast<int64_t *>(data[0]);
        p.kv_len_out = static_cast<int32_t *>(data[1]);
        p.n_free_out = static_cast<int32_t *>(data[2]);
        p.positions = static_cast<int32_t *>(data[3]);
        p.slots = static_cast<int64_t *>(data[4]);
        p.counts = static_cast<int32_t *>(data[5]);
        check(fn_plan(&p, where.stream.stream()), "engram_kv_plan");
        PyObject *r = PyTuple_New(6);
        if (!r) throw PyFailed();
        for (int i = 0; i < 6; ++i) {
            PyObject *x = give(a[from[i]], made[i]);
            if (!x) {
                Py_DECREF(r);
                return nullptr;
            }
            PyTuple_SET_ITEM(r, i, x);
        }
        return r;
    });
}

// (EngramError, addresses of the entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        Py_XSETREF(error_class, Py_NewRef(a[0]));
        fn_qk = reinterpret_cast<decltype(fn_qk)>(address<void>(a[1]));
        fn_append = reinterpret_cast<decltype(fn_append)>(address<void>(a[2]));
        fn_attend = reinterpret_cast<decltype(fn_attend)>(address<void>(a[3]));
        fn_bytes = reinterpret_cast<decltype(fn_bytes)>(address<void>(a[4]));
        fn_plan = reinterpret_cast<decltype(fn_plan)>(address<void>(a[5]));
        fn_append8 = reinterpret_cast<decltype(fn_append8)>(address<void>(a[6]));
        fn_attend8 = reinterpret_cast<decltype(fn_attend8)>(address<void>(a[7]));
        fn_bytes8 = reinterpret_cast<decltype(fn_bytes8)>(address<void>(a[8]));
        return Py_NewRef(Py_None);
    });
}

#define STEP_CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {STEP_CALL(bind), STEP_CALL(qk_norm_rope), STEP_CALL(kv_append), STEP_CALL(paged_attention),
                         STEP_CALL(kv_plan), STEP_CALL(kv_append_q8), STEP_CALL(paged_attention_q8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step(void) { return PyModule_Create(&module); }
