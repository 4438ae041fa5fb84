// Argument marshalling of the calls of the paged cache, of drafted trees and of
// several adapters per token, compiled: what __init__.py does for the SGMV
// calls in Python with ctypes. These calls run once per
// layer on operands of a few KB (a decode step's kernels take 3 to 4 us), and
// their dozen tensor arguments cost 6 us to check and convert in Python,
// under 1 us here. Tensors are checked for placement (one device, which the
// call is made on), dtype, shape and layout; everything else is left to the C
// functions, whose status is returned.
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <type_traits>

#include "sgmv.h"

namespace {

// An argument error: the Python exception is set.
struct Refused {};

// Python's other threads run while this lives: a launch waits where the GPU's queue is full.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

[[noreturn]] void refuse(PyObject *type, const char *name, const char *what) {
    PyErr_Format(type, "%s %s", name, what);
    throw Refused{};
}

// A call's tensors, all on the device of the first one asked for.
struct Operands {
    int device = -1;

    const at::Tensor &tensor(PyObject *o, const char *name) {
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, "must be a torch.Tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(PyExc_ValueError, name, "must be on a GPU device");
        if (device < 0) device = t.get_device();
        if (t.get_device() != device) refuse(PyExc_ValueError, name, "must be on the other operands' device");
        return t;
    }

    int32_t *ints(PyObject *o, const char *name, int64_t n) {
        const at::Tensor &t = tensor(o, name);
        if (t.scalar_type() != at::kInt || !t.is_contiguous()) refuse(PyExc_ValueError, name, "must be a contiguous int32 tensor");
        if (n >= 0 && t.numel() != n) {
            PyErr_Format(PyExc_ValueError, "%s must hold %lld entries, got %lld", name, (long long)n, (long long)t.numel());
            throw Refused{};
        }
        return static_cast<int32_t *>(t.data_ptr());
    }

    // To be the current device while the call is made: what its launch goes to where the stream is a default one.
    c10::DeviceGuard guard() const { return c10::DeviceGuard(at::Device(at::kCUDA, (c10::DeviceIndex)device)); }
};

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

// A size as the C functions take it: one that 32 bits do not hold becomes -1, which they refuse.
int32_t size32(int64_t v) { return v < 0 || v > INT32_MAX ? -1 : (int32_t)v; }

int32_t dtype_code(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return SGMV_BF16;
    if (t.scalar_type() == at::kFloat) return SGMV_F32;
    refuse(PyExc_TypeError, "unsupported dtype:", "use float32 or bfloat16");
}

struct Rows {
    void *p;
    int64_t stride;
};

// Rows of heads [T, heads, head_dim]: heads packed within a row, rows any distance apart.
Rows rows3(const at::Tensor &t, const char *name, at::ScalarType dtype, int64_t rows, int64_t heads, int64_t width) {
    if (t.scalar_type() != dtype) refuse(PyExc_TypeError, name, "must have the dtype of the other operands");
    if (t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != width) {
        PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld)", name, (long long)rows, (long long)heads,
                     (long long)width);
        throw Refused{};
    }
    if ((t.stride(2) != 1 && width > 1) || (t.stride(1) != width && heads > 1))
        refuse(PyExc_ValueError, name, ": the heads of a row must be packed");
    return {t.data_ptr(), rows > 1 ? t.stride(0) : heads * width};
}

struct Cache {
    void *K, *V;
    int64_t pages, heads, page, width;
};

Cache cache(Operands &x, PyObject *k, PyObject *v, at::ScalarType dtype) {
    const at::Tensor &K = x.tensor(k, "K_cache"), &V = x.tensor(v, "V_cache");
    if (K.scalar_type() != dtype || V.scalar_type() != dtype)
        refuse(PyExc_TypeError, "K_cache and V_cache", "must have the dtype of the other operands");
    if (K.dim() != 4 || !K.sizes().equals(V.sizes()) || !K.is_contiguous() || !V.is_contiguous())
        refuse(PyExc_ValueError, "K_cache and V_cache",
               "must be contiguous [pages, kv_heads, page_size, head_dim] tensors of one shape");
    return {K.data_ptr(), V.data_ptr(), K.size(0), K.size(1), K.size(2), K.size(3)};
}

const at::Tensor &table2(Operands &x, PyObject *o, int64_t requests) {
    const at::Tensor &t = x.tensor(o, "block_table");
    if (t.dim() != 2 || t.size(0) != requests) refuse(PyExc_ValueError, "block_table", "must have one row per request");
    return t;
}

template <typename F>
PyObject *call(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (seq_len, new_len, block_table, page_size, free_pages, pool_in, pool_out, q_start, kv_len, position, slot, stream)
PyObject *kv_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 12, [&] {
        Operands x;
        const int64_t B = x.tensor(a[0], "seq_len").numel(), T = x.tensor(a[10], "slot").numel();
        const at::Tensor &table = table2(x, a[2], B);
        const int64_t pages = x.tensor(a[4], "free_pages").numel();
        const int32_t *seq_len = x.ints(a[0], "seq_len", B), *new_len = x.ints(a[1], "new_len", B);
        int32_t *entries = x.ints(a[2], "block_table", -1), *ring = x.ints(a[4], "free_pages", pages);
        const int32_t *pool_in = x.ints(a[5], "pool_in", 4);
        int32_t *pool_out = x.ints(a[6], "pool_out", 4), *q_start = x.ints(a[7], "q_start", B + 1);
        int32_t *kv_len = x.ints(a[8], "kv_len", B), *position = x.ints(a[9], "position", T), *slot = x.ints(a[10], "slot", T);
        const int32_t width = size32(table.size(1)), page = size32(integer(a[3]));
        void *stream = reinterpret_cast<void *>(integer(a[11]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_kv_tables(seq_len, new_len, size32(B), entries, width, page, ring, size32(pages), pool_in, pool_out, q_start,
                              kv_len, position, slot, size32(T), stream);
    });
}

// (q_out, q, k, v, K_cache, V_cache, position, slot, table, interleaved, stream)
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 11, [&] {
        Operands x;
        const bool has_q = a[1] != Py_None, has_k = a[2] != Py_None;
        if (!has_q && !has_k) refuse(PyExc_ValueError, "sgmv_rope_append", "needs q or k");
        const at::Tensor &like = has_q ? x.tensor(a[1], "q") : x.tensor(a[2], "k");
        const int64_t T = x.tensor(a[6], "position").numel();
        if (like.dim() != 3 || like.size(0) != T) refuse(PyExc_ValueError, "q and k", "must have one row per token");
        const at::ScalarType dtype = like.scalar_type();
        const int64_t D = like.size(2);
        Rows q{}, q_out{}, k{}, v{};
        Cache c{nullptr, nullptr, 0, 0, 16, D};
        int64_t q_heads = 0;
        const int32_t *slot = nullptr;
        if (has_q) {
            q_heads = like.size(1);
            q = rows3(like, "q", dtype, T, q_heads, D);
            q_out = rows3(x.tensor(a[0], "q_out"), "q_out", dtype, T, q_heads, D);
        }
        if (has_k) {
            c = cache(x, a[4], a[5], dtype);
            if (c.width != D) refuse(PyExc_ValueError, "q and the cache", "must agree in head_dim");
            k = rows3(x.tensor(a[2], "k"), "k", dtype, T, c.heads, D);
            v = rows3(x.tensor(a[3], "v"), "v", dtype, T, c.heads, D);
            slot = x.ints(a[7], "slot", T);
        }
        const float *turn = nullptr;
        int64_t max_position = INT32_MAX, rot_dim = 0;
        if (a[8] != Py_None) {
            const at::Tensor &t = x.tensor(a[8], "table");
            if (t.scalar_type() != at::kFloat || t.dim() != 3 || t.size(2) != 2 || !t.is_contiguous())
                refuse(PyExc_ValueError, "table", "must be a contiguous float32 [max_position, rot_dim / 2, 2] tensor");
            turn = static_cast<const float *>(t.data_ptr());
            max_position = t.size(0);
            rot_dim = 2 * t.size(1);
        }
        const int32_t *position = x.ints(a[6], "position", T);
        const int32_t interleaved = truth(a[9]), code = dtype_code(like);
        void *stream = reinterpret_cast<void *>(integer(a[10]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_rope_append(q_out.p, q_out.stride, q.p, q.stride, size32(q_heads), k.p, k.stride, v.p, v.stride, c.K,
                                c.V, size32(c.pages), size32(c.heads), size32(c.page), size32(D), position, slot, size32(T),
                                turn, size32(max_position), size32(rot_dim), interleaved, code, stream);
    });
}

// A step's masks [T, words].
struct Mask {
    uint32_t *p;
    int64_t words;
};
Mask mask2(Operands &x, PyObject *o, int64_t T) {
    const at::Tensor &t = x.tensor(o, "mask");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != T || !t.is_contiguous())
        refuse(PyExc_ValueError, "mask", "must be a contiguous int32 [T, words] tensor");
    return {static_cast<uint32_t *>(t.data_ptr()), t.size(1)};
}

// (out, q, K_cache, V_cache, block_table, q_start, kv_len, scale, max_q_len, window, sinks, lse, workspace, stream), and
// for a tree the mask after them
template <bool kTree>
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, kTree ? 15 : 14, [&] {
        Operands x;
        const at::Tensor &q = x.tensor(a[1], "q");
        if (q.dim() != 3) refuse(PyExc_ValueError, "q", "must have 3 dimensions");
        const at::ScalarType dtype = q.scalar_type();
        const int64_t T = q.size(0), heads = q.size(1), D = q.size(2);
        const Rows qr = rows3(q, "q", dtype, T, heads, D), outr = rows3(x.tensor(a[0], "out"), "out", dtype, T, heads, D);
        const Cache c = cache(x, a[2], a[3], dtype);
        if (c.width != D) refuse(PyExc_ValueError, "q and the cache", "must agree in head_dim");
        const int64_t B = x.tensor(a[6], "kv_len").numel();
        const at::Tensor &table = table2(x, a[4], B);
        float *lse = nullptr;
        if (a[11] != Py_None) {
            const at::Tensor &t = x.tensor(a[11], "lse");
            if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != T || t.size(1) != heads || !t.is_contiguous())
                refuse(PyExc_ValueError, "lse", "must be a contiguous float32 [T, q_heads] tensor");
            lse = static_cast<float *>(t.data_ptr());
        }
        const at::Tensor &ws = x.tensor(a[12], "workspace");
        if (!ws.is_contiguous()) refuse(PyExc_ValueError, "workspace", "must be contiguous");
        const double scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
        const int32_t *entries = x.ints(a[4], "block_table", -1), *q_start = x.ints(a[5], "q_start", B + 1);
        const int32_t *kv_len = x.ints(a[6], "kv_len", B);
        const int32_t max_q_len = size32(integer(a[8])), window = size32(integer(a[9])), sinks = size32(integer(a[10]));
        const int32_t width = size32(table.size(1)), code = dtype_code(q);
        void *workspace = ws.data_ptr(), *stream = reinterpret_cast<void *>(integer(a[13]));
        const size_t bytes = ws.nbytes();
        const Mask mask = kTree ? mask2(x, a[14], T) : Mask{nullptr, 0};
        const auto on = x.guard();
        const Unlocked others;
        if (kTree)
            return sgmv_tree_attention(outr.p, outr.stride, lse, qr.p, qr.stride, size32(heads), c.K, c.V, size32(c.pages),
                                       size32(c.heads), size32(c.page), size32(D), entries, width, q_start, kv_len, mask.p,
                                       size32(mask.words), size32(B), size32(T), max_q_len, (float)scale, window, sinks, code,
                                       workspace, bytes, stream);
        return sgmv_paged_attention(outr.p, outr.stride, lse, qr.p, qr.stride, size32(heads), c.K, c.V, size32(c.pages),
                                    size32(c.heads), size32(c.page), size32(D), entries, width, q_start, kv_len, size32(B),
                                    size32(T), max_q_len, (float)scale, window, sinks, code, workspace, bytes, stream);
    });
}

// (parent, q_start, kv_len, position, mask, stream)
PyObject *tree_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 6, [&] {
        Operands x;
        const int64_t T = x.tensor(a[0], "parent").numel(), B = x.tensor(a[2], "kv_len").numel();
        const int32_t *parent = x.ints(a[0], "parent", T), *q_start = x.ints(a[1], "q_start", B + 1);
        const int32_t *kv_len = x.ints(a[2], "kv_len", B);
        int32_t *position = x.ints(a[3], "position", T);
        const Mask mask = mask2(x, a[4], T);
        void *stream = reinterpret_cast<void *>(integer(a[5]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_tree_tables(parent, q_start, kv_len, size32(B), position, mask.p, size32(mask.words), size32(T), stream);
    });
}

// (parent, token, target, slot, q_start, kv_len, page_size, block_table, free_pages, pool_in, pool_out, path, accepted,
// next_token, kept_len, stream)
PyObject *tree_accept(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 16, [&] {
        Operands x;
        const int64_t T = x.tensor(a[0], "parent").numel(), B = x.tensor(a[5], "kv_len").numel();
        const at::Tensor &table = table2(x, a[7], B);
        const int64_t pages = x.tensor(a[8], "free_pages").numel();
        const int32_t *parent = x.ints(a[0], "parent", T), *token = x.ints(a[1], "token", T);
        const int32_t *target = x.ints(a[2], "target", T), *slot = x.ints(a[3], "slot", T);
        const int32_t *q_start = x.ints(a[4], "q_start", B + 1), *kv_len = x.ints(a[5], "kv_len", B);
        const int32_t *entries = x.ints(a[7], "block_table", -1), *pool_in = x.ints(a[9], "pool_in", 4);
        int32_t *ring = x.ints(a[8], "free_pages", pages), *pool_out = x.ints(a[10], "pool_out", 4);
        int32_t *path = x.ints(a[11], "path", T), *accepted = x.ints(a[12], "accepted", B);
        int32_t *next_token = x.ints(a[13], "next_token", B), *kept_len = x.ints(a[14], "kept_len", B);
        const int32_t width = size32(table.size(1)), page = size32(integer(a[6]));
        void *stream = reinterpret_cast<void *>(integer(a[15]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_tree_accept(parent, token, target, slot, q_start, kv_len, size32(B), page, entries, width, ring,
                                size32(pages), pool_in, pool_out, path, accepted, next_token, kept_len, size32(T), stream);
    });
}

// (K_cache, V_cache, slot, q_start, path, stream): a layer's caches, or all of a cache's layers in one tensor
PyObject *kv_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 6, [&] {
        Operands x;
        const at::Tensor &K = x.tensor(a[0], "K_cache"), &V = x.tensor(a[1], "V_cache");
        const int64_t one = K.dim() == 5;
        if (K.scalar_type() != V.scalar_type()) refuse(PyExc_TypeError, "K_cache and V_cache", "must have one dtype");
        if ((K.dim() != 4 && !one) || !K.sizes().equals(V.sizes()) || !K.is_contiguous() || !V.is_contiguous())
            refuse(PyExc_ValueError, "K_cache and V_cache",
                   "must be contiguous [pages, kv_heads, page_size, head_dim] tensors of one shape, or have a dimension of "
                   "layers before these");
        const int64_t layers = one ? K.size(0) : 1, T = x.tensor(a[2], "slot").numel(), B = x.tensor(a[3], "q_start").numel() - 1;
        if (B < 0) refuse(PyExc_ValueError, "q_start", "must have one entry more than there are requests");
        const int32_t *slot = x.ints(a[2], "slot", T), *q_start = x.ints(a[3], "q_start", B + 1), *path = x.ints(a[4], "path", T);
        const int32_t code = dtype_code(K);
        void *k = K.data_ptr(), *v = V.data_ptr(), *stream = reinterpret_cast<void *>(integer(a[5]));
        const int64_t pages = K.size(one), heads = K.size(one + 1), page = K.size(one + 2), width = K.size(one + 3);
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_kv_commit(k, v, size32(layers), pages * heads * page * width, size32(pages), size32(heads), size32(page),
                              size32(width), slot, q_start, path, size32(B), size32(T), code, stream);
    });
}

// Rows [rows, width], packed within a row, rows any distance apart.
Rows rows2(const at::Tensor &t, const char *name, at::ScalarType dtype, int64_t rows, int64_t width) {
    if (t.scalar_type() != dtype) refuse(PyExc_TypeError, name, "must have the dtype of the other operands");
    if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || t.size(1) != width) {
        if (rows >= 0)
            PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld)", name, (long long)rows, (long long)width);
        else
            PyErr_Format(PyExc_ValueError, "%s must have rows of %lld", name, (long long)width);
        throw Refused{};
    }
    if (t.stride(1) != 1 && width > 1) refuse(PyExc_ValueError, name, ": a row's elements must be packed");
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : width};
}

// Choices, places or weights [T, choices].
template <typename E>
E *choices2(Operands &x, PyObject *o, const char *name, int64_t T, int64_t choices) {
    const at::Tensor &t = x.tensor(o, name);
    if (t.scalar_type() != (std::is_same<E, float>::value ? at::kFloat : at::kInt) || t.dim() != 2 || !t.is_contiguous() ||
        (T >= 0 && (t.size(0) != T || t.size(1) != choices)))
        refuse(PyExc_ValueError, name, std::is_same<E, float>::value ? "must be a contiguous float32 [T, choices] tensor"
                                                                      : "must be a contiguous int32 [T, choices] tensor");
    return static_cast<E *>(t.data_ptr());
}

// (choice, num_adapters, seg_start, seg_adapter, order, place, workspace or None, stream)
PyObject *sort_tokens(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 8, [&] {
        Operands x;
        const int32_t *choice = choices2<int32_t>(x, a[0], "choice", -1, 0);
        const at::Tensor &c = x.tensor(a[0], "choice");
        const int64_t T = c.size(0), choices = c.size(1), S = x.tensor(a[3], "seg_adapter").numel();
        int32_t *seg_start = x.ints(a[2], "seg_start", S + 1), *seg_adapter = x.ints(a[3], "seg_adapter", S);
        int32_t *order = x.ints(a[4], "order", T * choices), *place = choices2<int32_t>(x, a[5], "place", T, choices);
        const int32_t adapters = size32(integer(a[1]));
        void *ws = nullptr;
        size_t bytes = 0;
        if (a[6] != Py_None) {
            const at::Tensor &w = x.tensor(a[6], "workspace");
            if (!w.is_contiguous()) refuse(PyExc_ValueError, "workspace", "must be contiguous");
            ws = w.data_ptr();
            bytes = w.nbytes();
        }
        void *stream = reinterpret_cast<void *>(integer(a[7]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_sort_tokens(choice, size32(T), size32(choices), adapters, seg_start, seg_adapter, size32(S), order, place,
                                ws, bytes, stream);
    });
}

// (Xs, X, place, stream)
PyObject *spread_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 4, [&] {
        Operands x;
        const at::Tensor &X = x.tensor(a[1], "X"), &Xs = x.tensor(a[0], "Xs"), &p = x.tensor(a[2], "place");
        if (X.dim() != 2 || p.dim() != 2) refuse(PyExc_ValueError, "X and place", "must have 2 dimensions");
        const int64_t T = X.size(0), d = X.size(1), choices = p.size(1);
        const Rows in = rows2(X, "X", X.scalar_type(), T, d), out = rows2(Xs, "Xs", X.scalar_type(), -1, d);
        const int32_t *place = choices2<int32_t>(x, a[2], "place", T, choices);
        const int32_t code = dtype_code(X);
        const int64_t rows = Xs.size(0);
        void *stream = reinterpret_cast<void *>(integer(a[3]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_spread_rows(out.p, out.stride, size32(rows), in.p, in.stride, place, size32(T), size32(choices), size32(d),
                                code, stream);
    });
}

// (Y, Ys, place, weight or None, base or None, stream)
PyObject *combine_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 6, [&] {
        Operands x;
        const at::Tensor &Y = x.tensor(a[0], "Y"), &Ys = x.tensor(a[1], "Ys"), &p = x.tensor(a[2], "place");
        if (Y.dim() != 2 || p.dim() != 2) refuse(PyExc_ValueError, "Y and place", "must have 2 dimensions");
        const int64_t T = Y.size(0), d = Y.size(1), choices = p.size(1);
        const Rows out = rows2(Y, "Y", Y.scalar_type(), T, d), in = rows2(Ys, "Ys", Y.scalar_type(), -1, d);
        const int32_t *place = choices2<int32_t>(x, a[2], "place", T, choices);
        const float *weight = a[3] != Py_None ? choices2<float>(x, a[3], "weight", T, choices) : nullptr;
        const Rows base = a[4] != Py_None ? rows2(x.tensor(a[4], "base"), "base", Y.scalar_type(), T, d) : Rows{nullptr, 0};
        const int32_t code = dtype_code(Y);
        const int64_t rows = Ys.size(0);
        void *stream = reinterpret_cast<void *>(integer(a[5]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_combine_rows(out.p, out.stride, base.p, base.stride, in.p, in.stride, size32(rows), place, weight, size32(T),
                                 size32(choices), size32(d), code, stream);
    });
}

// (dYs or None, dweight or None, dY, Ys or None, place, weight or None, stream)
PyObject *combine_rows_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call(n, 7, [&] {
        Operands x;
        const at::Tensor &dY = x.tensor(a[2], "dY"), &p = x.tensor(a[4], "place");
        if (dY.dim() != 2 || p.dim() != 2) refuse(PyExc_ValueError, "dY and place", "must have 2 dimensions");
        const bool rows_out = a[0] != Py_None, weight_out = a[1] != Py_None;
        if (!rows_out && !weight_out) refuse(PyExc_ValueError, "sgmv_combine_rows_grad", "needs dYs or dweight");
        if (weight_out && a[3] == Py_None) refuse(PyExc_ValueError, "Ys", "is needed for dweight");
        const int64_t T = dY.size(0), d = dY.size(1), choices = p.size(1);
        const at::ScalarType dtype = dY.scalar_type();
        const Rows in = rows2(dY, "dY", dtype, T, d);
        int64_t rows = -1;
        Rows dYs{nullptr, 0}, Ys{nullptr, 0};
        if (rows_out) {
            dYs = rows2(x.tensor(a[0], "dYs"), "dYs", dtype, -1, d);
            rows = x.tensor(a[0], "dYs").size(0);
        }
        if (weight_out) {
            Ys = rows2(x.tensor(a[3], "Ys"), "Ys", dtype, rows, d);
            rows = x.tensor(a[3], "Ys").size(0);
        }
        float *dweight = weight_out ? choices2<float>(x, a[1], "dweight", T, choices) : nullptr;
        const int32_t *place = choices2<int32_t>(x, a[4], "place", T, choices);
        const float *weight = a[5] != Py_None ? choices2<float>(x, a[5], "weight", T, choices) : nullptr;
        const int32_t code = dtype_code(dY);
        void *stream = reinterpret_cast<void *>(integer(a[6]));
        const auto on = x.guard();
        const Unlocked others;
        return sgmv_combine_rows_grad(dYs.p, dYs.stride, dweight, in.p, in.stride, Ys.p, Ys.stride, size32(rows), place, weight,
                                      size32(T), size32(choices), size32(d), code, stream);
    });
}

PyMethodDef methods[] = {
    {"kv_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_tables)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention<false>)), METH_FASTCALL, nullptr},
    {"tree_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention<true>)), METH_FASTCALL, nullptr},
    {"tree_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_tables)), METH_FASTCALL, nullptr},
    {"tree_accept", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree_accept)), METH_FASTCALL, nullptr},
    {"kv_commit", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_commit)), METH_FASTCALL, nullptr},
    {"sort_tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sort_tokens)), METH_FASTCALL, nullptr},
    {"spread_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(spread_rows)), METH_FASTCALL, nullptr},
    {"combine_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(combine_rows)), METH_FASTCALL, nullptr},
    {"combine_rows_grad", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(combine_rows_grad)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_binding(void) { return PyModule_Create(&module); }
