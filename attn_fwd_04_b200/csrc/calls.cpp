// calls.cpp -- the binding's short way into libfa.so for the calls of a decode
// step: tables, norms with the rotation, appends, decode over the 8-bit cache.
//
// A step's kernels run for a few microseconds each, and a Python wrapper that
// looks at a dozen tensors takes longer than that (norm and rotation of 64
// tokens: 15 us through fa.py alone, 3 us on the GPU).  Each function here
// takes its wrapper's arguments in order, checks them with the tensors' own
// accessors, makes the outputs and scratch, and calls the same C entry point.
// It answers with the outputs; with a status where the entry point refused;
// or with None where anything is not the ordinary case (a type, shape, stride
// or device that does not fit, another GPU than the current one, a stream
// given by hand): the wrapper in fa.py then does the same work itself, and
// says what is wrong.  Nothing is computed here.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "fa.h"

namespace {

using at::ScalarType;
using at::Tensor;

// The entry points, looked up by fa.py in the library that it loaded.
struct Entry {
    decltype(&fa_rope_table) rope_table;
    decltype(&fa_qk_norm_rope) norm;
    decltype(&fa_qk_norm_rope_bwd) norm_bwd;
    decltype(&fa_qk_norm_rope_bwd_workspace) norm_bwd_bytes;
    decltype(&fa_append_paged_rope) append;
    decltype(&fa_append_paged_fp8) append_fp8;
    decltype(&fa_decode_paged_fp8) decode;
    decltype(&fa_decode_paged_fp8_workspace) decode_bytes;
} g_fa;
bool g_bound = false;

// Thrown where a call is not the ordinary case; never leaves this file.
struct Other {};

void need(bool ok) {
    if (!ok) throw Other{};
}

int fit(int64_t v) {
    need(v >= 0 && v <= INT_MAX);
    return static_cast<int>(v);
}

// A tensor argument: torch.Tensor or Parameter itself, on the current GPU.
const Tensor& tensor(PyObject* o) {
    need(THPVariable_CheckExact(o));
    const Tensor& t = THPVariable_Unpack(o);
    need(t.is_cuda() && t.layout() == c10::kStrided &&
         t.get_device() == c10::cuda::current_device());
    return t;
}

bool shaped(const Tensor& t, ScalarType type, at::IntArrayRef sizes) {
    return t.scalar_type() == type && t.sizes() == sizes && t.is_contiguous();
}

// None, or a tensor of this type and shape.
const void* optional(PyObject* o, ScalarType type, at::IntArrayRef sizes) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o);
    need(shaped(t, type, sizes));
    return t.const_data_ptr();
}

// [tokens, heads, d] bf16, [heads, d] contiguous: the stride between tokens.
int token_stride(const Tensor& t) {
    need(t.scalar_type() == ScalarType::BFloat16 && t.dim() == 3);
    const int64_t row = t.size(1) * t.size(2), st = t.stride(0);
    // (torch gives a dimension of one any stride)
    need(t.stride(2) == 1 && (t.stride(1) == t.size(2) || t.size(1) == 1) && st >= row &&
         st % 8 == 0);
    return fit(st);
}

Tensor bf16_like(const Tensor& t) {
    return at::empty(t.sizes(), t.options().memory_format(at::MemoryFormat::Contiguous));
}

fa_stream_t stream() {
    return reinterpret_cast<fa_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
}

double number(PyObject* o) {
    need(PyFloat_CheckExact(o) || PyLong_CheckExact(o));
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Other{};
    }
    return v;
}

int whole(PyObject* o) {
    need(PyLong_CheckExact(o));
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Other{};
    }
    return fit(v);
}

bool truth(PyObject* o) {
    need(PyBool_Check(o));
    return o == Py_True;
}

// Norm weights [d] of one type, and the rotation's tables, as every call has them.
struct Turn {
    const void *qw = nullptr, *kw = nullptr;
    int type = FA_WEIGHT_BF16;
    const float *cos = nullptr, *sin = nullptr;
    int max_pos = 0, rot = 0;

    Turn(PyObject* q_weight, PyObject* k_weight, PyObject* c, PyObject* s, int64_t d) {
        PyObject* any = q_weight != Py_None ? q_weight : k_weight;
        if (any != Py_None) {
            const ScalarType st =
                tensor(any).scalar_type() == ScalarType::Float ? ScalarType::Float
                                                                : ScalarType::BFloat16;
            type = st == ScalarType::Float ? FA_WEIGHT_FP32 : FA_WEIGHT_BF16;
            qw = optional(q_weight, st, {d});
            kw = optional(k_weight, st, {d});
        }
        need((c == Py_None) == (s == Py_None));
        if (c == Py_None) return;
        const Tensor& t = tensor(c);
        need(t.dim() == 2 && shaped(t, ScalarType::Float, t.sizes()));
        cos = t.const_data_ptr<float>();
        sin = static_cast<const float*>(optional(s, ScalarType::Float, t.sizes()));
        max_pos = fit(t.size(0));
        rot = fit(2 * t.size(1));
    }
};

// Queries and keys of the norms: packed or heads first, and their positions.
struct Rows {
    const Tensor &q, &k;
    int layout, B, N, H, Hk, d, sq = 0, sk = 0;
    const int32_t* positions;

    Rows(PyObject* qo, PyObject* ko, PyObject* pos) : q(tensor(qo)), k(tensor(ko)) {
        layout = q.dim() == 4 ? FA_LAYOUT_HEADS : FA_LAYOUT_PACKED;
        if (layout == FA_LAYOUT_HEADS) {
            need(k.dim() == 4 && shaped(q, ScalarType::BFloat16, q.sizes()) &&
                 shaped(k, ScalarType::BFloat16, {q.size(0), k.size(1), q.size(2), q.size(3)}));
            B = fit(q.size(0));
            N = fit(q.size(2));
            H = fit(q.size(1));
            Hk = fit(k.size(1));
            positions = static_cast<const int32_t*>(
                optional(pos, ScalarType::Int, {q.size(0), q.size(2)}));
        } else {
            sq = token_stride(q);
            sk = token_stride(k);
            need(k.size(0) == q.size(0) && k.size(2) == q.size(2));
            B = 1;
            N = fit(q.size(0));
            H = fit(q.size(1));
            Hk = fit(k.size(1));
            positions =
                static_cast<const int32_t*>(optional(pos, ScalarType::Int, {q.size(0)}));
        }
        d = fit(q.size(q.dim() - 1));
        need(B > 0 && N > 0);
    }

    // An output or gradient like `x`: the one given, or (None) a new one.
    Tensor like(PyObject* o, const Tensor& x, int& st) const {
        st = 0;
        if (o == Py_None) return bf16_like(x);
        const Tensor& t = tensor(o);
        need(t.sizes() == x.sizes());
        if (layout == FA_LAYOUT_HEADS) need(shaped(t, ScalarType::BFloat16, x.sizes()));
        else st = token_stride(t);
        return t;
    }
};

// A call with the library's workspace of its stream; where that is refused, as it
// is while the stream is captured, once more with scratch of the graph's own.
template <class Run, class Bytes>
int with_scratch(const Tensor& like, Run run, Bytes bytes_of) {
    int rc = run(nullptr, 0);
    if (rc != FA_ERR_UNSUPPORTED) return rc;
    int bytes = 0;
    rc = bytes_of(&bytes);
    if (rc != FA_OK) return rc;
    const Tensor ws = at::empty({bytes}, like.options().dtype(ScalarType::Byte));
    return run(ws.data_ptr(), bytes);
}

PyObject* tuple_of(std::initializer_list<Tensor> ts) {
    PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o;
        if (t.defined()) {
            o = THPVariable_Wrap(t);
        } else {
            Py_INCREF(Py_None);
            o = Py_None;
        }
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

// Runs `f`; what is not the ordinary case, and an exception (no memory, no GPU: all
// before the launch), becomes None, and the long way meets it again.
template <class F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want || !g_bound) Py_RETURN_NONE;
    try {
        return f();
    } catch (...) {
        if (PyErr_Occurred()) return nullptr;
        Py_RETURN_NONE;
    }
}

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out, k_out)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 11, [&]() -> PyObject* {
        const Rows r(a[0], a[1], a[6]);
        const Turn t(a[2], a[3], a[4], a[5], r.d);
        const float eps = static_cast<float>(number(a[7]));
        const bool inter = truth(a[8]);
        int sqo, sko;
        const Tensor qo = r.like(a[9], r.q, sqo), ko = r.like(a[10], r.k, sko);
        const int rc = g_fa.norm(r.q.const_data_ptr(), r.k.const_data_ptr(), qo.data_ptr(),
                                 ko.data_ptr(), t.qw, t.kw, t.type, t.cos, t.sin, t.max_pos,
                                 t.rot, inter, r.positions, r.layout, r.B, r.N, r.H, r.Hk, r.d,
                                 r.sq, r.sk, sqo, sko, eps, stream());
        return rc != FA_OK ? PyLong_FromLong(rc) : tuple_of({qo, ko});
    });
}

// (q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, positions, eps,
//  interleaved, dq, dk, dq_weight, dk_weight)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 15, [&]() -> PyObject* {
        const Rows r(a[0], a[1], a[8]);
        const Turn t(a[4], a[5], a[6], a[7], r.d);
        const float eps = static_cast<float>(number(a[9]));
        const bool inter = truth(a[10]);
        need(a[2] != Py_None && a[3] != Py_None);
        int sgq, sgk, sdq, sdk;
        const Tensor gq = r.like(a[2], r.q, sgq), gk = r.like(a[3], r.k, sgk);
        const Tensor dq = r.like(a[11], r.q, sdq), dk = r.like(a[12], r.k, sdk);
        auto grad = [&](PyObject* o, const void* w) {
            if (!w) {
                need(o == Py_None);
                return Tensor();
            }
            if (o == Py_None) return at::empty({r.d}, r.q.options().dtype(ScalarType::Float));
            const Tensor& g = tensor(o);
            need(shaped(g, ScalarType::Float, {r.d}));
            return g;
        };
        const Tensor dqw = grad(a[13], t.qw), dkw = grad(a[14], t.kw);
        const auto run = [&](void* ws, int bytes) {
            return g_fa.norm_bwd(
                r.q.const_data_ptr(), r.k.const_data_ptr(), gq.const_data_ptr(),
                gk.const_data_ptr(), dq.data_ptr(), dk.data_ptr(),
                dqw.defined() ? dqw.data_ptr<float>() : nullptr,
                dkw.defined() ? dkw.data_ptr<float>() : nullptr, t.qw, t.kw, t.type, t.cos, t.sin,
                t.max_pos, t.rot, inter, r.positions, r.layout, r.B, r.N, r.H, r.Hk, r.d, r.sq,
                r.sk, sgq, sgk, sdq, sdk, eps, ws, bytes, stream());
        };
        const int rc = with_scratch(r.q, run, [&](int* bytes) {
            return g_fa.norm_bwd_bytes(r.B, r.N, r.H, r.Hk, r.d, bytes);
        });
        return rc != FA_OK ? PyLong_FromLong(rc) : tuple_of({dq, dk, dqw, dkw});
    });
}

// A pool [P, heads, page_size, d] of this type, k and v alike.
struct Pool {
    const Tensor &k, &v;
    int P, Hk;
    Pool(PyObject* ko, PyObject* vo, ScalarType type, int page_size, int64_t d)
        : k(tensor(ko)), v(tensor(vo)) {
        need(k.dim() == 4 && k.size(2) == page_size && k.size(3) == d &&
             shaped(k, type, k.sizes()) && shaped(v, type, k.sizes()));
        P = fit(k.size(0));
        Hk = fit(k.size(1));
    }
};

// Scales [P, heads, page_size / block].
struct Scales {
    const Tensor &k, &v;
    int block;
    Scales(PyObject* ko, PyObject* vo, const Pool& pool, int page_size)
        : k(tensor(ko)), v(tensor(vo)) {
        need(k.dim() == 3 && k.size(2) > 0 && page_size % k.size(2) == 0 &&
             shaped(k, ScalarType::Float, {pool.P, pool.Hk, k.size(2)}) &&
             shaped(v, ScalarType::Float, k.sizes()));
        block = page_size / static_cast<int>(k.size(2));
    }
};

// A packed page table [n] or a block table [B, max_pages]; an empty one stands
// in for itself by `other`, which is not read through.
struct Table {
    const int32_t* at;
    int len, max_pages = 0;
    Table(PyObject* o, int B, const int32_t* other) {
        const Tensor& t = tensor(o);
        need((t.dim() == 1 || (t.dim() == 2 && t.size(0) == B)) &&
             shaped(t, ScalarType::Int, t.sizes()));
        if (t.dim() == 2) max_pages = fit(t.size(1));
        len = fit(t.numel());
        at = len ? t.const_data_ptr<int32_t>() : other;
    }
};

// (q_new, k_new, v_new, cu_new, k_pages, v_pages, k_scales, v_scales, page_table,
//  seq_lens, cos, sin, q_weight, k_weight, eps, interleaved, page_size, q_out);
// bf16 pages: k_scales and v_scales are None
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 18, [&]() -> PyObject* {
        const Tensor &k = tensor(a[1]), &v = tensor(a[2]);
        const int sk = token_stride(k), sv = token_stride(v);
        need(v.sizes() == k.sizes());
        const int64_t total = k.size(0), d = k.size(2);
        need(total > 0);
        Tensor qo;
        const void* q = nullptr;
        int H = 0, sq = 0;
        if (a[0] != Py_None) {
            const Tensor& qt = tensor(a[0]);
            sq = token_stride(qt);
            need(qt.size(0) == total && qt.size(2) == d);
            q = qt.const_data_ptr();
            H = fit(qt.size(1));
            if (a[17] == Py_None) {
                qo = bf16_like(qt);
            } else {
                qo = tensor(a[17]);
                need(shaped(qo, ScalarType::BFloat16, qt.sizes()));
            }
        } else {
            need(a[17] == Py_None && a[12] == Py_None);
        }
        const bool eight = a[6] != Py_None;
        const int page_size = whole(a[16]);
        const Pool pool(a[4], a[5], eight ? ScalarType::Float8_e4m3fn : ScalarType::BFloat16,
                        page_size, d);
        need(pool.Hk == k.size(1));
        const Tensor &cu = tensor(a[3]), &lens = tensor(a[9]);
        need(cu.dim() == 1 && shaped(cu, ScalarType::Int, cu.sizes()) && cu.numel() > 1);
        const int B = fit(cu.numel() - 1);
        need(shaped(lens, ScalarType::Int, {B}));
        const int32_t* len_p = lens.const_data_ptr<int32_t>();
        const Table table(a[8], B, len_p);
        const Turn t(a[12], a[13], a[10], a[11], d);
        const float eps = static_cast<float>(number(a[14]));
        const bool inter = truth(a[15]);
        void* out = qo.defined() ? qo.data_ptr() : nullptr;
        int rc;
        if (eight) {
            const Scales s(a[6], a[7], pool, page_size);
            rc = g_fa.append_fp8(q, k.const_data_ptr(), v.const_data_ptr(),
                                 cu.const_data_ptr<int32_t>(), out, pool.k.data_ptr(),
                                 pool.v.data_ptr(), s.k.data_ptr<float>(), s.v.data_ptr<float>(),
                                 s.block, table.at, table.len, table.max_pages, len_p, t.qw, t.kw,
                                 t.type, t.cos, t.sin, t.max_pos, t.rot, inter, B, H, pool.Hk,
                                 fit(total), pool.P, fit(d), page_size, sq, sk, sv, eps, stream());
        } else {
            need(a[7] == Py_None);
            rc = g_fa.append(q, k.const_data_ptr(), v.const_data_ptr(),
                             cu.const_data_ptr<int32_t>(), out, pool.k.data_ptr(),
                             pool.v.data_ptr(), table.at, table.len, table.max_pages, len_p, t.qw,
                             t.kw, t.type, t.cos, t.sin, t.max_pos, t.rot, inter, B, H, pool.Hk,
                             fit(total), pool.P, fit(d), page_size, sq, sk, sv, eps, stream());
        }
        // (the outputs in a tuple: None stands for another case)
        return rc != FA_OK ? PyLong_FromLong(rc) : tuple_of({qo});
    });
}

// (q, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens, page_size,
//  scale, o, lse)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 11, [&]() -> PyObject* {
        const Tensor& q = tensor(a[0]);
        need(q.dim() == 3 && shaped(q, ScalarType::BFloat16, q.sizes()) && q.numel() > 0);
        const int B = fit(q.size(0)), H = fit(q.size(1)), d = fit(q.size(2));
        const int page_size = whole(a[7]);
        const Pool pool(a[1], a[2], ScalarType::Float8_e4m3fn, page_size, d);
        need(pool.Hk > 0 && H % pool.Hk == 0);
        const Scales s(a[3], a[4], pool, page_size);
        const Tensor& lens = tensor(a[6]);
        need(shaped(lens, ScalarType::Int, {B}));
        const int32_t* len_p = lens.const_data_ptr<int32_t>();
        const Table table(a[5], B, len_p);
        const float scale = static_cast<float>(
            a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[8]));
        Tensor o;
        if (a[9] == Py_None) {
            o = bf16_like(q);
        } else {
            o = tensor(a[9]);
            need(shaped(o, ScalarType::BFloat16, q.sizes()));
        }
        float* lse = const_cast<float*>(
            static_cast<const float*>(optional(a[10], ScalarType::Float, {B, H})));
        const auto run = [&](void* ws, int bytes) {
            return g_fa.decode(q.const_data_ptr(), pool.k.const_data_ptr(),
                               pool.v.const_data_ptr(), s.k.const_data_ptr<float>(),
                               s.v.const_data_ptr<float>(), s.block, table.at, table.len,
                               table.max_pages, len_p, o.data_ptr(), lse, B, H, pool.Hk, pool.P, d,
                               page_size, scale, ws, bytes, stream());
        };
        const int rc = with_scratch(
            q, run, [&](int* bytes) { return g_fa.decode_bytes(B, H, pool.Hk, d, bytes); });
        return rc != FA_OK ? PyLong_FromLong(rc) : tuple_of({o});
    });
}

// (max_pos, rotary_dim, base, scaling, factor, original_len, low, high, mscale),
// the tables made on the current GPU
PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 9, [&]() -> PyObject* {
        const int max_pos = whole(a[0]), rot = whole(a[1]), scaling = whole(a[3]);
        need(max_pos > 0 && rot >= 2 && rot % 2 == 0);
        const double base = number(a[2]), factor = number(a[4]), low = number(a[6]),
                     high = number(a[7]), mscale = number(a[8]);
        const int original = whole(a[5]);
        const auto options = at::TensorOptions().dtype(ScalarType::Float).device(
            c10::Device(c10::kCUDA, c10::cuda::current_device()));
        const Tensor c = at::empty({max_pos, rot / 2}, options);
        const Tensor s = at::empty({max_pos, rot / 2}, options);
        const int rc = g_fa.rope_table(c.data_ptr<float>(), s.data_ptr<float>(), max_pos, rot,
                                       base, scaling, factor, original, low, high, mscale,
                                       stream());
        return rc != FA_OK ? PyLong_FromLong(rc) : tuple_of({c, s});
    });
}

// bind(addresses): those of Entry's functions, in its order
PyObject* bind(PyObject*, PyObject* arg) {
    constexpr Py_ssize_t count = sizeof(Entry) / sizeof(void*);
    void* at[count];
    if (!PyTuple_Check(arg) || PyTuple_GET_SIZE(arg) != count) {
        PyErr_SetString(PyExc_TypeError, "bind: one address for each entry point");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < count; ++i) {
        at[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(arg, i));
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    static_assert(sizeof(g_fa) == sizeof(at), "function pointers only");
    std::memcpy(&g_fa, at, sizeof(at));
    g_bound = true;
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"bind", bind, METH_O, nullptr},
                           {"rope_table", FAST(rope_table), nullptr},
                           {"norm", FAST(norm), nullptr},
                           {"norm_bwd", FAST(norm_bwd), nullptr},
                           {"append", FAST(append), nullptr},
                           {"decode", FAST(decode), nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods,
                        nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
    PyObject* m = PyModule_Create(&g_module);
    // for fa.py, which takes no other torch's
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
