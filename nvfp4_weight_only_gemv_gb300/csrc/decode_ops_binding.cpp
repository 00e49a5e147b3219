// Checks and marshalling of the decode step's operators for Python (decode_ops.py).
//
// These calls are made several times per layer and token on rows of a few kilobytes, where a
// microsecond of the interpreter is a tenth of the whole call: checked in Python, a norm took 8 us, a
// rotary append 16 us and an attention call 12 us on the host, more than their kernels run. The functions take
// their arguments by position, raise TypeError or ValueError for a tensor that does not fit, and
// return the status of the C entry point, whose address `bind` receives.

#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "nvfp4_gemv.h"

namespace {

using RmsNorm = nvfp4_status (*)(const nvfp4_rms_norm_args*, void*);
using RopeAppend = nvfp4_status (*)(const nvfp4_rope_append_args*, void*);
using CacheRead = nvfp4_status (*)(const nvfp4_cache_read_args*, void*);
using PagedAttention = nvfp4_status (*)(const nvfp4_paged_attention_args*, const nvfp4_attention_scores*, void*);
RmsNorm g_rms_norm = nullptr;
RopeAppend g_rope_append = nullptr;
CacheRead g_cache_read = nullptr;
PagedAttention g_paged_attention = nullptr;

enum : unsigned { kF32 = 1, kBf16 = 2, kE4m3 = 4, kI32 = 8, kU8 = 16, kWide = kF32 | kBf16, kCache = kBf16 | kE4m3 | kU8 };

unsigned kind(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return kF32;
        case at::kBFloat16: return kBf16;
        case at::kFloat8_e4m3fn: return kE4m3;
        case at::kInt: return kI32;
        case at::kByte: return kU8;
        default: return 0;
    }
}
int code(const at::Tensor& t) { return kind(t) == kF32 ? NVFP4_F32 : kind(t) == kBf16 ? NVFP4_BF16 : NVFP4_E4M3; }

const char* names_of(unsigned kinds) {
    switch (kinds) {
        case kF32: return "torch.float32";
        case kBf16: return "torch.bfloat16";
        case kE4m3: return "torch.float8_e4m3fn";
        case kI32: return "torch.int32";
        case kU8: return "torch.uint8";
        case kWide: return "torch.float32 or torch.bfloat16";
        case kCache: return "torch.bfloat16, torch.float8_e4m3fn or torch.uint8 (4 bits)";
        default: return "torch.float32, torch.bfloat16 or torch.float8_e4m3fn";
    }
}

// The error of a check is a Python exception that is already set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* format, const char* a, const char* b = "", long long c = 0, long long d = 0) {
    PyErr_Format(type, format, a, b, c, d);
    throw Refused{};
}

struct Checks {
    int dev = -2;  // the current CUDA device; no tensor is on -2
    Checks() {
        c10::DeviceIndex current = 0;
        if (c10::cuda::GetDevice(&current) == cudaSuccess) dev = current;
    }
    const at::Tensor& any(PyObject* o, const char* name, unsigned kinds, int dims) const {
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
        if (!(kind(t) & kinds)) refuse(PyExc_TypeError, "%s must be %s", name, names_of(kinds));
        if (t.dim() != dims) refuse(PyExc_ValueError, "%s must have %s%lld dims (got %lld)", name, "", dims, t.dim());
        if (t.get_device() != dev)
            refuse(PyExc_ValueError, "%s: every tensor must be on the current CUDA device%s cuda:%lld (got cuda:%lld)", name, "", dev,
                   t.get_device());
        if (t.size(dims - 1) > 1 && t.stride(dims - 1) != 1)
            refuse(PyExc_ValueError, "%s must have unit stride in its last dimension", name);
        return t;
    }
    const at::Tensor& whole(PyObject* o, const char* name, unsigned kinds, int dims) const {
        const at::Tensor& t = any(o, name, kinds, dims);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
        return t;
    }
    // a contiguous vector of n values
    const at::Tensor& vector(PyObject* o, const char* name, unsigned kinds, long long n) const {
        const at::Tensor& t = whole(o, name, kinds, 1);
        if (t.size(0) != n) refuse(PyExc_ValueError, "%s must have %s%lld values (got %lld)", name, "", n, t.size(0));
        return t;
    }
    const float* head_scale(PyObject* o, const char* name, const at::Tensor& cache) const {
        if (o == Py_None) return nullptr;
        if (kind(cache) == kBf16) refuse(PyExc_ValueError, "%s belongs to a float8_e4m3fn or 4-bit cache", name);
        return static_cast<const float*>(vector(o, name, kF32, cache.size(1)).data_ptr());
    }
    void* stream(PyObject* o) const {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
        void* s = PyLong_AsVoidPtr(o);
        if (!s && PyErr_Occurred()) throw Refused{};
        return s;
    }
};

long long integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return static_cast<float>(v);
}
int truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v;
}
int size32(int64_t v, const char* name) {
    if (v > INT32_MAX) refuse(PyExc_ValueError, "%s is too large", name);
    return static_cast<int>(v);
}
void same_shape(const at::Tensor& a, const at::Tensor& b, const char* name, const char* like) {
    if (a.sizes() != b.sizes()) refuse(PyExc_ValueError, "%s must have the shape of %s", name, like);
}

// Runs `f`, whose failed checks have set an exception, and returns the status as a Python int.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
    try {
        if (given != wanted) refuse(PyExc_TypeError, "%s%s%lld arguments wanted (got %lld)", "", "", wanted, given);
        return PyLong_FromLong(f());
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// (x, weight, eps, residual, residual_out, out, scales, group, stream)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> int {
        const Checks c;
        nvfp4_rms_norm_args g{};
        const at::Tensor& x = c.any(a[0], "x", kWide, 2);
        g.rows = size32(x.size(0), "x");
        g.cols = size32(x.size(1), "x");
        const at::Tensor& w = c.vector(a[1], "weight", kWide, g.cols);
        const at::Tensor& y = c.any(a[5], "out", kWide | kE4m3, 2);
        same_shape(y, x, "out", "x");
        g.x = x.data_ptr(); g.weight = w.data_ptr(); g.y = y.data_ptr();
        g.ldx = x.stride(0); g.ldy = y.stride(0);
        g.x_type = code(x); g.w_type = code(w); g.y_type = code(y);
        g.eps = real(a[2]);
        if (a[3] != Py_None) {
            const at::Tensor& r = c.any(a[3], "residual", kWide, 2);
            const at::Tensor& ro = c.any(a[4], "residual_out", kind(r), 2);
            same_shape(r, x, "residual", "x");
            same_shape(ro, x, "residual_out", "x");
            g.residual = r.data_ptr(); g.residual_out = ro.data_ptr();
            g.ldr = r.stride(0); g.ldro = ro.stride(0);
            g.residual_type = code(r);
        } else if (a[4] != Py_None) {
            refuse(PyExc_ValueError, "%s", "residual_out without a residual");
        }
        g.group = static_cast<int32_t>(integer(a[7], "group"));
        if (g.y_type == NVFP4_E4M3) {
            const at::Tensor& s = c.whole(a[6], "scales", kF32, 2);
            const long long per_row = g.group > 0 ? g.cols / g.group : 1;
            if ((g.group > 0 && g.cols % g.group) || s.size(0) != g.rows || s.size(1) != per_row)
                refuse(PyExc_ValueError, "%s must be [rows, 1], or [rows, cols / group] for a group that divides the columns", "scales");
            g.scales = static_cast<float*>(s.data_ptr());
        } else if (a[6] != Py_None || g.group) {
            refuse(PyExc_ValueError, "%s belong to a float8_e4m3fn output", "scales and group");
        }
        return g_rms_norm(&g, c.stream(a[8]));
    });
}

struct Caches {
    const at::Tensor& k;
    const at::Tensor& v;
    int type;
    int64_t head_dim;
};
Caches caches(const Checks& c, PyObject* ko, PyObject* vo) {
    const at::Tensor& k = c.any(ko, "k_cache", kCache, 4);
    const at::Tensor& v = c.any(vo, "v_cache", kind(k), 4);
    same_shape(v, k, "v_cache", "k_cache");
    const int64_t heads = k.size(1), page = k.size(2), dim = k.size(3);
    for (const at::Tensor* t : {&k, &v})
        if (t->numel() && ((page > 1 && t->stride(2) != dim) || (heads > 1 && t->stride(1) != page * dim)))
            refuse(PyExc_ValueError, "%s must be contiguous inside a page", t == &k ? "k_cache" : "v_cache");
    if (kind(k) != kU8) return {k, v, code(k), dim};
    // records of 16 keys and 9 head_dim bytes
    if (dim % 9) refuse(PyExc_ValueError, "%s hold 9 bytes for 16 values of a head: %s%lld bytes do not divide", "4-bit caches", "", dim);
    if (page % 16) refuse(PyExc_ValueError, "%s have pages of a multiple of 16 keys%s (got %lld)", "4-bit caches", "", page);
    return {k, v, NVFP4_E2M1, dim / 9 * 16};
}

// (q, k, v, positions, inv_freq, k_cache, v_cache, page_table, seq_ids, interleaved, mscale, q_norm,
//  k_norm, eps, k_scale, v_scale, out, stream)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 18, [&]() -> int {
        const Checks c;
        nvfp4_rope_append_args g{};
        const at::Tensor& k = c.any(a[1], "k", kWide, 3);
        const at::Tensor& v = c.any(a[2], "v", kind(k), 3);
        same_shape(v, k, "v", "k");
        const Caches cache = caches(c, a[5], a[6]);
        g.tokens = size32(k.size(0), "k");
        g.kv_heads = size32(k.size(1), "k");
        g.head_dim = size32(k.size(2), "k");
        if (cache.k.size(1) != g.kv_heads || cache.head_dim != g.head_dim)
            refuse(PyExc_ValueError, "%s do not have the heads of k", "the caches");
        const at::Tensor& pos = c.vector(a[3], "positions", kI32, g.tokens);
        const at::Tensor& freq = c.whole(a[4], "inv_freq", kF32, 1);
        if (2 * freq.size(0) > g.head_dim)
            refuse(PyExc_ValueError, "%s turns %s%lld values of a head of %lld", "inv_freq", "", 2 * freq.size(0), g.head_dim);
        const at::Tensor& table = c.any(a[7], "page_table", kI32, 2);
        g.seqs = size32(table.size(0), "page_table");
        if (a[8] != Py_None) g.seq_ids = static_cast<const int32_t*>(c.vector(a[8], "seq_ids", kI32, g.tokens).data_ptr());
        else if (g.seqs == 0 ? g.tokens != 0 : g.tokens % g.seqs != 0)
            refuse(PyExc_ValueError, "%s do not divide among the sequences: pass seq_ids", "the tokens");
        unsigned norm_kind = kWide;
        if (a[11] != Py_None) {
            const at::Tensor& w = c.vector(a[11], "q_norm", norm_kind, g.head_dim);
            norm_kind = kind(w);
            g.q_norm = w.data_ptr(); g.norm_type = code(w);
        }
        if (a[12] != Py_None) {
            const at::Tensor& w = c.vector(a[12], "k_norm", norm_kind, g.head_dim);
            g.k_norm = w.data_ptr(); g.norm_type = code(w);
        }
        if (a[0] != Py_None) {
            const at::Tensor& q = c.any(a[0], "q", kind(k), 3);
            if (q.size(0) != g.tokens || q.size(2) != g.head_dim)
                refuse(PyExc_ValueError, "%s must be [tokens, heads, head_dim] like k", "q");
            const at::Tensor& out = c.whole(a[16], "out", kBf16, 3);
            same_shape(out, q, "out", "q");
            g.q_heads = size32(q.size(1), "q");
            g.q = q.data_ptr(); g.q_out = out.data_ptr();
            g.q_token_stride = q.stride(0); g.q_head_stride = q.stride(1);
        } else if (a[16] != Py_None || g.q_norm) {
            refuse(PyExc_ValueError, "%s belong to q", "out and q_norm");
        }
        g.k = k.data_ptr(); g.v = v.data_ptr();
        g.k_token_stride = k.stride(0); g.k_head_stride = k.stride(1);
        g.v_token_stride = v.stride(0); g.v_head_stride = v.stride(1);
        g.positions = static_cast<const int32_t*>(pos.data_ptr());
        g.inv_freq = static_cast<const float*>(freq.data_ptr());
        g.rotary_half = size32(freq.size(0), "inv_freq");
        g.k_cache = cache.k.data_ptr(); g.v_cache = cache.v.data_ptr();
        g.k_page_stride = cache.k.stride(0); g.v_page_stride = cache.v.stride(0);
        g.k_scale = c.head_scale(a[14], "k_scale", cache.k);
        g.v_scale = c.head_scale(a[15], "v_scale", cache.v);
        g.page_table = static_cast<const int32_t*>(table.data_ptr());
        g.table_stride = table.stride(0);
        g.x_type = code(k); g.cache_type = cache.type;
        g.pages = size32(cache.k.size(0), "k_cache");
        g.max_pages = size32(table.size(1), "page_table");
        g.page_size = size32(cache.k.size(2), "k_cache");
        g.interleaved = truth(a[9]);
        g.mscale = real(a[10]);
        g.eps = real(a[13]);
        return g_rope_append(&g, c.stream(a[17]));
    });
}

// (positions, k_cache, v_cache, page_table, seq_ids, k_scale, v_scale, k_out, v_out, stream)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> int {
        const Checks c;
        nvfp4_cache_read_args g{};
        const Caches cache = caches(c, a[1], a[2]);
        const at::Tensor& pos = c.whole(a[0], "positions", kI32, 1);
        g.tokens = size32(pos.size(0), "positions");
        g.kv_heads = size32(cache.k.size(1), "k_cache");
        g.head_dim = size32(cache.head_dim, "k_cache");
        const at::Tensor& table = c.any(a[3], "page_table", kI32, 2);
        g.seqs = size32(table.size(0), "page_table");
        if (a[4] != Py_None) g.seq_ids = static_cast<const int32_t*>(c.vector(a[4], "seq_ids", kI32, g.tokens).data_ptr());
        else if (g.seqs == 0 ? g.tokens != 0 : g.tokens % g.seqs != 0)
            refuse(PyExc_ValueError, "%s do not divide among the sequences: pass seq_ids", "the tokens");
        const at::Tensor& ko = c.whole(a[7], "k_out", kBf16, 3);
        const at::Tensor& vo = c.whole(a[8], "v_out", kBf16, 3);
        for (const at::Tensor* t : {&ko, &vo})
            if (t->size(0) != g.tokens || t->size(1) != g.kv_heads || t->size(2) != g.head_dim)
                refuse(PyExc_ValueError, "%s must be [tokens, kv_heads, head_dim]", t == &ko ? "k_out" : "v_out");
        g.positions = static_cast<const int32_t*>(pos.data_ptr());
        g.k_cache = cache.k.data_ptr(); g.v_cache = cache.v.data_ptr();
        g.k_page_stride = cache.k.stride(0); g.v_page_stride = cache.v.stride(0);
        g.k_scale = c.head_scale(a[5], "k_scale", cache.k);
        g.v_scale = c.head_scale(a[6], "v_scale", cache.v);
        g.page_table = static_cast<const int32_t*>(table.data_ptr());
        g.table_stride = table.stride(0);
        g.k_out = ko.data_ptr(); g.v_out = vo.data_ptr();
        g.cache_type = cache.type;
        g.pages = size32(cache.k.size(0), "k_cache");
        g.max_pages = size32(table.size(1), "page_table");
        g.page_size = size32(cache.k.size(2), "k_cache");
        return g_cache_read(&g, c.stream(a[9]));
    });
}

// (q, k_cache, v_cache, page_table, lengths, scale, window, softcap, slopes, k_scale, v_scale, workspace, out, lse, stream)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> int {
        const Checks c;
        nvfp4_paged_attention_args g{};
        const at::Tensor& q = c.any(a[0], "q", kBf16, 3);
        const Caches cache = caches(c, a[1], a[2]);
        const at::Tensor& table = c.any(a[3], "page_table", kI32, 2);
        g.seqs = size32(table.size(0), "page_table");
        const at::Tensor& lengths = c.vector(a[4], "lengths", kI32, g.seqs);
        const int64_t tokens = q.size(0);
        g.q_heads = size32(q.size(1), "q");
        g.head_dim = size32(q.size(2), "q");
        g.kv_heads = size32(cache.k.size(1), "k_cache");
        if (cache.head_dim != g.head_dim) refuse(PyExc_ValueError, "%s do not have the head size of q", "the caches");
        if (g.seqs ? tokens % g.seqs != 0 : tokens != 0)
            refuse(PyExc_ValueError, "%s does not have the same number of rows for every sequence of page_table", "q");
        if (g.kv_heads ? g.q_heads % g.kv_heads != 0 : g.q_heads != 0)
            refuse(PyExc_ValueError, "%s do not divide among the kv heads", "the query heads");
        g.rows = g.seqs ? size32(tokens / g.seqs, "q") : 0;
        const at::Tensor& ws = c.whole(a[11], "workspace", kU8, 1);
        const at::Tensor& out = c.whole(a[12], "out", kBf16, 3);
        same_shape(out, q, "out", "q");
        if (a[13] != Py_None) {
            const at::Tensor& lse = c.whole(a[13], "lse", kF32, 2);
            if (lse.size(0) != tokens || lse.size(1) != g.q_heads)
                refuse(PyExc_ValueError, "%s must be [rows, heads] like q", "lse");
            g.lse = static_cast<float*>(lse.data_ptr());
        }
        g.q = q.data_ptr(); g.out = out.data_ptr(); g.workspace = ws.data_ptr();
        g.workspace_bytes = ws.numel();
        g.q_token_stride = q.stride(0); g.q_head_stride = q.stride(1);
        g.k_cache = cache.k.data_ptr(); g.v_cache = cache.v.data_ptr();
        g.k_page_stride = cache.k.stride(0); g.v_page_stride = cache.v.stride(0);
        g.k_scale = c.head_scale(a[9], "k_scale", cache.k);
        g.v_scale = c.head_scale(a[10], "v_scale", cache.v);
        g.page_table = static_cast<const int32_t*>(table.data_ptr());
        g.table_stride = table.stride(0);
        g.lengths = static_cast<const int32_t*>(lengths.data_ptr());
        g.cache_type = cache.type;
        g.pages = size32(cache.k.size(0), "k_cache");
        g.max_pages = size32(table.size(1), "page_table");
        g.page_size = size32(cache.k.size(2), "k_cache");
        g.window = static_cast<int32_t>(integer(a[6], "window"));
        g.scale = real(a[5]);
        nvfp4_attention_scores scores{};
        scores.softcap = real(a[7]);
        // a cap that only becomes zero here is too small, and no leave to go without one
        if (scores.softcap == 0.0f && PyFloat_AsDouble(a[7]) != 0.0) return NVFP4_ERR_SHAPE;
        if (a[8] != Py_None) scores.slopes = static_cast<const float*>(c.vector(a[8], "slopes", kF32, g.q_heads).data_ptr());
        return g_paged_attention(&g, &scores, c.stream(a[14]));
    });
}

// (address of nvfp4_rms_norm, of nvfp4_rope_append, of nvfp4_cache_read, of nvfp4_paged_attention_scored)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> int {
        void* at[4];
        for (int i = 0; i < 4; ++i) {
            at[i] = PyLong_AsVoidPtr(a[i]);
            if (!at[i]) {
                if (PyErr_Occurred()) throw Refused{};
                refuse(PyExc_ValueError, "%s", "null address");
            }
        }
        g_rms_norm = reinterpret_cast<RmsNorm>(at[0]);
        g_rope_append = reinterpret_cast<RopeAppend>(at[1]);
        g_cache_read = reinterpret_cast<CacheRead>(at[2]);
        g_paged_attention = reinterpret_cast<PagedAttention>(at[3]);
        return 0;
    });
}

#define NVFP4_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {NVFP4_METHOD(bind), NVFP4_METHOD(rms_norm), NVFP4_METHOD(rope_append), NVFP4_METHOD(cache_read),
                           NVFP4_METHOD(paged_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_decode_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode_ops() { return PyModule_Create(&g_module); }
