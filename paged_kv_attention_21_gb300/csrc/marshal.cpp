// marshal.cpp -- the Python binding's argument checks for the rotary, quantised-pool,
// score-rule and eviction entry points, next to torch's tensors: type, device, shape and layout of each tensor,
// then one call through the C ABI on torch's current stream or the one given.  A call takes
// the host 2.2 us, 1.65 of them the launch; the same checks over torch's Python attributes
// took 6 us more.
//
// Functions take positional arguments (the wrappers in __init__.py name them) and return
// the library's status; a tensor that fails a check raises ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <string>
#include <type_traits>

#include "../../include/pkv.h"

namespace {

// The library's entry points, looked up by init().
struct Library {
    decltype(&pkv_rope_rotate) rope_rotate;
    decltype(&pkv_quant_append) append;
    decltype(&pkv_quant_read) read;
    decltype(&pkv_quant_load_blocks) load_blocks;
    decltype(&pkv_quant_decode) decode;
    decltype(&pkv_score_decode) score_decode;
    decltype(&pkv_score_prefill) score_prefill;
    decltype(&pkv_score_mass) score_mass;
    decltype(&pkv_evict_select) evict_select;
    decltype(&pkv_evict_compact) evict_compact;
} g_lib{};
PyObject* g_table;    // the name "table"
PyObject* g_tensors;  // the name "tensors"

struct Refusal : std::exception {
    PyObject* type;
    char text[256];
    Refusal(PyObject* t, const char* fmt, ...) __attribute__((format(printf, 3, 4))) : type(t) {
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(text, sizeof(text), fmt, ap);
        va_end(ap);
    }
};
// A Python exception is already set.
struct Raised : std::exception {};

constexpr int64_t kAny = -1;  // matches any size

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refusal(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

// The address of o's data (null for None) once its type, device, shape and layout hold.
void* address(PyObject* o, const char* name, at::ScalarType type, int64_t device, std::initializer_list<int64_t> shape,
              bool dense = true) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
        throw Refusal(PyExc_ValueError, "%s: dtype %s, expected %s", name, c10::toString(t.scalar_type()), c10::toString(type));
    if (!t.is_cuda() || t.get_device() != device)
        throw Refusal(PyExc_ValueError, "%s: on %s, expected the current CUDA device", name, t.device().str().c_str());
    bool same = t.dim() == static_cast<int64_t>(shape.size());
    size_t i = 0;
    for (int64_t want : shape) {
        if (!same) break;
        same = want == kAny || t.sizes()[i] == want;
        ++i;
    }
    if (!same) {
        std::string got, want;
        for (int64_t s : t.sizes()) got += (got.empty() ? "" : ", ") + std::to_string(s);
        for (int64_t s : shape) want += (want.empty() ? "" : ", ") + (s == kAny ? std::string("any") : std::to_string(s));
        throw Refusal(PyExc_ValueError, "%s: shape (%s), expected (%s)", name, got.c_str(), want.c_str());
    }
    if (dense && !t.is_contiguous()) throw Refusal(PyExc_ValueError, "%s: tensor arguments must be contiguous", name);
    return t.data_ptr();
}

int64_t rows_of(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() < 1) throw Refusal(PyExc_ValueError, "%s: expected a tensor of rows", name);
    return t.sizes()[0];
}

long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
int32_t int32(PyObject* o, const char* name) {
    const long long v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Refusal(PyExc_ValueError, "%s: %lld does not fit 32 bits", name, v);
    return static_cast<int32_t>(v);
}
// The current device, or without one an index that no tensor has.
int64_t current_device() { return c10::cuda::device_count() > 0 ? c10::cuda::current_device() : -2; }
// o: a stream's address, or None for torch's current stream of the device.
pkv_stream_t stream_of(PyObject* o, int64_t device) {
    if (o == Py_None)
        return device < 0 ? nullptr
                          : reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (v == static_cast<unsigned long long>(-1) && PyErr_Occurred()) throw Raised();
    return reinterpret_cast<pkv_stream_t>(static_cast<uintptr_t>(v));
}

// A copy of the ctypes structure behind o.
template <typename T>
T structure(PyObject* o, const char* name) {
    Py_buffer view;
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw Raised();
    T v;
    const bool fits = view.len == static_cast<Py_ssize_t>(sizeof(T));
    if (fits) memcpy(&v, view.buf, sizeof(T));
    PyBuffer_Release(&view);
    if (!fits) throw Refusal(PyExc_ValueError, "%s: expected the structure of the C declaration", name);
    return v;
}

// The rotation behind o.  The table that make_rope keeps beside its address (a structure that
// was filled by hand has none) was on the device that was current then: it must be on this one.
pkv_rope rotation(PyObject* o, int64_t device) {
    const pkv_rope r = structure<pkv_rope>(o, "rope");
    PyObject* table = PyObject_GetAttr(o, g_table);
    if (!table) {
        PyErr_Clear();
        return r;
    }
    const bool is_tensor = THPVariable_Check(table);
    const c10::Device on = is_tensor ? THPVariable_Unpack(table).device() : c10::Device(c10::kCPU);
    Py_DECREF(table);
    if (is_tensor && (!on.is_cuda() || on.index() != device))
        throw Refusal(PyExc_ValueError, "rope table: on %s, expected the current CUDA device", on.str().c_str());
    return r;
}

struct Pools {
    pkv_cache_desc desc;
    void *k, *v;
    const float *k_scale, *v_scale;
    int64_t device;
    pkv_stream_t stream;
};
// args: desc, k_pool, v_pool, k_scale, v_scale, stream
Pools pools(PyObject* const* a) {
    Pools p;
    p.desc = structure<pkv_cache_desc>(a[0], "desc");
    p.device = current_device();
    p.stream = stream_of(a[5], p.device);
    const int64_t hkv = p.desc.num_kv_heads, d = p.desc.head_dim;
    const int64_t record = p.desc.kv_dtype == PKV_KV_INT8 ? 16 * d + 64 : 9 * d;
    p.k = address(a[1], "k_pool", at::kByte, p.device, {p.desc.num_blocks, hkv, record});
    p.v = address(a[2], "v_pool", at::kByte, p.device, {p.desc.num_blocks, hkv, record});
    p.k_scale = static_cast<const float*>(address(a[3], "k_scale", at::kFloat, p.device, {hkv}));
    p.v_scale = static_cast<const float*>(address(a[4], "v_scale", at::kFloat, p.device, {hkv}));
    return p;
}
constexpr int kPoolArgs = 6;

const int32_t* indexes(PyObject* o, const char* name, int64_t device, std::initializer_list<int64_t> shape) {
    return static_cast<const int32_t*>(address(o, name, at::kInt, device, shape));
}

int32_t count(int64_t n, const char* name) {
    if (n > INT32_MAX) throw Refusal(PyExc_ValueError, "%s: %lld rows", name, static_cast<long long>(n));
    return static_cast<int32_t>(n);
}

// [tokens][heads][head_dim] rows of any token and head strides.
pkv_rows strided_rows(PyObject* in, PyObject* out, const char* name, const char* out_name, at::ScalarType type, int64_t device,
                      int64_t tokens) {
    const at::Tensor& x = tensor(in, name);
    if (x.dim() != 3 || (x.sizes()[2] > 1 && x.strides()[2] != 1))
        throw Refusal(PyExc_ValueError, "%s: expected [tokens][heads][head_dim] with contiguous dims", name);
    if (x.sizes()[0] != tokens)
        throw Refusal(PyExc_ValueError, "%s: %lld tokens, but %lld positions", name, static_cast<long long>(x.sizes()[0]),
                      static_cast<long long>(tokens));
    pkv_rows r{};
    r.in = address(in, name, type, device, {tokens, x.sizes()[1], x.sizes()[2]}, false);
    r.out = const_cast<void*>(r.in);
    r.in_token_stride = r.out_token_stride = x.strides()[0];
    r.in_head_stride = r.out_head_stride = x.strides()[1];
    r.num_heads = count(x.sizes()[1], name);
    if (out != Py_None) {
        r.out = address(out, out_name, type, device, {tokens, x.sizes()[1], x.sizes()[2]}, false);
        const at::Tensor& y = tensor(out, out_name);
        if (y.sizes()[2] > 1 && y.strides()[2] != 1) throw Refusal(PyExc_ValueError, "%s: expected contiguous dims", out_name);
        r.out_token_stride = y.strides()[0];
        r.out_head_stride = y.strides()[1];
    }
    return r;
}

// bf16 rows whose heads are contiguous; *stride: elements between tokens.
void* token_rows(PyObject* o, const char* name, int64_t device, int64_t tokens, int64_t heads, int64_t dim, int64_t* stride) {
    void* at = address(o, name, at::kBFloat16, device, {tokens, heads, dim}, false);
    if (o == Py_None) throw Refusal(PyExc_ValueError, "%s is None", name);
    const at::Tensor& t = tensor(o, name);
    if (t.strides()[2] != 1 || (heads > 1 && t.strides()[1] != dim))
        throw Refusal(PyExc_ValueError, "%s: a token's heads must be contiguous", name);
    *stride = tokens > 1 ? t.strides()[0] : heads * dim;
    return at;
}

// Runs body with nargs checked, the library loaded, and C++ exceptions turned into Python's.
template <typename F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, F body) {
    try {
        if (nargs != want) throw Refusal(PyExc_TypeError, "expected %zd arguments, got %zd", want, nargs);
        if (!g_lib.decode) throw Refusal(PyExc_RuntimeError, "init() has not been called");
        return PyLong_FromLong(body());
    } catch (const Raised&) {
    } catch (const Refusal& e) {
        PyErr_SetString(e.type, e.text);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The library's call, which throws nothing: an exception must not leave while the lock is away.
template <typename F>
pkv_status without_gil(F call) {
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS st = call();
    Py_END_ALLOW_THREADS return st;
}

// rope, positions, q, q_out, k, k_out, stream
PyObject* rope_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const int64_t device = current_device();
        const pkv_rope rope = rotation(a[0], device);
        const int64_t tokens = rows_of(a[1], "positions");
        const pkv_stream_t stream = stream_of(a[6], device);
        const at::Tensor& q = tensor(a[2], "q");
        const at::ScalarType type = q.scalar_type();
        const int32_t code = type == at::kBFloat16 ? PKV_BF16 : type == at::kHalf ? PKV_F16 : PKV_F32;
        if (code == PKV_F32 && type != at::kFloat)
            throw Refusal(PyExc_ValueError, "q: dtype %s, expected BFloat16, Half or Float", c10::toString(type));
        const pkv_rows rows = strided_rows(a[2], a[3], "q", "q_out", type, device, tokens);
        const int32_t dim = count(q.sizes()[2], "head_dim");
        pkv_rows krows;
        const bool has_k = a[4] != Py_None;
        if (has_k) {
            krows = strided_rows(a[4], a[5], "k", "k_out", type, device, tokens);
            if (tensor(a[4], "k").sizes()[2] != dim) throw Refusal(PyExc_ValueError, "k: expected q's head_dim");
        }
        const int32_t* positions = indexes(a[1], "positions", device, {tokens});
        const int32_t num_tokens = count(tokens, "positions");
        return without_gil([&] {
            return g_lib.rope_rotate(&rope, code, positions, num_tokens, dim, &rows, has_k ? &krows : nullptr,
                                     stream);
        });
    });
}

// pools, rope, block_tables, token_to_seq, positions, k_new, v_new, q, q_out
PyObject* quant_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, kPoolArgs + 8, [&] {
        const Pools p = pools(args);
        PyObject* const* a = args + kPoolArgs;
        const int64_t tokens = rows_of(a[3], "positions"), seqs = rows_of(a[1], "block_tables"), dim = p.desc.head_dim;
        pkv_rope rope;
        const bool has_rope = a[0] != Py_None;
        if (has_rope) rope = rotation(a[0], p.device);
        const int32_t* tables = indexes(a[1], "block_tables", p.device, {seqs, p.desc.max_blocks_per_seq});
        const int32_t* tts = indexes(a[2], "token_to_seq", p.device, {tokens});
        const int32_t* positions = indexes(a[3], "positions", p.device, {tokens});
        int64_t k_stride, v_stride, q_stride = 0, qo_stride = 0;
        const void* k = token_rows(a[4], "k_new", p.device, tokens, p.desc.num_kv_heads, dim, &k_stride);
        const void* v = token_rows(a[5], "v_new", p.device, tokens, p.desc.num_kv_heads, dim, &v_stride);
        if (k_stride != v_stride)
            throw Refusal(PyExc_ValueError, "k_new and v_new: token strides %lld and %lld differ", static_cast<long long>(k_stride),
                          static_cast<long long>(v_stride));
        void *q = nullptr, *q_out = nullptr;
        if (a[6] != Py_None) {
            q_out = q = token_rows(a[6], "q", p.device, tokens, p.desc.num_q_heads, dim, &q_stride);
            qo_stride = q_stride;
            if (a[7] != Py_None) q_out = token_rows(a[7], "q_out", p.device, tokens, p.desc.num_q_heads, dim, &qo_stride);
        }
        const int32_t num_seqs = count(seqs, "block_tables"), num_tokens = count(tokens, "positions");
        return without_gil([&] {
            return g_lib.append(&p.desc, has_rope ? &rope : nullptr, p.k, p.v, p.k_scale, p.v_scale, tables, num_seqs, tts,
                                positions, num_tokens, k, v, k_stride, q, q_out, q_stride, qo_stride, p.stream);
        });
    });
}

// pools, block_tables, token_to_seq, positions, k_out, v_out
PyObject* quant_read(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, kPoolArgs + 5, [&] {
        const Pools p = pools(args);
        PyObject* const* a = args + kPoolArgs;
        if (a[3] == Py_None && a[4] == Py_None) throw Refusal(PyExc_ValueError, "k_out or v_out is needed");
        const int64_t tokens = rows_of(a[2], "positions"), seqs = rows_of(a[0], "block_tables");
        const at::ScalarType type = tensor(a[3] == Py_None ? a[4] : a[3], "k_out").scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat)
            throw Refusal(PyExc_ValueError, "outputs: dtype %s, expected BFloat16 or Float", c10::toString(type));
        const int32_t* tables = indexes(a[0], "block_tables", p.device, {seqs, p.desc.max_blocks_per_seq});
        const int32_t* tts = indexes(a[1], "token_to_seq", p.device, {tokens});
        const int32_t* positions = indexes(a[2], "positions", p.device, {tokens});
        void* k = address(a[3], "k_out", type, p.device, {tokens, p.desc.num_kv_heads, p.desc.head_dim});
        void* v = address(a[4], "v_out", type, p.device, {tokens, p.desc.num_kv_heads, p.desc.head_dim});
        const int32_t num_seqs = count(seqs, "block_tables"), num_tokens = count(tokens, "positions");
        return without_gil([&] {
            return g_lib.read(&p.desc, p.k, p.v, p.k_scale, p.v_scale, tables, num_seqs, tts, positions, num_tokens, type == at::kFloat ? PKV_F32 : PKV_BF16, k, v, p.stream);
        });
    });
}

// pools, src_blocks, dst_blocks, k_cache, v_cache
PyObject* quant_load_blocks(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, kPoolArgs + 4, [&] {
        const Pools p = pools(args);
        PyObject* const* a = args + kPoolArgs;
        const int64_t pairs = rows_of(a[0], "src_blocks"), blocks = rows_of(a[2], "k_cache");
        const int32_t* src = indexes(a[0], "src_blocks", p.device, {pairs});
        const int32_t* dst = indexes(a[1], "dst_blocks", p.device, {pairs});
        const std::initializer_list<int64_t> shape = {blocks, p.desc.num_kv_heads, p.desc.block_size, p.desc.head_dim};
        void* k = address(a[2], "k_cache", at::kBFloat16, p.device, shape);
        void* v = address(a[3], "v_cache", at::kBFloat16, p.device, shape);
        const int32_t num_pairs = count(pairs, "src_blocks");
        return without_gil([&] {
            return g_lib.load_blocks(&p.desc, p.k, p.v, p.k_scale, p.v_scale, src, dst, num_pairs, blocks, k, v, p.stream);
        });
    });
}

// pools, q, block_tables, context_lens, max_context_len, sm_scale, window, sinks, chunk_blocks, out, lse, workspace
PyObject* quant_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, kPoolArgs + 11, [&] {
        const Pools p = pools(args);
        PyObject* const* a = args + kPoolArgs;
        const int64_t seqs = rows_of(a[2], "context_lens"), hq = p.desc.num_q_heads, dim = p.desc.head_dim;
        const void* q = address(a[0], "q", at::kBFloat16, p.device, {seqs, hq, dim});
        const int32_t* tables = indexes(a[1], "block_tables", p.device, {seqs, p.desc.max_blocks_per_seq});
        const int32_t* lens = indexes(a[2], "context_lens", p.device, {seqs});
        const int32_t max_len = int32(a[3], "max_context_len"), window = int32(a[5], "window"), chunk = int32(a[7], "chunk_blocks");
        const double sm_scale = PyFloat_AsDouble(a[4]);
        if (sm_scale == -1.0 && PyErr_Occurred()) throw Raised();
        const float* sinks = static_cast<const float*>(address(a[6], "sinks", at::kFloat, p.device, {hq}));
        void* out = address(a[8], "out", at::kBFloat16, p.device, {seqs, hq, dim});
        float* lse = static_cast<float*>(address(a[9], "lse", at::kFloat, p.device, {seqs, hq}));
        void* ws = address(a[10], "workspace", at::kByte, p.device, {kAny});
        const size_t ws_bytes = ws ? static_cast<size_t>(rows_of(a[10], "workspace")) : 0;
        const int32_t num_seqs = count(seqs, "context_lens");
        return without_gil([&] {
            return g_lib.decode(&p.desc, q, p.k, p.v, p.k_scale, p.v_scale, tables, lens, num_seqs, max_len,
                                static_cast<float>(sm_scale), window, sinks, chunk, out, lse, ws, ws_bytes, p.stream);
        });
    });
}

// ------------------------------------------- the score rule and eviction --

// A bf16 pool, or an e4m3 pool's codes as bytes or float8_e4m3fn.
void* paged_pool(PyObject* o, const char* name, const pkv_cache_desc& desc, int64_t device) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    at::ScalarType type = at::kBFloat16;
    if (desc.kv_dtype == PKV_KV_FP8_E4M3)
        type = t.scalar_type() == at::kFloat8_e4m3fn ? at::kFloat8_e4m3fn : at::kByte;
    return address(o, name, type, device, {desc.num_blocks, desc.num_kv_heads, desc.block_size, desc.head_dim});
}

const float* floats(PyObject* o, const char* name, int64_t device, std::initializer_list<int64_t> shape) {
    return static_cast<const float*>(address(o, name, at::kFloat, device, shape));
}

// The score rule behind o.  The tensors that make_score keeps beside their addresses (a
// structure that was filled by hand has none) are held to this call's sizes and device.
pkv_score score_of(PyObject* o, int64_t device, int64_t hq, int64_t seqs) {
    pkv_score s = structure<pkv_score>(o, "score");
    PyObject* kept = PyObject_GetAttr(o, g_tensors);
    if (!kept) {
        PyErr_Clear();
        return s;
    }
    struct Held {
        PyObject* p;
        ~Held() { Py_DECREF(p); }
    } held{kept};
    if (!PyTuple_Check(kept) || PyTuple_GET_SIZE(kept) != 3) throw Refusal(PyExc_ValueError, "score: tensors are not make_score's");
    s.slopes = floats(PyTuple_GET_ITEM(kept, 0), "slopes", device, {hq});
    s.sinks = floats(PyTuple_GET_ITEM(kept, 1), "sinks", device, {hq});
    s.prefix_lens = indexes(PyTuple_GET_ITEM(kept, 2), "prefix_lens", device, {seqs});
    return s;
}

// Host int32 values behind an object with a buffer (a numpy array); None for none.
struct HostInts {
    Py_buffer view{};
    const int32_t* data = nullptr;
    HostInts(PyObject* o, const char* name, int64_t want) {
        if (o == Py_None) return;
        if (PyObject_GetBuffer(o, &view, PyBUF_CONTIG_RO) != 0) throw Raised();
        if (view.itemsize != 4 || view.len != 4 * want) {
            const long long got = view.len;
            PyBuffer_Release(&view);
            throw Refusal(PyExc_ValueError, "%s: %lld bytes, expected %lld int32 values", name, got, static_cast<long long>(want));
        }
        data = static_cast<const int32_t*>(view.buf);
    }
    HostInts(const HostInts&) = delete;
    ~HostInts() {
        if (data) PyBuffer_Release(&view);
    }
};

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return static_cast<float>(v);
}

// desc, score, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, max_context_len, chunk_blocks, out,
// lse, workspace, stream
PyObject* score_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const int64_t device = current_device();
        const pkv_cache_desc desc = structure<pkv_cache_desc>(a[0], "desc");
        const pkv_stream_t stream = stream_of(a[14], device);
        const int64_t seqs = rows_of(a[8], "context_lens"), hq = desc.num_q_heads, hkv = desc.num_kv_heads, dim = desc.head_dim;
        const pkv_score score = score_of(a[1], device, hq, seqs);
        const void* q = address(a[2], "q", at::kBFloat16, device, {seqs, hq, dim});
        const void* k = paged_pool(a[3], "k_cache", desc, device);
        const void* v = paged_pool(a[4], "v_cache", desc, device);
        const float* ks = floats(a[5], "k_scale", device, {hkv});
        const float* vs = floats(a[6], "v_scale", device, {hkv});
        const int32_t* tables = indexes(a[7], "block_tables", device, {seqs, desc.max_blocks_per_seq});
        const int32_t* lens = indexes(a[8], "context_lens", device, {seqs});
        const int32_t max_len = int32(a[9], "max_context_len"), chunk = int32(a[10], "chunk_blocks");
        void* out = address(a[11], "out", at::kBFloat16, device, {seqs, hq, dim});
        float* lse = const_cast<float*>(floats(a[12], "lse", device, {seqs, hq}));
        void* ws = address(a[13], "workspace", at::kByte, device, {kAny});
        const size_t ws_bytes = ws ? static_cast<size_t>(rows_of(a[13], "workspace")) : 0;
        const int32_t num_seqs = count(seqs, "context_lens");
        return without_gil([&] {
            return g_lib.score_decode(&desc, &score, q, k, v, ks, vs, tables, lens, num_seqs, max_len, chunk, out, lse, ws,
                                      ws_bytes, stream);
        });
    });
}

// desc, score, q, qo_indptr, k_cache, v_cache, k_scale, v_scale, block_tables, kv_lens, qo_indptr_host, kv_lens_host,
// causal, out, lse, stream
PyObject* score_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const int64_t device = current_device();
        const pkv_cache_desc desc = structure<pkv_cache_desc>(a[0], "desc");
        const pkv_stream_t stream = stream_of(a[15], device);
        const int64_t seqs = rows_of(a[9], "kv_lens"), rows = rows_of(a[2], "q");
        const int64_t hq = desc.num_q_heads, hkv = desc.num_kv_heads, dim = desc.head_dim;
        const pkv_score score = score_of(a[1], device, hq, seqs);
        const void* q = address(a[2], "q", at::kBFloat16, device, {rows, hq, dim});
        const int32_t* qo = indexes(a[3], "qo_indptr", device, {seqs + 1});
        const void* k = paged_pool(a[4], "k_cache", desc, device);
        const void* v = paged_pool(a[5], "v_cache", desc, device);
        const float* ks = floats(a[6], "k_scale", device, {hkv});
        const float* vs = floats(a[7], "v_scale", device, {hkv});
        const int32_t* tables = indexes(a[8], "block_tables", device, {seqs, desc.max_blocks_per_seq});
        const int32_t* lens = indexes(a[9], "kv_lens", device, {seqs});
        const HostInts qo_host(a[10], "qo_indptr_host", seqs + 1), lens_host(a[11], "kv_lens_host", seqs);
        const int causal = PyObject_IsTrue(a[12]);
        if (causal < 0) throw Raised();
        void* out = address(a[13], "out", at::kBFloat16, device, {rows, hq, dim});
        float* lse = const_cast<float*>(floats(a[14], "lse", device, {rows, hq}));
        const int32_t num_seqs = count(seqs, "kv_lens"), total = count(rows, "q");
        return without_gil([&] {
            return g_lib.score_prefill(&desc, &score, q, qo, k, v, ks, vs, tables, lens, num_seqs, total, qo_host.data,
                                       lens_host.data, causal, out, lse, stream);
        });
    });
}

// desc, score, q, qo_indptr, k_cache, k_scale, block_tables, kv_lens, max_q_len, max_kv_len, causal, lse, keep, mass,
// stream
PyObject* score_mass(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const int64_t device = current_device();
        const pkv_cache_desc desc = structure<pkv_cache_desc>(a[0], "desc");
        const pkv_stream_t stream = stream_of(a[14], device);
        const int64_t seqs = rows_of(a[7], "kv_lens"), rows = rows_of(a[2], "q");
        const int64_t hq = desc.num_q_heads, hkv = desc.num_kv_heads;
        const pkv_score score = score_of(a[1], device, hq, seqs);
        const void* q = address(a[2], "q", at::kBFloat16, device, {rows, hq, desc.head_dim});
        const int32_t* qo = indexes(a[3], "qo_indptr", device, {seqs + 1});
        const void* k = paged_pool(a[4], "k_cache", desc, device);
        const float* ks = floats(a[5], "k_scale", device, {hkv});
        const int32_t* tables = indexes(a[6], "block_tables", device, {seqs, desc.max_blocks_per_seq});
        const int32_t* lens = indexes(a[7], "kv_lens", device, {seqs});
        const int32_t max_q = int32(a[8], "max_q_len"), max_kv = int32(a[9], "max_kv_len");
        const int causal = PyObject_IsTrue(a[10]);
        if (causal < 0) throw Raised();
        const float* lse = floats(a[11], "lse", device, {rows, hq});
        const float keep = number(a[12]);
        float* mass = const_cast<float*>(floats(a[13], "mass", device, {seqs, hkv, kAny}));
        const int64_t stride = mass ? tensor(a[13], "mass").sizes()[2] : 0;
        const int32_t num_seqs = count(seqs, "kv_lens"), total = count(rows, "q");
        return without_gil([&] {
            return g_lib.score_mass(&desc, &score, q, qo, k, ks, tables, lens, num_seqs, total, max_q, max_kv, causal, lse,
                                    keep, mass, stride, stream);
        });
    });
}

// mass, kv_lens, max_kv_len, budget, first, recent, kept, kept_lens, stream
PyObject* evict_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const int64_t device = current_device();
        const pkv_stream_t stream = stream_of(a[8], device);
        const int64_t seqs = rows_of(a[1], "kv_lens");
        const float* mass = floats(a[0], "mass", device, {seqs, kAny, kAny});
        if (!mass && a[0] == Py_None) throw Refusal(PyExc_ValueError, "mass is None");
        const int64_t heads = tensor(a[0], "mass").sizes()[1], stride = tensor(a[0], "mass").sizes()[2];
        const int32_t* lens = indexes(a[1], "kv_lens", device, {seqs});
        const int32_t max_kv = int32(a[2], "max_kv_len"), budget = int32(a[3], "budget"), first = int32(a[4], "first"),
                      recent = int32(a[5], "recent");
        int32_t* kept = const_cast<int32_t*>(indexes(a[6], "kept", device, {seqs, heads, kAny}));
        const int64_t kept_stride = kept ? tensor(a[6], "kept").sizes()[2] : 0;
        int32_t* kept_lens = const_cast<int32_t*>(indexes(a[7], "kept_lens", device, {seqs}));
        const int32_t num_seqs = count(seqs, "kv_lens"), num_heads = count(heads, "mass");
        return without_gil([&] {
            return g_lib.evict_select(mass, stride, lens, num_seqs, num_heads, max_kv, budget, first, recent, kept,
                                      kept_stride, kept_lens, stream);
        });
    });
}

// desc, k_cache, v_cache, block_tables, kept, kept_lens, max_kept (None: kept's rows), dst_desc, k_dst, v_dst,
// dst_tables, mass, mass_out, stream
PyObject* evict_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const int64_t device = current_device();
        const pkv_cache_desc desc = structure<pkv_cache_desc>(a[0], "desc"), dst = structure<pkv_cache_desc>(a[7], "dst_desc");
        const pkv_stream_t stream = stream_of(a[13], device);
        const int64_t seqs = rows_of(a[5], "kept_lens"), hkv = desc.num_kv_heads;
        const void* k = paged_pool(a[1], "k_cache", desc, device);
        const void* v = paged_pool(a[2], "v_cache", desc, device);
        const int32_t* tables = indexes(a[3], "block_tables", device, {seqs, desc.max_blocks_per_seq});
        const int32_t* kept = indexes(a[4], "kept", device, {seqs, hkv, kAny});
        const int64_t kept_stride = a[4] == Py_None ? 0 : tensor(a[4], "kept").sizes()[2];
        const int32_t* kept_lens = indexes(a[5], "kept_lens", device, {seqs});
        void* kd = paged_pool(a[8], "k_dst", dst, device);
        void* vd = paged_pool(a[9], "v_dst", dst, device);
        const int32_t* dst_tables = indexes(a[10], "dst_tables", device, {seqs, dst.max_blocks_per_seq});
        const float* mass = floats(a[11], "mass", device, {seqs, hkv, kAny});
        float* mass_out = const_cast<float*>(floats(a[12], "mass_out", device, {seqs, hkv, kAny}));
        const int64_t stride = a[11] == Py_None ? 0 : tensor(a[11], "mass").sizes()[2];
        const int64_t out_stride = a[12] == Py_None ? 0 : tensor(a[12], "mass_out").sizes()[2];
        const int32_t max_kept = a[6] == Py_None ? count(kept_stride, "kept") : int32(a[6], "max_kept");
        const int32_t num_seqs = count(seqs, "kept_lens");
        return without_gil([&] {
            return g_lib.evict_compact(&desc, k, v, tables, kept, kept_stride, kept_lens, num_seqs, max_kept, &dst, kd, vd,
                                       dst_tables, mass, stride, mass_out, out_stride, stream);
        });
    });
}

// Look the entry points up in the library at `path`.
PyObject* init(PyObject*, PyObject* path) {
    const char* name = PyUnicode_AsUTF8(path);
    if (!name) return nullptr;
    void* lib = dlopen(name, RTLD_NOW | RTLD_LOCAL);
    if (!lib) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
    Library l{};
    auto find = [&](auto& fn, const char* symbol) {
        fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(dlsym(lib, symbol));
        if (!fn && !PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: no %s", name, symbol);
    };
    find(l.rope_rotate, "pkv_rope_rotate");
    find(l.append, "pkv_quant_append");
    find(l.read, "pkv_quant_read");
    find(l.load_blocks, "pkv_quant_load_blocks");
    find(l.decode, "pkv_quant_decode");
    find(l.score_decode, "pkv_score_decode");
    find(l.score_prefill, "pkv_score_prefill");
    find(l.score_mass, "pkv_score_mass");
    find(l.evict_select, "pkv_evict_select");
    find(l.evict_compact, "pkv_evict_compact");
    if (PyErr_Occurred()) return nullptr;
    if (!g_table && !(g_table = PyUnicode_InternFromString("table"))) return nullptr;
    if (!g_tensors && !(g_tensors = PyUnicode_InternFromString("tensors"))) return nullptr;
    g_lib = l;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"init", init, METH_O, nullptr},
    {"rope_rotate", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_rotate)), METH_FASTCALL, nullptr},
    {"quant_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_append)), METH_FASTCALL, nullptr},
    {"quant_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_read)), METH_FASTCALL, nullptr},
    {"quant_load_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_load_blocks)), METH_FASTCALL, nullptr},
    {"quant_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_decode)), METH_FASTCALL, nullptr},
    {"score_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(score_decode)), METH_FASTCALL, nullptr},
    {"score_prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(score_prefill)), METH_FASTCALL, nullptr},
    {"score_mass", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(score_mass)), METH_FASTCALL, nullptr},
    {"evict_select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict_select)), METH_FASTCALL, nullptr},
    {"evict_compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict_compact)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
