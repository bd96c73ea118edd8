// The binding's calls of the step operators (planning, norm + rotation + cache
// write, attention of new tokens, plain and shaped): tensors checked, turned into pointers and
// passed to the library's entry points in one native call.
//
// A step's kernels take 2 to 10 us on small batches; checking a dozen tensors
// from Python took 4 to 9 us a call, and the foreign call's conversions 2 us
// more, so eager steps were bound by them.  Here a tensor costs some 20 ns.
//
// Each function takes its arguments by position, the current device and the
// stream's handle last, and returns the library's status.  A tensor of a wrong
// type, shape or place raises TypeError or ValueError before any call.

#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <limits>
#include <string>

#include "pa.h"

namespace {

// A Python exception to raise.
struct Refused {
    PyObject* type;
    std::string text;
};

std::string dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        default: return c10::toString(t);
    }
}

std::string list(at::IntArrayRef shape) {
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

// The arguments of one call.
class Call {
  public:
    Call(const char* where, PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : where_(where), args_(args) {
        if (n != want) throw Refused{PyExc_TypeError, std::string(where) + ": wrong number of arguments"};
        device_ = integer(n - 2);
        const auto handle = PyLong_AsUnsignedLongLong(args[n - 1]);
        if (PyErr_Occurred()) throw Refused{nullptr, ""};
        stream_ = reinterpret_cast<void*>(static_cast<uintptr_t>(handle));
    }

    bool none(int i) const { return args_[i] == Py_None; }
    void* stream() const { return stream_; }

    int integer(Py_ssize_t i) const {
        const long long v = PyLong_AsLongLong(args_[i]);
        if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
        if (v < std::numeric_limits<int>::min() || v > std::numeric_limits<int>::max())
            throw Refused{PyExc_ValueError, std::string(where_) + ": an argument is outside 32 bits"};
        return static_cast<int>(v);
    }
    // a size, as the entry points take it
    int size(int64_t v) const {
        if (v > std::numeric_limits<int>::max()) throw Refused{PyExc_ValueError, std::string(where_) + ": a size is past 31 bits"};
        return static_cast<int>(v);
    }
    float number(int i) const {
        const double v = PyFloat_AsDouble(args_[i]);
        if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
        return static_cast<float>(v);
    }

    const at::Tensor& tensor(int i, const char* name) const {
        if (!THPVariable_Check(args_[i])) refuse(PyExc_TypeError, name, "must be a torch.Tensor");
        return THPVariable_Unpack(args_[i]);
    }
    const at::Tensor& tensor(int i, const char* name, int64_t dims) const {
        const at::Tensor& t = tensor(i, name);
        if (t.dim() != dims) refuse(PyExc_ValueError, name, "must have " + std::to_string(dims) + " dimensions, got " + list(t.sizes()));
        return t;
    }

    // Address of a contiguous tensor of the current device; `shape` null: any.
    void* any(int i, const char* name, at::ScalarType dtype, const std::initializer_list<int64_t>* shape = nullptr) const {
        const at::Tensor& t = placed(i, name, dtype, shape);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, name, "must be contiguous");
        return const_cast<void*>(t.const_data_ptr());
    }
    void* at_(int i, const char* name, at::ScalarType dtype, std::initializer_list<int64_t> shape) const {
        return any(i, name, dtype, &shape);
    }
    // The like, and null for None.
    void* optional(int i, const char* name, at::ScalarType dtype) const { return none(i) ? nullptr : any(i, name, dtype); }
    void* optional(int i, const char* name, at::ScalarType dtype, std::initializer_list<int64_t> shape) const {
        return none(i) ? nullptr : any(i, name, dtype, &shape);
    }
    // Address and token stride of a bf16 tensor [T, heads, d] whose heads are contiguous within a token.
    void* token_rows(int i, const char* name, int64_t tokens, int64_t heads, int64_t d, int64_t& stride) const {
        const std::initializer_list<int64_t> shape = {tokens, heads, d};
        const at::Tensor& t = placed(i, name, at::kBFloat16, &shape);
        if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
            refuse(PyExc_ValueError, name, "must have the heads of a token contiguous");
        stride = tokens > 1 ? t.stride(0) : heads * d;
        return const_cast<void*>(t.const_data_ptr());
    }

    // A sequence of at most 64 small integers (bytes serve), its length in `n`.
    void small_ints(int i, const char* name, int8_t (&to)[64], int& n) const {
        PyObject* all = PySequence_Tuple(args_[i]);
        if (!all) {
            PyErr_Clear();
            refuse(PyExc_TypeError, name, "must be a sequence of integers");
        }
        const Py_ssize_t size = PyTuple_GET_SIZE(all);
        bool whole = true, fits = size <= 64;
        for (Py_ssize_t k = 0; whole && fits && k < size; ++k) {
            int overflow = 0;
            const long v = PyLong_AsLongAndOverflow(PyTuple_GET_ITEM(all, k), &overflow);
            whole = !PyErr_Occurred();
            fits = overflow == 0 && v >= -128 && v < 128;
            if (whole && fits) to[k] = static_cast<int8_t>(v);
        }
        Py_DECREF(all);
        PyErr_Clear();
        if (!whole) refuse(PyExc_TypeError, name, "must be a sequence of integers");
        if (!fits) refuse(PyExc_ValueError, name, "must be at most 64 small integers");
        n = static_cast<int>(size);
    }

    [[noreturn]] void refuse(PyObject* type, const char* name, const std::string& why) const {
        throw Refused{type, std::string(where_) + ": " + name + " " + why};
    }

  private:
    const at::Tensor& placed(int i, const char* name, at::ScalarType dtype, const std::initializer_list<int64_t>* shape) const {
        const at::Tensor& t = tensor(i, name);
        if (t.scalar_type() != dtype)
            refuse(PyExc_TypeError, name, "must be " + dtype_name(dtype) + ", got " + dtype_name(t.scalar_type()));
        if (!t.is_cuda() || t.get_device() != device_)
            refuse(PyExc_ValueError, name, "must be a CUDA tensor of the current device (" + std::to_string(device_) + "), got " + t.device().str());
        if (shape && t.sizes() != at::IntArrayRef(*shape))
            refuse(PyExc_ValueError, name, "must be " + list(*shape) + ", got " + list(t.sizes()));
        return t;
    }

    const char* where_;
    PyObject* const* args_;
    int device_;
    void* stream_;
};

// Runs `body` and returns its status, or raises.
template <class Body>
PyObject* guarded(const char* where, PyObject* const* args, Py_ssize_t n, Py_ssize_t want, Body body) {
    try {
        const Call c(where, args, n, want);
        return PyLong_FromLong(body(c));
    } catch (const Refused& r) {
        if (r.type) PyErr_SetString(r.type, r.text.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <class F>
int unlocked(F f) {
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f();
    Py_END_ALLOW_THREADS
    return status;
}

template <class T>
T* as(void* p) { return static_cast<T*>(p); }

// (block_tables, context_lens, query_start, positions, slot_mapping, seq_rows, new_lens, row_lens, row_tables,
//  row_blocks, free_blocks, free_count, block_size, num_blocks, status, device, stream)
PyObject* plan_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("pa_plan_step", args, n, 17, [](const Call& c) {
        const int64_t S = c.tensor(5, "seq_rows", 1).size(0), T = c.tensor(3, "positions", 1).size(0);
        const at::Tensor& rows = c.tensor(8, "row_tables", 2);
        const int64_t R = rows.size(0), MB = rows.size(1);
        void* tables = c.at_(0, "block_tables", at::kInt, {S, MB});
        void* ctx = c.at_(1, "context_lens", at::kInt, {S});
        void* start = c.at_(2, "query_start", at::kInt, {S + 1});
        void* positions = c.at_(3, "positions", at::kInt, {T});
        void* slots = c.at_(4, "slot_mapping", at::kLong, {T});
        void* seq_rows = c.at_(5, "seq_rows", at::kInt, {S});
        void* new_lens = c.at_(6, "new_lens", at::kInt, {S});
        void* row_lens = c.at_(7, "row_lens", at::kInt, {R});
        void* row_tables = c.at_(8, "row_tables", at::kInt, {R, MB});
        void* row_blocks = c.at_(9, "row_blocks", at::kInt, {R});
        void* free_blocks = c.optional(10, "free_blocks", at::kInt);
        void* free_count = c.optional(11, "free_count", at::kInt, {1});
        const int capacity = c.none(10) ? 0 : c.size(c.tensor(10, "free_blocks").numel());
        const int seqs = c.size(S), held = c.size(R), width = c.size(MB), tokens = c.size(T);
        const int block_size = c.integer(12), num_blocks = c.integer(13);
        void* status = c.optional(14, "status", at::kInt);
        return unlocked([&] {
            return pa_plan_step(as<int32_t>(tables), as<int32_t>(ctx), as<int32_t>(start), as<int32_t>(positions),
                                as<int64_t>(slots), as<int32_t>(seq_rows), as<int32_t>(new_lens), as<int32_t>(row_lens),
                                as<int32_t>(row_tables), as<int32_t>(row_blocks), as<int32_t>(free_blocks),
                                as<int32_t>(free_count), capacity, seqs, held, width, tokens, block_size, num_blocks,
                                as<int32_t>(status), c.stream());
        });
    });
}

// (rows, row_tables, row_blocks, free_blocks, free_count, status, device, stream)
PyObject* release_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("pa_release_rows", args, n, 8, [](const Call& c) {
        const int64_t S = c.tensor(0, "rows", 1).size(0);
        const at::Tensor& tables = c.tensor(1, "row_tables", 2);
        const int64_t R = tables.size(0), MB = tables.size(1);
        void* rows = c.at_(0, "rows", at::kInt, {S});
        void* row_tables = c.at_(1, "row_tables", at::kInt, {R, MB});
        void* row_blocks = c.at_(2, "row_blocks", at::kInt, {R});
        void* free_blocks = c.any(3, "free_blocks", at::kInt);
        void* free_count = c.at_(4, "free_count", at::kInt, {1});
        const int capacity = c.size(c.tensor(3, "free_blocks").numel()), released = c.size(S), held = c.size(R), width = c.size(MB);
        void* status = c.optional(5, "status", at::kInt);
        return unlocked([&] {
            return pa_release_rows(as<int32_t>(rows), released, as<int32_t>(row_tables), as<int32_t>(row_blocks), held, width,
                                   as<int32_t>(free_blocks), as<int32_t>(free_count), capacity, as<int32_t>(status),
                                   c.stream());
        });
    });
}

// (q_out, k_cache, v_cache, q, k, v, positions, slot_mapping, cos_sin, q_weight, k_weight, eps, interleaved, status,
//  k_scale, v_scale, device, stream)
PyObject* qk_norm_rope_cache(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("pa_qk_norm_rope_cache", args, n, 18, [](const Call& c) {
        const at::Tensor& queries = c.tensor(3, "q", 3);
        const at::Tensor& cache = c.tensor(1, "k_cache", 4);
        const int64_t T = queries.size(0), Hq = queries.size(1), D = queries.size(2);
        const int64_t NB = cache.size(0), Hkv = cache.size(1), B = cache.size(2);
        const bool f8 = !c.none(14);
        const at::ScalarType type = f8 ? at::kByte : at::kBFloat16;
        int64_t qs, ks, vs;
        void* q = c.token_rows(3, "q", T, Hq, D, qs);
        void* k = c.token_rows(4, "k", T, Hkv, D, ks);
        void* v = c.token_rows(5, "v", T, Hkv, D, vs);
        void* q_out = c.at_(0, "q_out", at::kBFloat16, {T, Hq, D});
        void* k_cache = c.at_(1, "k_cache", type, {NB, Hkv, B, D});
        void* v_cache = c.at_(2, "v_cache", type, {NB, Hkv, B, D});
        void* positions = c.at_(6, "positions", at::kInt, {T});
        void* slots = c.at_(7, "slot_mapping", at::kLong, {T});
        const at::Tensor& table = c.tensor(8, "cos_sin", 2);
        void* cos_sin = c.any(8, "cos_sin", at::kFloat);
        void* q_weight = c.optional(9, "q_weight", at::kFloat, {D});
        void* k_weight = c.optional(10, "k_weight", at::kFloat, {D});
        const float eps = c.number(11);
        const int interleaved = c.integer(12) != 0;
        void* status = c.optional(13, "status", at::kInt);
        const float k_scale = f8 ? c.number(14) : 0.f, v_scale = f8 ? c.number(15) : 0.f;
        const int max_positions = c.size(table.size(0)), rot = c.size(table.size(1)), tokens = c.size(T), hq = c.size(Hq),
                  hkv = c.size(Hkv), d = c.size(D), b = c.size(B), nb = c.size(NB);
        if (tokens == 0) return (int)PA_OK;                      // (empty tensors have no address)
        return unlocked([&] {
            return f8 ? pa_qk_norm_rope_cache_fp8(q_out, k_cache, v_cache, q, k, v, qs, ks, vs, as<float>(q_weight),
                                                  as<float>(k_weight), eps, as<float>(cos_sin), max_positions, rot, interleaved,
                                                  as<int32_t>(positions), as<int64_t>(slots), tokens, hq, hkv, d, b, nb, k_scale,
                                                  v_scale, as<int32_t>(status), c.stream())
                      : pa_qk_norm_rope_cache(q_out, k_cache, v_cache, q, k, v, qs, ks, vs, as<float>(q_weight),
                                              as<float>(k_weight), eps, as<float>(cos_sin), max_positions, rot, interleaved,
                                              as<int32_t>(positions), as<int64_t>(slots), tokens, hq, hkv, d, b, nb,
                                              as<int32_t>(status), c.stream());
        });
    });
}

// (out, q, k_cache, v_cache, block_tables, query_start, context_lens, max_query_len, block_size, scale, n_q_heads,
//  n_kv_heads, d_head, max_context_len, tree_mask, workspace, status, k_scale, v_scale, device, stream)
PyObject* decode_multi(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("pa_decode_multi", args, n, 21, [](const Call& c) {
        const at::Tensor& result = c.tensor(0, "out");
        if (result.scalar_type() != at::kBFloat16 && result.scalar_type() != at::kFloat)
            throw Refused{PyExc_TypeError, "pa_decode_multi: out must be bfloat16 or float32"};
        const int64_t T = c.tensor(1, "q", 3).size(0), NB = c.tensor(2, "k_cache", 4).size(0);
        const at::Tensor& entries = c.tensor(4, "block_tables", 2);
        const int64_t S = entries.size(0), MB = entries.size(1);
        const int most = c.integer(7), B = c.integer(8), Hq = c.integer(10), Hkv = c.integer(11), D = c.integer(12),
                  max_ctx = c.integer(13);
        const float scale = c.number(9);
        const bool f8 = !c.none(17);
        const at::ScalarType type = f8 ? at::kByte : at::kBFloat16;
        void* out = c.at_(0, "out", result.scalar_type(), {T, Hq, D});
        void* q = c.at_(1, "q", at::kBFloat16, {T, Hq, D});
        void* k = c.at_(2, "k_cache", type, {NB, Hkv, B, D});
        void* v = c.at_(3, "v_cache", type, {NB, Hkv, B, D});
        void* tables = c.at_(4, "block_tables", at::kInt, {S, MB});
        void* start = c.at_(5, "query_start", at::kInt, {S + 1});
        void* ctx = c.at_(6, "context_lens", at::kInt, {S});
        void* mask = c.optional(14, "tree_mask", at::kLong, {T});
        void* ws = c.any(15, "workspace", at::kByte);
        const size_t ws_bytes = static_cast<size_t>(c.tensor(15, "workspace").numel());
        void* status = c.optional(16, "status", at::kInt);
        const int dtype = result.scalar_type() == at::kFloat ? PA_DTYPE_F32 : PA_DTYPE_BF16;
        const int seqs = c.size(S), width = c.size(MB), tokens = c.size(T), nb = c.size(NB);
        const float k_scale = f8 ? c.number(17) : 0.f, v_scale = f8 ? c.number(18) : 0.f;
        return unlocked([&] {
            return f8 ? pa_decode_multi_fp8(out, dtype, q, k, v, as<int32_t>(tables), as<int32_t>(start), as<int32_t>(ctx),
                                            as<int64_t>(mask), B, scale, k_scale, v_scale, Hq, Hkv, D, seqs, tokens, most, width,
                                            nb, max_ctx, ws, ws_bytes, as<int32_t>(status), c.stream())
                      : pa_decode_multi(out, dtype, q, k, v, as<int32_t>(tables), as<int32_t>(start), as<int32_t>(ctx),
                                        as<int64_t>(mask), B, scale, Hq, Hkv, D, seqs, tokens, most, width, nb, max_ctx, ws,
                                        ws_bytes, as<int32_t>(status), c.stream());
        });
    });
}

// The axes of a rotation: positions [T] (axes None) or [A, T], and the axis of each pair.
struct Axes {
    const void* positions;
    int8_t of_pair[64];
    int num = 0;
    Axes(const Call& c, int at, int axes_at, int64_t T, int rot) {
        if (c.none(axes_at)) {
            positions = c.at_(at, "positions", at::kInt, {T});
            return;
        }
        num = c.size(c.tensor(at, "positions", 2).size(0));
        positions = c.at_(at, "positions", at::kInt, {num, T});
        int pairs;
        c.small_ints(axes_at, "axes", of_pair, pairs);
        if (2 * pairs != rot) c.refuse(PyExc_ValueError, "axes", "must have one entry for each pair that cos_sin turns");
        if (num == 0) c.refuse(PyExc_ValueError, "positions", "must have an axis");
    }
};

// (q_out, k_cache, v_cache, q, k, v, positions, axes, slot_mapping, cos_sin, q_weight, k_weight, eps, interleaved, status,
//  k_scale, v_scale, k_scales, v_scales, device, stream)
PyObject* qk_norm_mrope_cache(PyObject*, PyObject* const* args, Py_ssize_t n) {
    const bool to_scaled = n == 21 && args[17] != Py_None;
    return guarded(to_scaled ? "pa_qk_norm_rope_cache_scaled" : "pa_qk_norm_mrope_cache", args, n, 21, [](const Call& c) {
        const at::Tensor& queries = c.tensor(3, "q", 3);
        const at::Tensor& cache = c.tensor(1, "k_cache", 4);
        const int64_t T = queries.size(0), Hq = queries.size(1), D = queries.size(2);
        const int64_t NB = cache.size(0), Hkv = cache.size(1), B = cache.size(2);
        const bool scaled = !c.none(17), f8 = !c.none(15);
        const at::ScalarType type = f8 || scaled ? at::kByte : at::kBFloat16;
        int64_t qs, ks, vs;
        void* q = c.token_rows(3, "q", T, Hq, D, qs);
        void* k = c.token_rows(4, "k", T, Hkv, D, ks);
        void* v = c.token_rows(5, "v", T, Hkv, D, vs);
        void* q_out = c.at_(0, "q_out", at::kBFloat16, {T, Hq, D});
        void* k_cache = c.at_(1, "k_cache", type, {NB, Hkv, B, D});
        void* v_cache = c.at_(2, "v_cache", type, {NB, Hkv, B, D});
        const at::Tensor& table = c.tensor(9, "cos_sin", 2);
        const int max_positions = c.size(table.size(0)), rot = c.size(table.size(1));
        const Axes axes(c, 6, 7, T, rot);
        void* slots = c.at_(8, "slot_mapping", at::kLong, {T});
        void* cos_sin = c.any(9, "cos_sin", at::kFloat);
        void* q_weight = c.optional(10, "q_weight", at::kFloat, {D});
        void* k_weight = c.optional(11, "k_weight", at::kFloat, {D});
        const float eps = c.number(12);
        const int inter = c.integer(13) != 0;
        void* status = c.optional(14, "status", at::kInt);
        const float k_scale = f8 ? c.number(15) : 0.f, v_scale = f8 ? c.number(16) : 0.f;
        void* k_scales = c.optional(17, "k_scales", at::kByte, {NB, Hkv});
        void* v_scales = scaled ? c.at_(18, "v_scales", at::kByte, {NB, Hkv}) : nullptr;
        const int tokens = c.size(T), hq = c.size(Hq), hkv = c.size(Hkv), d = c.size(D), b = c.size(B), nb = c.size(NB);
        if (tokens == 0) return (int)PA_OK;                      // (empty tensors have no address)
        const int32_t* at = static_cast<const int32_t*>(axes.positions);
        return unlocked([&] {
            if (scaled)
                return pa_qk_norm_rope_cache_scaled(q_out, k_cache, v_cache, as<uint8_t>(k_scales), as<uint8_t>(v_scales), q, k, v,
                                                    qs, ks, vs, as<float>(q_weight), as<float>(k_weight), eps, as<float>(cos_sin),
                                                    max_positions, rot, inter, at, axes.num, axes.of_pair, as<int64_t>(slots),
                                                    tokens, hq, hkv, d, b, nb, as<int32_t>(status), c.stream());
            if (f8)
                return pa_qk_norm_mrope_cache_fp8(q_out, k_cache, v_cache, q, k, v, qs, ks, vs, as<float>(q_weight),
                                                  as<float>(k_weight), eps, as<float>(cos_sin), max_positions, rot, inter, at,
                                                  axes.num, axes.of_pair, as<int64_t>(slots), tokens, hq, hkv, d, b, nb, k_scale,
                                                  v_scale, as<int32_t>(status), c.stream());
            return pa_qk_norm_mrope_cache(q_out, k_cache, v_cache, q, k, v, qs, ks, vs, as<float>(q_weight), as<float>(k_weight),
                                          eps, as<float>(cos_sin), max_positions, rot, inter, at, axes.num, axes.of_pair,
                                          as<int64_t>(slots), tokens, hq, hkv, d, b, nb, as<int32_t>(status), c.stream());
        });
    });
}

// (k_cache, v_cache, k_scales, v_scales, k, v, slot_mapping, status, device, stream)
PyObject* reshape_and_cache_scaled(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("pa_reshape_and_cache_scaled", args, n, 10, [](const Call& c) {
        const at::Tensor& cache = c.tensor(0, "k_cache", 4);
        const int64_t NB = cache.size(0), Hkv = cache.size(1), B = cache.size(2), D = cache.size(3);
        const int64_t T = c.tensor(6, "slot_mapping", 1).size(0);
        int64_t ks, vs;
        void* k_cache = c.at_(0, "k_cache", at::kByte, {NB, Hkv, B, D});
        void* v_cache = c.at_(1, "v_cache", at::kByte, {NB, Hkv, B, D});
        void* k_scales = c.at_(2, "k_scales", at::kByte, {NB, Hkv});
        void* v_scales = c.at_(3, "v_scales", at::kByte, {NB, Hkv});
        void* k = c.token_rows(4, "k", T, Hkv, D, ks);
        void* v = c.token_rows(5, "v", T, Hkv, D, vs);
        void* slots = c.at_(6, "slot_mapping", at::kLong, {T});
        void* status = c.optional(7, "status", at::kInt);
        const int tokens = c.size(T), hkv = c.size(Hkv), d = c.size(D), b = c.size(B), nb = c.size(NB);
        if (tokens == 0) return (int)PA_OK;
        return unlocked([&] {
            return pa_reshape_and_cache_scaled(k_cache, v_cache, as<uint8_t>(k_scales), as<uint8_t>(v_scales), k, v, ks, vs,
                                               as<int64_t>(slots), tokens, hkv, d, b, nb, as<int32_t>(status), c.stream());
        });
    });
}

// (out, q, k_cache, v_cache, block_tables, query_start, context_lens, max_query_len, block_size, scale, n_q_heads,
//  n_kv_heads, d_head, max_context_len, visible, softcap, slopes, k_scales, v_scales, workspace, status, device, stream)
PyObject* attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("pa_attend", args, n, 23, [](const Call& c) {
        const at::Tensor& result = c.tensor(0, "out");
        if (result.scalar_type() != at::kBFloat16 && result.scalar_type() != at::kFloat)
            throw Refused{PyExc_TypeError, "pa_attend: out must be bfloat16 or float32"};
        const int64_t T = c.tensor(1, "q", 3).size(0), NB = c.tensor(2, "k_cache", 4).size(0);
        const at::Tensor& entries = c.tensor(4, "block_tables", 2);
        const int64_t S = entries.size(0), MB = entries.size(1);
        const int most = c.integer(7), B = c.integer(8), Hq = c.integer(10), Hkv = c.integer(11), D = c.integer(12),
                  max_ctx = c.integer(13);
        const float scale = c.number(9), cap = c.number(15);
        const bool scaled = !c.none(17);
        const at::ScalarType type = scaled ? at::kByte : at::kBFloat16;
        void* out = c.at_(0, "out", result.scalar_type(), {T, Hq, D});
        void* q = c.at_(1, "q", at::kBFloat16, {T, Hq, D});
        void* k = c.at_(2, "k_cache", type, {NB, Hkv, B, D});
        void* v = c.at_(3, "v_cache", type, {NB, Hkv, B, D});
        void* tables = c.at_(4, "block_tables", at::kInt, {S, MB});
        void* start = c.at_(5, "query_start", at::kInt, {S + 1});
        void* ctx = c.at_(6, "context_lens", at::kInt, {S});
        void* visible = c.optional(14, "visible", at::kInt, {T, 2});
        void* slopes = c.optional(16, "slopes", at::kFloat, {Hq});
        void* k_scales = c.optional(17, "k_scales", at::kByte, {NB, Hkv});
        void* v_scales = scaled ? c.at_(18, "v_scales", at::kByte, {NB, Hkv}) : nullptr;
        void* ws = c.any(19, "workspace", at::kByte);
        const size_t ws_bytes = static_cast<size_t>(c.tensor(19, "workspace").numel());
        void* status = c.optional(20, "status", at::kInt);
        const int dtype = result.scalar_type() == at::kFloat ? PA_DTYPE_F32 : PA_DTYPE_BF16;
        const int seqs = c.size(S), width = c.size(MB), tokens = c.size(T), nb = c.size(NB);
        return unlocked([&] {
            return scaled ? pa_attend_scaled(out, dtype, q, k, v, as<uint8_t>(k_scales), as<uint8_t>(v_scales), as<int32_t>(tables),
                                             as<int32_t>(start), as<int32_t>(ctx), as<int32_t>(visible), as<float>(slopes), cap, B,
                                             scale, Hq, Hkv, D, seqs, tokens, most, width, nb, max_ctx, ws, ws_bytes,
                                             as<int32_t>(status), c.stream())
                          : pa_attend(out, dtype, q, k, v, as<int32_t>(tables), as<int32_t>(start), as<int32_t>(ctx),
                                      as<int32_t>(visible), as<float>(slopes), cap, B, scale, Hq, Hkv, D, seqs, tokens, most, width,
                                      nb, max_ctx, ws, ws_bytes, as<int32_t>(status), c.stream());
        });
    });
}

#define PA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD(plan_step), PA_METHOD(release_rows), PA_METHOD(qk_norm_rope_cache),
                         PA_METHOD(decode_multi), PA_METHOD(qk_norm_mrope_cache), PA_METHOD(reshape_and_cache_scaled),
                         PA_METHOD(attend), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step_calls() { return PyModule_Create(&module); }
