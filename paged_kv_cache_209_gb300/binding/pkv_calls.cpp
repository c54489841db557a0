// The calls of a serving step's small launches, from Python tensors to libpkv without
// Python in between: a step of a few sequences runs for 3 to 10 us on the GPU, and
// checking and marshalling its dozen tensors in Python took 8 to 25 (planning a step 29
// us, here 5.5 to 8). Checks and outputs are those that pkv.py documents; a function returns
// (outputs, status), and pkv.py raises PkvError for a status that is not PKV_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "pkv.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string shape_text(at::IntArrayRef s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

const Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " is a tensor");
    return THPVariable_Unpack(o);
}
// The tensors of a call: on one device (the current one), of the given type and shape, contiguous.
struct Call {
    int here;
    const Tensor& on(const char* name, PyObject* o, at::ScalarType type) const {
        const Tensor& t = tensor(name, o);
        if (t.scalar_type() != type) throw Refused(std::string(name) + " is " + c10::toString(type) + ", not " + c10::toString(t.scalar_type()));
        if (!t.is_cuda() || t.get_device() != here)
            throw Refused("libpkv takes CUDA tensors only, on the current device (" + std::string(name) + " is on " + t.device().str() + ")");
        return t;
    }
    const Tensor& whole(const char* name, PyObject* o, at::ScalarType type) const {
        const Tensor& t = on(name, o, type);
        if (!t.is_contiguous()) throw Refused("libpkv takes contiguous tensors only (" + std::string(name) + ")");
        return t;
    }
    const Tensor& whole(const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef shape) const {
        const Tensor& t = whole(name, o, type);
        if (t.sizes() != shape) throw Refused(std::string(name) + " is " + shape_text(shape) + ", not " + shape_text(t.sizes()));
        return t;
    }
    const int32_t* ints(const char* name, PyObject* o, at::IntArrayRef shape) const {
        return static_cast<const int32_t*>(whole(name, o, at::kInt, shape).const_data_ptr());
    }
    // A fresh tensor (past the dispatcher, which takes as long as the allocation).
    Tensor fresh(at::ScalarType type, at::IntArrayRef shape) const {
        return Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(here)), std::nullopt));
    }
};

int64_t integer(const char* name, PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " is an integer");
    }
    return v;
}
int32_t integer32(const char* name, PyObject* o) {
    const int64_t v = integer(name, o);
    if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " is a 32-bit integer");
    return static_cast<int32_t>(v);
}
double number(const char* name, PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " is a number");
    }
    return v;
}
void* pointer(PyObject* o) { return o == Py_None ? nullptr : reinterpret_cast<void*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(o))); }
at::ScalarType type_of(int dtype) { return dtype == PKV_F32 ? at::kFloat : at::kBFloat16; }

// A checked call waits for the GPU: other Python threads run meanwhile.
template <typename F>
int call(uint32_t flags, F f) {
    if (!(flags & PKV_FLAG_CHECKED)) return f();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f();
    Py_END_ALLOW_THREADS
    return status;
}

PyObject* result(PyObject* out, int status) {
    if (out == nullptr) return nullptr;
    PyObject* r = Py_BuildValue("(Ni)", out, status);
    return r;
}
PyObject* none() { return Py_NewRef(Py_None); }
PyObject* two(PyObject* a, PyObject* b) {
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, a);
    PyTuple_SET_ITEM(r, 1, b);
    return r;
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", wanted, given);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "libpkv binding");
    }
    return nullptr;
}

// Geometry of a 4-bit cache.
struct Q4 {
    const Tensor& cache;
    pkv_cache_desc desc;
};
Q4 q4_of(const Call& c, PyObject* o) {
    const Tensor& t = tensor("cache", o);
    if (t.dim() != 3 || t.scalar_type() != at::kByte || (t.size(2) != PKV_Q4_RECORD_BYTES(64) && t.size(2) != PKV_Q4_RECORD_BYTES(128)))
        throw Refused("a 4-bit cache is uint8 [num_blocks][num_kv_heads][16 * head_dim + 128], head_dim 64 or 128");
    c.whole("cache", o, at::kByte);
    if (t.size(1) > INT32_MAX) throw Refused("a 4-bit cache's heads are a 32-bit number");
    return {t, pkv_cache_desc{t.size(0), 16, static_cast<int32_t>(t.size(1)), static_cast<int32_t>((t.size(2) - 128) / 16), PKV_INT4}};
}

struct Tables {
    const int32_t* at;
    int32_t batch, width;
};
Tables tables_of(const Call& c, PyObject* o) {
    const Tensor& t = c.whole("block_tables", o, at::kInt);
    if (t.dim() != 2) throw Refused("block_tables is [batch][max_blocks]");
    if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) throw Refused("batch and max_blocks are 32-bit numbers");
    return {static_cast<const int32_t*>(t.const_data_ptr()), static_cast<int32_t>(t.size(0)), static_cast<int32_t>(t.size(1))};
}

// attention_q4(here, q, cache, block_tables, context_lens, query_start | None, scale, max_query_len, out | None,
// workspace, flags, stream)
PyObject* attention_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Call c{integer32("here", a[0])};
        const Q4 p = q4_of(c, a[2]);
        const Tensor& q = c.whole("q", a[1], at::kBFloat16);
        if (q.dim() != 3 || q.size(2) != p.desc.head_dim || q.size(1) > INT32_MAX) throw Refused("q is bf16 [rows][q_heads][head_dim]");
        const Tables t = tables_of(c, a[3]);
        const int64_t rows = q.size(0);
        const bool decode = a[5] == Py_None;
        if (decode && rows != t.batch) throw Refused("q has one row per sequence");
        const int32_t* lens = c.ints("context_lens", a[4], {t.batch});
        const int32_t* start = decode ? nullptr : c.ints("query_start", a[5], {t.batch + 1});
        const float scale = static_cast<float>(number("scale", a[6]));
        const int32_t most = integer32("max_query_len", a[7]);
        const Tensor out = a[8] == Py_None ? c.fresh(at::kBFloat16, q.sizes()) : c.whole("out", a[8], at::kBFloat16, q.sizes());
        const Tensor& work = tensor("workspace", a[9]);
        c.whole("workspace", a[9], work.scalar_type());
        const uint32_t flags = static_cast<uint32_t>(integer("flags", a[10]));
        int status = PKV_OK;
        if (rows > 0) {  // (no query anywhere: no row to write)
            void* stream = pointer(a[11]);
            const int32_t heads = static_cast<int32_t>(q.size(1));
            status = call(flags, [&]() -> int {
                if (decode)
                    return pkv_decode_attention_q4(q.const_data_ptr(), p.cache.const_data_ptr(), t.at, t.width, lens, t.batch, heads, scale,
                                                   out.mutable_data_ptr(), work.mutable_data_ptr(), work.nbytes(), &p.desc, flags, stream);
                return pkv_multiquery_attention_q4(q.const_data_ptr(), p.cache.const_data_ptr(), t.at, t.width, lens, start, t.batch, heads, most,
                                                   scale, out.mutable_data_ptr(), work.mutable_data_ptr(), work.nbytes(), &p.desc, flags, stream);
            });
        }
        return result(a[8] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[8]), status);
    });
}

// gather_q4(here, cache, block_tables, context_lens, row_start, num_rows, token_start | None, out dtype, k_out | None,
// v_out | None, flags, stream)
PyObject* gather_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Call c{integer32("here", a[0])};
        const Q4 p = q4_of(c, a[1]);
        const Tables t = tables_of(c, a[2]);
        const int32_t* lens = c.ints("context_lens", a[3], {t.batch});
        const int32_t* start = c.ints("row_start", a[4], {t.batch + 1});
        const int64_t rows = integer("num_rows", a[5]);
        const int32_t* first = a[6] == Py_None ? nullptr : c.ints("token_start", a[6], {t.batch});
        const int32_t dtype = integer32("out_dtype", a[7]);
        const int64_t shape[3] = {rows, p.desc.num_kv_heads, p.desc.head_dim};
        if (rows < 0) throw Refused("num_rows is at least 0");
        Tensor out[2];
        const char* names[2] = {"k_out", "v_out"};
        for (int i = 0; i < 2; ++i)
            out[i] = a[8 + i] == Py_None ? c.fresh(type_of(dtype), shape) : c.whole(names[i], a[8 + i], type_of(dtype), shape);
        const uint32_t flags = static_cast<uint32_t>(integer("flags", a[10]));
        void* stream = pointer(a[11]);
        const int status = call(flags, [&]() -> int {
            return pkv_gather_q4(p.cache.const_data_ptr(), t.at, t.width, lens, first, start, t.batch, rows, out[0].mutable_data_ptr(),
                                 out[1].mutable_data_ptr(), dtype, &p.desc, flags, stream);
        });
        return result(two(a[8] == Py_None ? THPVariable_Wrap(out[0]) : Py_NewRef(a[8]), a[9] == Py_None ? THPVariable_Wrap(out[1]) : Py_NewRef(a[9])), status);
    });
}

// Rows [tokens][heads][head_dim] of which a token's heads follow one another: their address, and the stride between tokens.
struct Rows {
    const Tensor& t;
    int64_t stride;
};
Rows rows_of(const Call& c, const char* name, PyObject* o, at::ScalarType type, int64_t tokens, int64_t heads, int64_t d) {
    const Tensor& t = c.on(name, o, type);
    const int64_t shape[3] = {tokens, heads, d};
    if (t.sizes() != at::IntArrayRef(shape)) throw Refused(std::string(name) + " is " + shape_text(shape) + ", not " + shape_text(t.sizes()));
    if (tokens && heads && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))) throw Refused("a token's heads in " + std::string(name) + " follow one another");
    return {t, tokens > 1 ? t.stride(0) : heads * d};
}

// append_rotary(here, q | None, k, v, positions, table, slot_mapping, k_cache, v_cache | None, scales | None, interleaved,
// q_out | None, flags, stream); append_q4 with positions and table None, and no q
PyObject* append_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject* {
        const Call c{integer32("here", a[0])};
        pkv_cache_desc desc;
        void *v_cache = nullptr, *scales = nullptr;
        const Tensor& pool = tensor("k_cache", a[7]);
        if (a[8] == Py_None) {
            if (a[9] != Py_None) throw Refused("scales need v_cache");
            desc = q4_of(c, a[7]).desc;
        } else {
            const bool q8 = a[9] != Py_None;
            const auto type = pool.scalar_type();
            if (pool.dim() != 4) throw Refused("a pool is [num_blocks][num_kv_heads][16][head_dim]");
            if (q8 ? type != at::kChar : type != at::kFloat && type != at::kBFloat16)
                throw Refused(q8 ? "k_codes is int8 [num_blocks][num_kv_heads][16][head_dim]" : "unsupported dtype of the pools");
            const int64_t nb = pool.size(0), kv = pool.size(1), bs = pool.size(2), d = pool.size(3);
            c.whole("k_cache", a[7], type);
            v_cache = c.whole("v_cache", a[8], type, q8 ? at::IntArrayRef({nb, kv, d, bs}) : pool.sizes()).mutable_data_ptr();
            if (q8) scales = c.whole("scales", a[9], at::kFloat, {nb, kv, 2, bs}).mutable_data_ptr();
            desc = pkv_cache_desc{nb, static_cast<int32_t>(bs), static_cast<int32_t>(kv), static_cast<int32_t>(d),
                                  q8 ? PKV_INT8 : type == at::kFloat ? PKV_F32 : PKV_BF16};
        }
        const at::ScalarType type = desc.dtype == PKV_F32 ? at::kFloat : at::kBFloat16;
        const Tensor& slots = c.whole("slot_mapping", a[6], at::kLong);
        if (slots.dim() != 1) throw Refused("slot_mapping is [tokens]");
        const int64_t tokens = slots.size(0);
        const Rows k = rows_of(c, "k", a[2], type, tokens, desc.num_kv_heads, desc.head_dim);
        const Rows v = rows_of(c, "v", a[3], type, tokens, desc.num_kv_heads, desc.head_dim);
        const uint32_t flags = static_cast<uint32_t>(integer("flags", a[12]));
        void* stream = pointer(a[13]);
        void* pool_at = pool.mutable_data_ptr();
        if (a[4] == Py_None) {  // no positions: pkv_append_q4
            c.whole("k", a[2], type);
            c.whole("v", a[3], type);
            const int status = call(flags, [&]() -> int {
                return pkv_append_q4(k.t.const_data_ptr(), v.t.const_data_ptr(), static_cast<const int64_t*>(slots.const_data_ptr()), tokens, pool_at, &desc, flags, stream);
            });
            return result(none(), status);
        }
        const Tensor& table = c.whole("table", a[5], at::kFloat);
        if (table.dim() != 2) throw Refused("table is [positions][rotary_dim]");
        if (table.size(0) > INT32_MAX || table.size(1) > INT32_MAX) throw Refused("the table's sizes are 32-bit numbers");
        const int32_t* positions = c.ints("positions", a[4], {tokens});
        const void* q_at = nullptr;
        int64_t q_stride = 0, out_stride = 0;
        int32_t heads = 0;
        Tensor out;
        if (a[1] != Py_None) {
            const Tensor& q = tensor("q", a[1]);
            if (q.dim() != 3 || q.size(1) > INT32_MAX) throw Refused("q is [tokens][q_heads][head_dim]");
            const Rows r = rows_of(c, "q", a[1], type, tokens, q.size(1), desc.head_dim);
            heads = static_cast<int32_t>(q.size(1));
            q_at = r.t.const_data_ptr();
            q_stride = r.stride;
            if (a[11] == Py_None) {
                out = c.fresh(type, {tokens, q.size(1), desc.head_dim});
                out_stride = q.size(1) * desc.head_dim;
            } else {
                const Rows o = rows_of(c, "q_out", a[11], type, tokens, q.size(1), desc.head_dim);
                out = o.t;
                out_stride = o.stride;
            }
        } else if (a[11] != Py_None) {
            throw Refused("q_out needs q");
        }
        const int interleaved = PyObject_IsTrue(a[10]);
        const int status = call(flags, [&]() -> int {
            return pkv_append_rotary(q_at, q_stride, k.t.const_data_ptr(), k.stride, v.t.const_data_ptr(), v.stride, positions,
                                     static_cast<const float*>(table.const_data_ptr()), static_cast<int32_t>(table.size(0)), static_cast<int32_t>(table.size(1)),
                                     interleaved, static_cast<const int64_t*>(slots.const_data_ptr()), tokens, heads,
                                     out.defined() ? out.mutable_data_ptr() : nullptr, out_stride, pool_at, v_cache, static_cast<float*>(scales),
                                     &desc, flags, stream);
        });
        return result(!out.defined() ? none() : a[11] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[11]), status);
    });
}

// rotary_table(here, frequencies, num_positions, first_position, factor, out | None, stream)
PyObject* rotary_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const Call c{integer32("here", a[0])};
        const Tensor& f = c.whole("frequencies", a[1], at::kDouble);
        if (f.dim() != 1 || f.size(0) > INT32_MAX / 2) throw Refused("frequencies are [rotary_dim / 2]");
        const int64_t positions = integer("num_positions", a[2]), first = integer("first_position", a[3]);
        if (positions < 0) throw Refused("num_positions is at least 0");
        const float factor = static_cast<float>(number("factor", a[4]));
        const int64_t shape[2] = {positions, 2 * f.size(0)};
        const Tensor out = a[5] == Py_None ? c.fresh(at::kFloat, shape) : c.whole("out", a[5], at::kFloat, shape);
        const int status = pkv_rotary_table(static_cast<const double*>(f.const_data_ptr()), static_cast<int32_t>(shape[1]), first, positions, factor,
                                            static_cast<float*>(out.mutable_data_ptr()), pointer(a[6]));
        return result(a[5] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[5]), status);
    });
}

// `n` elements of a type in a fresh tensor's memory, from element `from` of that type on, as a tensor of their own. (A view
// through the dispatcher costs a microsecond.)
Tensor part_of(const Tensor& whole, at::ScalarType type, int64_t from, int64_t n) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    t.unsafeGetTensorImpl()->set_storage_offset(from);
    return t;
}

// plan_step(here, context_lens, new_tokens, held_blocks, free_blocks, free_count, block_tables, num_rows, num_blocks,
// out | None, flags, stream): out is the seven outputs
PyObject* plan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const Call c{integer32("here", a[0])};
        const Tables t = tables_of(c, a[6]);
        const int64_t batch = t.batch, rows = integer("num_rows", a[7]), blocks = integer("num_blocks", a[8]);
        const int32_t* lens = c.ints("context_lens", a[1], {batch});
        const int32_t* more = c.ints("new_tokens", a[2], {batch});
        const int32_t* held = c.ints("held_blocks", a[3], {batch});
        const Tensor& free = c.whole("free_blocks", a[4], at::kInt);
        if (free.dim() != 1) throw Refused("free_blocks is [capacity]");
        const int32_t* count = c.ints("free_count", a[5], {1});
        if (rows < 0) throw Refused("num_rows is at least 0");
        const int64_t sizes[7] = {rows, rows, batch + 1, batch, batch, 1, 2};
        void* at[7];
        Tensor outs[7];
        if (a[9] == Py_None) {
            // one allocation: the slots, then the numbers of 32 bits
            int64_t all = 2 * rows;
            for (int i = 1; i < 7; ++i) all += sizes[i];
            const Tensor whole = c.fresh(at::kInt, {all});
            outs[0] = part_of(whole, at::kLong, 0, rows);
            for (int64_t i = 1, from = 2 * rows; i < 7; from += sizes[i++]) outs[i] = part_of(whole, at::kInt, from, sizes[i]);
        } else {
            static const char* names[7] = {"slot_mapping", "positions", "query_start", "new_context_lens", "new_held_blocks", "new_free_count", "result"};
            if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 7)
                throw Refused("out holds slot_mapping, positions, query_start, new_context_lens, new_held_blocks, new_free_count, result");
            for (int i = 0; i < 7; ++i) outs[i] = c.whole(names[i], PyTuple_GET_ITEM(a[9], i), i ? at::kInt : at::kLong, {sizes[i]});
        }
        for (int i = 0; i < 7; ++i) at[i] = outs[i].mutable_data_ptr();
        auto ints = [&](int i) { return static_cast<int32_t*>(at[i]); };
        const uint32_t flags = static_cast<uint32_t>(integer("flags", a[10]));
        void* stream = pointer(a[11]);
        const int status = call(flags, [&]() -> int {
            return pkv_plan_step(lens, more, held, static_cast<const int32_t*>(free.const_data_ptr()), free.size(0), count, static_cast<int32_t*>(THPVariable_Unpack(a[6]).mutable_data_ptr()), t.width,
                                 t.batch, rows, blocks, static_cast<int64_t*>(at[0]), ints(1), ints(2), ints(3), ints(4), ints(5), ints(6), flags, stream);
        });
        if (a[9] != Py_None) return result(Py_NewRef(a[9]), status);
        PyObject* r = PyTuple_New(7);
        for (int i = 0; i < 7; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(outs[i]));
        return result(r, status);
    });
}

PyMethodDef methods[] = {{"attention_q4", reinterpret_cast<PyCFunction>(attention_q4), METH_FASTCALL, nullptr},
                         {"gather_q4", reinterpret_cast<PyCFunction>(gather_q4), METH_FASTCALL, nullptr},
                         {"append_rotary", reinterpret_cast<PyCFunction>(append_rotary), METH_FASTCALL, nullptr},
                         {"rotary_table", reinterpret_cast<PyCFunction>(rotary_table), METH_FASTCALL, nullptr},
                         {"plan_step", reinterpret_cast<PyCFunction>(plan_step), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_calls", "Calls of libpkv on torch tensors.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_calls() { return PyModule_Create(&module); }
