// Argument marshalling of the norm, block-scale and block-attention calls as a
// CPython extension: the checks binding.py documents, then the C ABI call.
//
// A decode step makes these calls once per layer and their kernels take a few
// microseconds; the same checks written in Python cost 10 us a call, here
// about 1. Every function returns the call's pa_status and raises TypeError
// or ValueError for tensors the C ABI must not see: type first, then shape and
// layout, the device last. No CUDA call is made before every check has passed.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <sstream>
#include <string>

#include "../../include/pagedattn.h"

namespace {

struct Refusal {
  PyObject *type;
  std::string what;
};
[[noreturn]] void type_error(const std::string &what) { throw Refusal{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string &what) { throw Refusal{PyExc_ValueError, what}; }
struct PythonError {};  // an error a Python call already set

struct Arg {
  const at::Tensor &t;
  const char *name;
};

Arg tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
  return Arg{THPVariable_Unpack(o), name};
}
Arg typed(PyObject *o, const char *name, at::ScalarType type) {
  Arg a = tensor(o, name);
  if (a.t.scalar_type() != type)
    type_error(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(a.t.scalar_type()));
  return a;
}
// The 16-bit float type that the call's element tensors share.
at::ScalarType element_type(PyObject *o, const char *name) {
  const Arg a = tensor(o, name);
  const at::ScalarType type = a.t.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf)
    type_error(std::string(name) + " must be a bfloat16 or float16 CUDA tensor");
  return type;
}
int32_t dtype_code(at::ScalarType type) { return type == at::kHalf ? PA_FP16 : PA_BF16; }

std::string sizes(at::IntArrayRef s) {
  std::ostringstream out;
  out << s;
  return out.str();
}
void dims(const Arg &a, int64_t n) {
  if (a.t.dim() != n)
    value_error(std::string(a.name) + " must have " + std::to_string(n) + " dimensions, got shape " +
                sizes(a.t.sizes()));
}
void shape(const Arg &a, at::IntArrayRef want) {
  if (a.t.sizes() != want)
    value_error(std::string(a.name) + " must have shape " + sizes(want) + ", got " + sizes(a.t.sizes()));
}
void contiguous(const Arg &a) {
  if (!a.t.is_contiguous()) value_error(std::string(a.name) + " must be contiguous");
}
// Rows of [heads, D] contiguous elements; returns the token stride (of one token or none: a row).
int64_t token_stride(const Arg &a) {
  const int64_t heads = a.t.size(1), d = a.t.size(2);
  if ((a.t.stride(2) != 1 && d != 1) || (a.t.stride(1) != d && heads != 1))
    value_error(std::string("each token row of ") + a.name + " must be [heads, D] contiguous");
  return a.t.size(0) <= 1 ? heads * d : a.t.stride(0);
}
int32_t int32(int64_t v, const char *name) {
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}
int64_t integer(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}

// Every tensor on the current CUDA device, whose current stream the call uses when `o` is None.
template <int N>
void *stream_on_device(PyObject *o, const Arg (&args)[N]) {
  for (const Arg &a : args)
    if (!a.t.is_cuda()) type_error(std::string(a.name) + " must be a CUDA tensor");
  const auto device = c10::cuda::current_device();
  for (const Arg &a : args)
    if (a.t.device().index() != device)
      value_error(std::string(a.name) + " is on " + a.t.device().str() + "; the current device is cuda:" +
                  std::to_string(device));
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
  void *s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) throw PythonError{};
  return s;
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
    return nullptr;
  }
  try {
    return PyLong_FromLong(static_cast<long>(f()));
  } catch (const Refusal &r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const PythonError &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// Weights of a norm, or none.
const void *weights(PyObject *o, const char *name, at::ScalarType type, int64_t d, const Arg &fallback,
                    const at::Tensor *&seen) {
  seen = &fallback.t;
  if (o == Py_None) return nullptr;
  const Arg a = typed(o, name, type);
  shape(a, {d});
  contiguous(a);
  seen = &a.t;
  return a.t.data_ptr();
}

// norm_rope(q, key, q_weight, k_weight, eps, positions, cos_sin_cache, q_out, key_out, is_neox, stream)
PyObject *norm_rope(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> pa_status {
    const at::ScalarType type = element_type(v[0], "q");
    const Arg q = typed(v[0], "q", type), key = typed(v[1], "key", type);
    const Arg positions = typed(v[5], "positions", at::kLong), table = typed(v[6], "cos_sin_cache", at::kFloat);
    const Arg q_out = typed(v[7], "q_out", type), key_out = typed(v[8], "key_out", type);
    dims(q, 3);
    dims(key, 3);
    dims(table, 2);
    const int64_t T = q.t.size(0), H = q.t.size(1), D = q.t.size(2), Hkv = key.t.size(1);
    shape(key, {T, Hkv, D});
    shape(q_out, {T, H, D});
    shape(key_out, {T, Hkv, D});
    shape(positions, {T});
    const int64_t qs = token_stride(q), ks = token_stride(key), qos = token_stride(q_out), kos = token_stride(key_out);
    contiguous(positions);
    contiguous(table);
    const at::Tensor *wq, *wk;
    const void *qw = weights(v[2], "q_weight", type, D, q, wq), *kw = weights(v[3], "k_weight", type, D, q, wk);
    const float eps = static_cast<float>(number(v[4]));
    void *stream = stream_on_device(v[10], {q, key, positions, table, q_out, key_out, Arg{*wq, "q_weight"},
                                            Arg{*wk, "k_weight"}});
    return pa_norm_rope(q.t.data_ptr(), qs, key.t.data_ptr(), ks, qw, kw, eps,
                        static_cast<const int64_t *>(positions.t.data_ptr()),
                        static_cast<const float *>(table.t.data_ptr()), int32(table.t.size(0), "max_position"),
                        int32(table.t.size(1), "rotary_dim"), truth(v[9]), int32(T, "num_tokens"),
                        int32(H, "num_heads"), int32(Hkv, "num_kv_heads"), int32(D, "head_dim"), q_out.t.data_ptr(),
                        qos, key_out.t.data_ptr(), kos, dtype_code(type), stream);
  });
}

// norm_rope_cache(q, key, value, q_weight, k_weight, eps, key_cache, value_cache, slot_mapping, positions,
//                 cos_sin_cache, k_scale, v_scale, q_out, is_neox, stream); scales None: 16-bit caches
PyObject *norm_rope_cache(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> pa_status {
    const at::ScalarType type = element_type(v[0], "q");
    const bool kv8 = v[11] != Py_None;
    const at::ScalarType cache = kv8 ? at::kByte : type;
    const Arg q = typed(v[0], "q", type), key = typed(v[1], "key", type), value = typed(v[2], "value", type);
    const Arg kc = typed(v[6], "key_cache", cache), vc = typed(v[7], "value_cache", cache);
    const Arg slots = typed(v[8], "slot_mapping", at::kLong), positions = typed(v[9], "positions", at::kLong);
    const Arg table = typed(v[10], "cos_sin_cache", at::kFloat), q_out = typed(v[13], "q_out", type);
    dims(q, 3);
    dims(key, 3);
    dims(kc, 4);
    dims(table, 2);
    const int64_t T = q.t.size(0), H = q.t.size(1), D = q.t.size(2), Hkv = key.t.size(1);
    const int64_t nb = kc.t.size(0), bs = kc.t.size(1);
    shape(key, {T, Hkv, D});
    shape(value, {T, Hkv, D});
    shape(kc, {nb, bs, Hkv, D});
    shape(vc, {nb, bs, Hkv, D});
    shape(slots, {T});
    shape(positions, {T});
    shape(q_out, {T, H, D});
    const int64_t qs = token_stride(q), ks = token_stride(key), vs = token_stride(value), qos = token_stride(q_out);
    contiguous(kc);
    contiguous(vc);
    contiguous(slots);
    contiguous(positions);
    contiguous(table);
    const at::Tensor *wq, *wk;
    const void *qw = weights(v[3], "q_weight", type, D, q, wq), *kw = weights(v[4], "k_weight", type, D, q, wk);
    const float eps = static_cast<float>(number(v[5]));
    const float k_scale = kv8 ? static_cast<float>(number(v[11])) : 1.f;
    const float v_scale = kv8 ? static_cast<float>(number(v[12])) : 1.f;
    void *stream = stream_on_device(v[15], {q, key, value, kc, vc, slots, positions, table, q_out,
                                            Arg{*wq, "q_weight"}, Arg{*wk, "k_weight"}});
    const auto *sp = static_cast<const int64_t *>(slots.t.data_ptr());
    const auto *pp = static_cast<const int64_t *>(positions.t.data_ptr());
    const auto *tp = static_cast<const float *>(table.t.data_ptr());
    const int32_t max_position = int32(table.t.size(0), "max_position"), rot = int32(table.t.size(1), "rotary_dim");
    const int32_t t = int32(T, "num_tokens"), h = int32(H, "num_heads"), hkv = int32(Hkv, "num_kv_heads");
    const int32_t d = int32(D, "head_dim"), b = int32(bs, "block_size");
    if (kv8)
      return pa_norm_rope_reshape_and_cache_fp8(q.t.data_ptr(), qs, key.t.data_ptr(), value.t.data_ptr(), ks, vs, qw,
                                                kw, eps, kc.t.data_ptr(), vc.t.data_ptr(), sp, pp, tp, max_position,
                                                rot, truth(v[14]), t, h, hkv, d, b, nb, k_scale, v_scale,
                                                q_out.t.data_ptr(), qos, dtype_code(type), stream);
    return pa_norm_rope_reshape_and_cache(q.t.data_ptr(), qs, key.t.data_ptr(), value.t.data_ptr(), ks, vs, qw, kw,
                                          eps, kc.t.data_ptr(), vc.t.data_ptr(), sp, pp, tp, max_position, rot,
                                          truth(v[14]), t, h, hkv, d, b, nb, q_out.t.data_ptr(), qos,
                                          dtype_code(type), stream);
  });
}

// 8-bit caches with block scales and the lengths of a step.
struct BlockCache {
  Arg kc, vc, ks, vs, tables, lens, starts;
  int64_t nb, bs, hkv, d, b, m;
};
BlockCache block_cache(PyObject *const *v) {  // key_cache, value_cache, k_scales, v_scales, tables, lens, starts
  BlockCache c{typed(v[0], "key_cache", at::kByte),
               typed(v[1], "value_cache", at::kByte),
               typed(v[2], "k_scales", at::kFloat),
               typed(v[3], "v_scales", at::kFloat),
               typed(v[4], "block_tables", at::kInt),
               typed(v[5], "seq_lens", at::kInt),
               typed(v[6], "query_start_loc", at::kInt),
               0, 0, 0, 0, 0, 0};
  dims(c.kc, 4);
  dims(c.tables, 2);
  c.nb = c.kc.t.size(0);
  c.bs = c.kc.t.size(1);
  c.hkv = c.kc.t.size(2);
  c.d = c.kc.t.size(3);
  c.b = c.tables.t.size(0);
  c.m = c.tables.t.size(1);
  shape(c.vc, {c.nb, c.bs, c.hkv, c.d});
  shape(c.ks, {c.nb, c.hkv});
  shape(c.vs, {c.nb, c.hkv});
  shape(c.lens, {c.b});
  shape(c.starts, {c.b + 1});
  contiguous(c.kc);
  contiguous(c.vc);
  contiguous(c.ks);
  contiguous(c.vs);
  contiguous(c.tables);
  contiguous(c.lens);
  contiguous(c.starts);
  return c;
}

// block_scatter(key, value, key_cache, value_cache, k_scales, v_scales, block_tables, seq_lens, query_start_loc,
//               max_query_len, stream)
PyObject *block_scatter(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> pa_status {
    const at::ScalarType type = element_type(v[0], "key");
    const Arg key = typed(v[0], "key", type), value = typed(v[1], "value", type);
    const BlockCache c = block_cache(v + 2);
    dims(key, 3);
    const int64_t T = key.t.size(0);
    shape(key, {T, c.hkv, c.d});
    shape(value, {T, c.hkv, c.d});
    const int64_t ks = token_stride(key), vs = token_stride(value);
    const int32_t max_query_len = int32(integer(v[9]), "max_query_len");
    void *stream = stream_on_device(v[10], {key, value, c.kc, c.vc, c.ks, c.vs, c.tables, c.lens, c.starts});
    return pa_reshape_and_cache_fp8_block(
        key.t.data_ptr(), value.t.data_ptr(), ks, vs, c.kc.t.data_ptr(), c.vc.t.data_ptr(),
        static_cast<float *>(c.ks.t.data_ptr()), static_cast<float *>(c.vs.t.data_ptr()),
        static_cast<const int32_t *>(c.tables.t.data_ptr()), int32(c.m, "max_blocks_per_seq"),
        static_cast<const int32_t *>(c.lens.t.data_ptr()), static_cast<const int32_t *>(c.starts.t.data_ptr()),
        int32(c.b, "num_seqs"), int32(T, "total_q_tokens"), max_query_len, int32(c.hkv, "num_kv_heads"),
        int32(c.d, "head_dim"), int32(c.bs, "block_size"), c.nb, dtype_code(type), stream);
  });
}

// block_attention(q, key_cache, value_cache, k_scales, v_scales, block_tables, seq_lens, query_start_loc,
//                 max_query_len, max_seq_len, scale, out, workspace, stream)
PyObject *block_attention(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> pa_status {
    const at::ScalarType type = element_type(v[0], "q");
    const Arg q = typed(v[0], "q", type), out = typed(v[11], "out", type), workspace = tensor(v[12], "workspace");
    const BlockCache c = block_cache(v + 1);
    dims(q, 3);
    const int64_t T = q.t.size(0), H = q.t.size(1);
    shape(q, {T, H, c.d});
    shape(out, {T, H, c.d});
    const int64_t qs = token_stride(q);
    contiguous(out);
    contiguous(workspace);
    const int32_t max_query_len = int32(integer(v[8]), "max_query_len");
    const int32_t max_seq_len = int32(integer(v[9]), "max_seq_len");
    const float scale = static_cast<float>(number(v[10]));
    void *stream = stream_on_device(v[13], {q, out, workspace, c.kc, c.vc, c.ks, c.vs, c.tables, c.lens, c.starts});
    return pa_attention_varlen_fp8_block(
        q.t.data_ptr(), qs, c.kc.t.data_ptr(), c.vc.t.data_ptr(), static_cast<const float *>(c.ks.t.data_ptr()),
        static_cast<const float *>(c.vs.t.data_ptr()), static_cast<const int32_t *>(c.tables.t.data_ptr()),
        int32(c.m, "max_blocks_per_seq"), static_cast<const int32_t *>(c.lens.t.data_ptr()),
        static_cast<const int32_t *>(c.starts.t.data_ptr()), int32(c.b, "num_seqs"), int32(T, "total_q_tokens"),
        max_query_len, max_seq_len, int32(H, "num_heads"), int32(c.hkv, "num_kv_heads"), int32(c.d, "head_dim"),
        int32(c.bs, "block_size"), c.nb, scale, out.t.data_ptr(), workspace.t.data_ptr(), workspace.t.nbytes(),
        dtype_code(type), stream);
  });
}

// copy_block_scales(k_scales, v_scales, block_mapping, stream)
PyObject *copy_block_scales(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> pa_status {
    const Arg ks = typed(v[0], "k_scales", at::kFloat), vs = typed(v[1], "v_scales", at::kFloat);
    const Arg mapping = typed(v[2], "block_mapping", at::kLong);
    dims(ks, 2);
    dims(mapping, 2);
    const int64_t nb = ks.t.size(0), hkv = ks.t.size(1), pairs = mapping.t.size(0);
    shape(vs, {nb, hkv});
    shape(mapping, {pairs, 2});
    contiguous(ks);
    contiguous(vs);
    contiguous(mapping);
    void *stream = stream_on_device(v[3], {ks, vs, mapping});
    return pa_copy_block_scales(static_cast<float *>(ks.t.data_ptr()), static_cast<float *>(vs.t.data_ptr()),
                                static_cast<const int64_t *>(mapping.t.data_ptr()), int32(pairs, "num_pairs"),
                                int32(hkv, "num_kv_heads"), nb, stream);
  });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"norm_rope", fast(norm_rope), METH_FASTCALL, nullptr},
                         {"norm_rope_cache", fast(norm_rope_cache), METH_FASTCALL, nullptr},
                         {"block_scatter", fast(block_scatter), METH_FASTCALL, nullptr},
                         {"block_attention", fast(block_attention), METH_FASTCALL, nullptr},
                         {"copy_block_scales", fast(copy_block_scales), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
