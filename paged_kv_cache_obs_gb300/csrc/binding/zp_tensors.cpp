// zp_tensors.cpp — tensors to C structs for the calls that a step makes once per layer.
//
// The kernels behind these calls take 4 to 50 us, and reading a tensor's address, sizes, strides, type
// and device from Python costs about 1 us a tensor: with the checks below, 8 us for rotary positions
// and 15 us for a cache write were spent on the host.  Here the same takes the time of the launch.
// This module only checks and marshals: it calls the entry points of the library that the Python
// binding has loaded, whose addresses it is given, and knows nothing of their kernels.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <stdexcept>
#include <string>

#include "zipage.h"

namespace {

struct PythonError {};  // one is set

struct Library {
  decltype(&zp_rope_apply) rope_apply;
  decltype(&zp_kv8_append) kv8_append;
  decltype(&zp_kv8_pack_blocks) kv8_pack_blocks;
  decltype(&zp_kv8_unpack_blocks) kv8_unpack_blocks;
  decltype(&zp_kv8_decode_attn) kv8_decode_attn;
  decltype(&zp_paged_window_attn) paged_window_attn;
  decltype(&zp_rope_apply_axes) rope_apply_axes;
  decltype(&zp_step_slots_held) step_slots_held;
  decltype(&zp_kv_append) kv_append;
  decltype(&zp_prompt_attn) prompt_attn;
  decltype(&zp_kv8_window_attn) kv8_window_attn;
} lib;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) refuse("expected a tensor");
  return THPVariable_Unpack(o);
}
int device_of(const at::Tensor& t) { return t.is_cuda() ? t.device().index() : -1; }

int32_t i32(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v < INT_MIN || v > INT_MAX) refuse("expected 32-bit numbers");
  return static_cast<int32_t>(v);
}
int64_t i64(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
template <class T>
T* address(PyObject* o) {
  void* const p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw PythonError{};
  return static_cast<T*>(p);
}

// bf16 rows [tokens][heads][head_dim] with any token and head strides.
zp_rows rows(PyObject* o, int dev, int64_t tokens, int64_t heads, int64_t d) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != d || t.stride(2) != 1 ||
      t.scalar_type() != at::kBFloat16 || device_of(t) != dev)
    refuse("expected bf16 rows [" + std::to_string(tokens) + ", " + std::to_string(heads) + ", " + std::to_string(d) +
           "] with a contiguous last dimension, all tensors on one device");
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}
// int32 of n entries or more, one number each (or one row of a table each).
const int32_t* entries(PyObject* o, int dev, int64_t n, bool rows = false) {
  const at::Tensor& t = tensor(o);
  if (t.dim() < 1 || t.size(0) < n || !(rows ? t.dim() == 2 : t.numel() == t.size(0)) || t.scalar_type() != at::kInt ||
      !t.is_contiguous() || device_of(t) != dev)
    refuse("expected a contiguous int32 " + (rows ? "table [" + std::to_string(n) + ", max_blocks]" : "tensor of " + std::to_string(n) + " entries") +
           ", all tensors on one device");
  return static_cast<const int32_t*>(t.data_ptr());
}
const int32_t* table(PyObject* o, int dev, int64_t n, int32_t& max_blocks) {
  const int32_t* const p = entries(o, dev, n, true);
  const at::Tensor& t = tensor(o);
  if (t.size(1) > INT_MAX) refuse("expected a block table [requests, max_blocks]");
  max_blocks = static_cast<int32_t>(t.size(1));
  return p;
}
int32_t count(PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o);
  if (t.dim() < 1 || t.size(0) > INT_MAX) refuse(std::string("expected ") + what);
  return static_cast<int32_t>(t.size(0));
}

zp_kv_pool pool(PyObject* o, int dev, const zp_params& p) {
  const at::Tensor& t = tensor(o);
  if (t.dim() < 2 || t.scalar_type() != at::kBFloat16 || !t.is_contiguous() || device_of(t) != dev ||
      t.numel() != p.num_layers * t.size(1) * 2 * p.num_kv_heads * p.block_size * p.head_dim)
    refuse("expected a contiguous bf16 pool [num_layers, blocks, 2, num_kv_heads, block_size, head_dim]");
  return {t.data_ptr(), t.size(1)};
}
zp_kv8_pool kv8(PyObject* c, PyObject* s, int dev, const zp_params& p) {
  const at::Tensor &codes = tensor(c), &scales = tensor(s);
  // E4M3, or bytes that hold its codes; other types of one byte stand for other values
  const bool type = codes.scalar_type() == at::kFloat8_e4m3fn || codes.scalar_type() == at::kByte || codes.scalar_type() == at::kChar;
  if (codes.dim() < 2 || !type || scales.scalar_type() != at::kFloat || !codes.is_contiguous() ||
      !scales.is_contiguous() || device_of(scales) != dev ||
      scales.numel() != p.num_layers * codes.size(1) * 2 * p.num_kv_heads ||
      codes.numel() != scales.numel() * p.block_size * p.head_dim)
    refuse("expected contiguous codes [num_layers, blocks, 2, num_kv_heads, block_size, head_dim] in E4M3 (float8_e4m3fn, uint8 or int8) and fp32 "
           "scales [num_layers, blocks, 2, num_kv_heads], all tensors on one device");
  return {codes.data_ptr(), static_cast<float*>(scales.data_ptr()), codes.size(1)};
}
void* workspace(PyObject* o, int dev, size_t& bytes) {
  const at::Tensor& t = tensor(o);
  if (!t.is_contiguous() || device_of(t) != dev) refuse("expected a contiguous workspace, all tensors on one device");
  bytes = t.nbytes();
  return t.data_ptr();
}
// The stream to launch on: the given one, or the current one of the tensors' device, which has to be
// the current device (the library launches there).
zp_stream stream(PyObject* o, int dev) {
  if (dev < 0 || dev != c10::cuda::current_device()) refuse("the tensors have to be on the current CUDA device");
  if (o != Py_None) return address<void>(o);
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

// The call itself, without the interpreter's lock.
template <class F>
PyObject* call(F f) {
  zp_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

// The rows of q and k (either may be None) and where their results go.
struct Turned {
  zp_rows r[4];
  int32_t heads[2] = {0, 0};
  bool have[2];
  Turned(PyObject* const* in, PyObject* const* out, int dev, int32_t T, int32_t d) {
    for (int i = 0; i < 2; ++i) {
      have[i] = in[i] != Py_None;
      if (!have[i]) continue;
      const at::Tensor& x = tensor(in[i]);
      if (x.dim() != 3 || x.size(1) > INT_MAX) refuse("expected rows [tokens, heads, head_dim]");
      heads[i] = static_cast<int32_t>(x.size(1));
      r[2 * i] = rows(in[i], dev, T, heads[i], d);
      r[2 * i + 1] = out[i] == Py_None ? r[2 * i] : rows(out[i], dev, T, heads[i], d);
    }
  }
  const zp_rows* at(int i) const { return have[i / 2] ? &r[i] : nullptr; }
};

// rope, q, k, positions, q_out, k_out, stream
PyObject* rope_apply(PyObject* const* a) {
  const zp_rope* const rope = address<const zp_rope>(a[0]);
  const int dev = device_of(tensor(a[3]));
  const int32_t T = count(a[3], "positions [tokens]");
  const Turned x(a + 1, a + 4, dev, T, rope->head_dim);
  const int32_t* const pos = entries(a[3], dev, T);
  const zp_stream st = stream(a[6], dev);
  return call([&] { return lib.rope_apply(rope, x.at(0), x.at(1), x.heads[0], x.at(2), x.at(3), x.heads[1], pos, T, st); });
}

// axes, q, k, positions, q_out, k_out, stream
PyObject* rope_apply_axes(PyObject* const* a) {
  const zp_rope_axes* const axes = address<const zp_rope_axes>(a[0]);
  const at::Tensor& p = tensor(a[3]);
  const int dev = device_of(p);
  // a row of each axis; the same row may stand for all
  if (p.dim() != 2 || p.size(0) != axes->num_axes || p.size(1) > INT_MAX || p.scalar_type() != at::kInt || (p.size(1) > 1 && p.stride(1) != 1))
    refuse("expected int32 positions [" + std::to_string(axes->num_axes) + ", tokens] with contiguous rows");
  const int32_t T = static_cast<int32_t>(p.size(1));
  const Turned x(a + 1, a + 4, dev, T, axes->rope.head_dim);
  const zp_stream st = stream(a[6], dev);
  const int32_t* const pos = static_cast<const int32_t*>(p.data_ptr());
  const int64_t step = p.size(0) > 1 ? p.stride(0) : 0;
  return call([&] {
    return lib.rope_apply_axes(axes, x.at(0), x.at(1), x.heads[0], x.at(2), x.at(3), x.heads[1], pos, step, T, st);
  });
}

// cached, new_tokens, first_pos, free_ids, free_at, num_blocks, block_tables, token_start, seq_lens, positions, slots, params,
// workspace, stream, held_blocks
PyObject* step_slots_held(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[11]);
  const int dev = device_of(tensor(a[10]));
  const int32_t B = count(a[0], "cached [requests]"), T = count(a[10], "slots [tokens]"), free = count(a[3], "free block ids");
  const auto optional = [&](PyObject* o, int64_t n) { return o == Py_None ? nullptr : entries(o, dev, n); };
  const int32_t *const cached = entries(a[0], dev, B), *const more = entries(a[1], dev, B), *const first = optional(a[2], B);
  const int32_t *const ids = entries(a[3], dev, free), *const at = optional(a[4], 1);
  int32_t max_blocks;
  const int32_t* const tables = table(a[6], dev, B, max_blocks);
  const int32_t *const start = entries(a[7], dev, static_cast<int64_t>(B) + 1), *const lens = entries(a[8], dev, B);
  const int32_t *const pos = optional(a[9], T), *const slots = entries(a[10], dev, T), *const held = optional(a[14], B);
  const int64_t blocks = i64(a[5]);
  size_t bytes;
  void* const ws = workspace(a[12], dev, bytes);
  const zp_stream st = stream(a[13], dev);
  const auto out = [](const int32_t* x) { return const_cast<int32_t*>(x); };
  return call([&] {
    return lib.step_slots_held(cached, more, first, out(held), B, ids, free, out(at), blocks, out(tables), max_blocks, out(start), out(lens), out(pos),
                          out(slots), T, &p, ws, bytes, st);
  });
}

// pool, layer, k, v, slots, params, workspace, stream
PyObject* kv_append(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[5]);
  const int dev = device_of(tensor(a[0]));
  const zp_kv_pool to = pool(a[0], dev, p);
  const int32_t layer = i32(a[1]), T = count(a[2], "keys [tokens, heads, head_dim]");
  const zp_rows k = rows(a[2], dev, T, p.num_kv_heads, p.head_dim), v = rows(a[3], dev, T, p.num_kv_heads, p.head_dim);
  const int32_t* const slots = entries(a[4], dev, T);
  size_t bytes;
  void* const ws = workspace(a[6], dev, bytes);
  const zp_stream st = stream(a[7], dev);
  return call([&] { return lib.kv_append(&to, layer, &k, &v, slots, T, &p, ws, bytes, st); });
}

// codes, scales, layer, k, v, token_start, cached, block_tables, params, workspace, stream
PyObject* kv8_append(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[8]);
  const int dev = device_of(tensor(a[0]));
  const zp_kv8_pool to = kv8(a[0], a[1], dev, p);
  const int32_t layer = i32(a[2]), T = count(a[3], "keys [tokens, heads, head_dim]"), B = count(a[6], "cached [requests]");
  const zp_rows k = rows(a[3], dev, T, p.num_kv_heads, p.head_dim), v = rows(a[4], dev, T, p.num_kv_heads, p.head_dim);
  const int32_t* const start = entries(a[5], dev, static_cast<int64_t>(B) + 1);
  const int32_t* const cached = entries(a[6], dev, B);
  int32_t max_blocks;
  const int32_t* const tables = table(a[7], dev, B, max_blocks);
  size_t bytes;
  void* const ws = workspace(a[9], dev, bytes);
  const zp_stream st = stream(a[10], dev);
  return call([&] { return lib.kv8_append(&to, layer, &k, &v, T, start, cached, B, tables, max_blocks, &p, ws, bytes, st); });
}

// pool, src_ids, codes, scales, dst_ids, fill, layer_begin, layer_count, params, workspace, stream
PyObject* kv8_pack_blocks(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[8]);
  const int dev = device_of(tensor(a[2]));
  const zp_kv_pool from = pool(a[0], dev, p);
  const zp_kv8_pool to = kv8(a[2], a[3], dev, p);
  const int32_t n = count(a[1], "block ids");
  const int32_t *const src = entries(a[1], dev, n), *const dst = entries(a[4], dev, n);
  const int32_t* const fill = a[5] == Py_None ? nullptr : entries(a[5], dev, n);
  const int32_t begin = i32(a[6]), layers = i32(a[7]);
  size_t bytes;
  void* const ws = workspace(a[9], dev, bytes);
  const zp_stream st = stream(a[10], dev);
  return call([&] { return lib.kv8_pack_blocks(&from, src, fill, &to, dst, n, begin, layers, &p, ws, bytes, st); });
}

// codes, scales, src_ids, pool, dst_ids, layer_begin, layer_count, params, workspace, stream
PyObject* kv8_unpack_blocks(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[7]);
  const int dev = device_of(tensor(a[0]));
  const zp_kv8_pool from = kv8(a[0], a[1], dev, p);
  const zp_kv_pool to = pool(a[3], dev, p);
  const int32_t n = count(a[2], "block ids");
  const int32_t *const src = entries(a[2], dev, n), *const dst = entries(a[4], dev, n);
  const int32_t begin = i32(a[5]), layers = i32(a[6]);
  size_t bytes;
  void* const ws = workspace(a[8], dev, bytes);
  const zp_stream st = stream(a[9], dev);
  return call([&] { return lib.kv8_unpack_blocks(&from, src, &to, dst, n, begin, layers, &p, ws, bytes, st); });
}

// codes, scales, layer, q, block_tables, seq_lens, out, params, workspace, window, sinks, stream
PyObject* kv8_decode_attn(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[7]);
  const int dev = device_of(tensor(a[0]));
  const zp_kv8_pool from = kv8(a[0], a[1], dev, p);
  const int32_t layer = i32(a[2]), B = count(a[3], "queries [requests, heads, head_dim]");
  const zp_rows q = rows(a[3], dev, B, p.num_q_heads, p.head_dim), out = rows(a[6], dev, B, p.num_q_heads, p.head_dim);
  int32_t max_blocks;
  const int32_t* const tables = table(a[4], dev, B, max_blocks);
  const int32_t* const lens = entries(a[5], dev, B);
  size_t bytes;
  void* const ws = workspace(a[8], dev, bytes);
  const int32_t window = i32(a[9]), sinks = i32(a[10]);
  const zp_stream st = stream(a[11], dev);
  return call([&] {
    return lib.kv8_decode_attn(&from, layer, &q, tables, lens, B, max_blocks, window, sinks, &out, &p, ws, bytes, st);
  });
}

// pool, layer, q, q_start, block_tables, seq_lens, out, params, workspace, window, sinks, max_q, stream
PyObject* paged_window_attn(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[7]);
  const int dev = device_of(tensor(a[0]));
  const zp_kv_pool from = pool(a[0], dev, p);
  const int32_t layer = i32(a[1]), T = count(a[2], "queries [tokens, heads, head_dim]"), B = count(a[5], "lengths [requests]");
  const zp_rows q = rows(a[2], dev, T, p.num_q_heads, p.head_dim), out = rows(a[6], dev, T, p.num_q_heads, p.head_dim);
  const int32_t* const start = entries(a[3], dev, static_cast<int64_t>(B) + 1);
  int32_t max_blocks;
  const int32_t* const tables = table(a[4], dev, B, max_blocks);
  const int32_t* const lens = entries(a[5], dev, B);
  size_t bytes;
  void* const ws = workspace(a[8], dev, bytes);
  const int32_t window = i32(a[9]), sinks = i32(a[10]), max_q = i32(a[11]);
  const zp_stream st = stream(a[12], dev);
  return call([&] {
    return lib.paged_window_attn(&from, layer, &q, start, T, max_q, tables, lens, B, max_blocks, window, sinks, &out, &p, ws,
                                 bytes, st);
  });
}

// codes, scales, layer, q, q_start, block_tables, seq_lens, out, params, workspace, window, sinks, max_q, stream
PyObject* kv8_window_attn(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[8]);
  const int dev = device_of(tensor(a[0]));
  const zp_kv8_pool from = kv8(a[0], a[1], dev, p);
  const int32_t layer = i32(a[2]), T = count(a[3], "queries [tokens, heads, head_dim]"), B = count(a[6], "lengths [requests]");
  const zp_rows q = rows(a[3], dev, T, p.num_q_heads, p.head_dim), out = rows(a[7], dev, T, p.num_q_heads, p.head_dim);
  const int32_t* const start = entries(a[4], dev, static_cast<int64_t>(B) + 1);
  int32_t max_blocks;
  const int32_t* const tables = table(a[5], dev, B, max_blocks);
  const int32_t* const lens = entries(a[6], dev, B);
  size_t bytes;
  void* const ws = workspace(a[9], dev, bytes);
  const int32_t window = i32(a[10]), sinks = i32(a[11]), max_q = i32(a[12]);
  const zp_stream st = stream(a[13], dev);
  return call([&] {
    return lib.kv8_window_attn(&from, layer, &q, start, T, max_q, tables, lens, B, max_blocks, window, sinks, &out, &p, ws, bytes, st);
  });
}

// q, k, v, token_start, out, params, workspace, max_len, window, sinks, stream
PyObject* prompt_attn(PyObject* const* a) {
  const zp_params& p = *address<const zp_params>(a[5]);
  const int dev = device_of(tensor(a[0]));
  const int32_t T = count(a[0], "queries [tokens, heads, head_dim]"), n = count(a[3], "token_start [prompts + 1]");
  if (n < 1) refuse("expected token_start [prompts + 1]");
  const zp_rows q = rows(a[0], dev, T, p.num_q_heads, p.head_dim), out = rows(a[4], dev, T, p.num_q_heads, p.head_dim);
  const zp_rows k = rows(a[1], dev, T, p.num_kv_heads, p.head_dim), v = rows(a[2], dev, T, p.num_kv_heads, p.head_dim);
  const int32_t* const start = entries(a[3], dev, n);
  size_t bytes;
  void* const ws = workspace(a[6], dev, bytes);
  const int32_t max_len = i32(a[7]), window = i32(a[8]), sinks = i32(a[9]);
  const zp_stream st = stream(a[10], dev);
  return call([&] { return lib.prompt_attn(&q, &k, &v, start, T, n - 1, max_len, window, sinks, &out, &p, ws, bytes, st); });
}

// The addresses of the library's entry points, in the order of Library.
PyObject* bind(PyObject* const* a) {
  lib.rope_apply = reinterpret_cast<decltype(lib.rope_apply)>(address<void>(a[0]));
  lib.kv8_append = reinterpret_cast<decltype(lib.kv8_append)>(address<void>(a[1]));
  lib.kv8_pack_blocks = reinterpret_cast<decltype(lib.kv8_pack_blocks)>(address<void>(a[2]));
  lib.kv8_unpack_blocks = reinterpret_cast<decltype(lib.kv8_unpack_blocks)>(address<void>(a[3]));
  lib.kv8_decode_attn = reinterpret_cast<decltype(lib.kv8_decode_attn)>(address<void>(a[4]));
  lib.paged_window_attn = reinterpret_cast<decltype(lib.paged_window_attn)>(address<void>(a[5]));
  lib.rope_apply_axes = reinterpret_cast<decltype(lib.rope_apply_axes)>(address<void>(a[6]));
  lib.step_slots_held = reinterpret_cast<decltype(lib.step_slots_held)>(address<void>(a[7]));
  lib.kv_append = reinterpret_cast<decltype(lib.kv_append)>(address<void>(a[8]));
  lib.prompt_attn = reinterpret_cast<decltype(lib.prompt_attn)>(address<void>(a[9]));
  lib.kv8_window_attn = reinterpret_cast<decltype(lib.kv8_window_attn)>(address<void>(a[10]));
  Py_RETURN_NONE;
}

// No C++ exception passes into the interpreter.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %d arguments", N);
  try {
    return F(a);
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
constexpr PyMethodDef def(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {def<bind, 11>("bind"),
                         def<rope_apply, 7>("rope_apply"),
                         def<kv8_append, 11>("kv8_append"),
                         def<kv8_pack_blocks, 11>("kv8_pack_blocks"),
                         def<kv8_unpack_blocks, 10>("kv8_unpack_blocks"),
                         def<kv8_decode_attn, 12>("kv8_decode_attn"),
                         def<paged_window_attn, 13>("paged_window_attn"),
                         def<rope_apply_axes, 7>("rope_apply_axes"),
                         def<step_slots_held, 15>("step_slots_held"),
                         def<kv_append, 8>("kv_append"),
                         def<prompt_attn, 11>("prompt_attn"),
                         def<kv8_window_attn, 14>("kv8_window_attn"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "zp_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_zp_tensors() { return PyModule_Create(&module_def); }
