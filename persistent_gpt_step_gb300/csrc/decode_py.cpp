// decode_py.cpp — the decode-step operators on torch tensors: argument checks,
// output memory and the call of the C ABI, as a CPython module for decode.py.
//
// One small decode step is a few microseconds of device time; looking at eight
// tensors from Python takes longer than that (append of one token: 17.7 us a call
// from Python through ctypes, 4.4 us here).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/gpt.h"

namespace {

// The library's entries and the binding's error class, set by init().
decltype(&gpt_kv_append) f_kv_append;
decltype(&gpt_decode_attention) f_decode_attention;
decltype(&gpt_decode_attention_workspace) f_workspace;
decltype(&gpt_next_token) f_next_token;
decltype(&gpt_last_error) f_last_error;
PyObject* g_error;

[[noreturn]] void raise(int code, const std::string& msg) {
  if (PyObject* e = PyObject_CallFunction(g_error, "is", code, msg.c_str())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}
template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  raise(GPT_ERR_INVALID_ARG, s.str());
}
void check(int rc) {
  if (rc != GPT_OK) raise(rc, f_last_error(nullptr));
}

const char* type_name(at::ScalarType t) {
  return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kInt ? "torch.int32" : c10::toString(t);
}

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

// The call's device, that of its first tensor and the current one, and its stream.
struct Place {
  c10::DeviceIndex device;
  cudaStream_t stream;
  std::optional<c10::cuda::CUDAStreamGuard> guard;  // memory for a given stream: the allocator hands it out in that stream's order

  Place(const at::Tensor& t, const char* name, PyObject* given_stream) {
    if (!t.is_cuda()) refuse(name, " must be a CUDA tensor");
    device = t.get_device();
    const int now = c10::cuda::current_device();
    if (device != now) refuse(name, " is on cuda:", (int)device, ", not the current device");
    if (!given(given_stream)) {
      stream = c10::cuda::getCurrentCUDAStream(device).stream();
      return;
    }
    PyObject* raw = PyObject_GetAttrString(given_stream, "cuda_stream");
    if (!raw) throw python_error();
    stream = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw python_error();
    if (stream != c10::cuda::getCurrentCUDAStream(device).stream())
      guard.emplace(c10::cuda::getStreamFromExternal(stream, device));
  }
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, device), std::nullopt));
  }
};

// A tensor of this type and shape on the device, its elements side by side.
const at::Tensor& expect(const Place& at, const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  if (t.scalar_type() != type) refuse(name, " must be ", type_name(type), ", got ", type_name(t.scalar_type()));
  if (!t.is_cuda() || t.get_device() != at.device) refuse(name, " is on ", t.device(), ", not on cuda:", (int)at.device);
  if (t.sizes() != shape) refuse(name, " has shape ", t.sizes(), ", expected ", shape);
  if (shape.back() > 1 && t.strides().back() != 1) refuse("the last dimension of ", name, " must be contiguous");
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse(name, " requires a gradient, which this operator does not have: call it under torch.no_grad()");
  return t;
}
const at::Tensor& expect(const Place& at, PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  return expect(at, tensor(o, name), name, type, shape);
}
// A tensor that the call has written: what autograd saved of it before no longer holds.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject* o) {
  if (given(o)) written(THPVariable_Unpack(o));
}
template <typename T>
T* data(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T>
T* data_or_null(const Place& at, PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  return given(o) ? data<T>(expect(at, o, name, type, shape)) : nullptr;
}
uint32_t* status_word(const Place& at, PyObject* o) { return data_or_null<uint32_t>(at, o, "status", at::kInt, {1}); }

// Stride of dimension i; 0 where there is one entry, whose stride says nothing.
int64_t stride(const at::Tensor& t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; }

int32_t type_code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return GPT_DTYPE_BF16;
  if (t.scalar_type() != at::kFloat) refuse(name, " must be torch.float32 or torch.bfloat16, got ", type_name(t.scalar_type()));
  return GPT_DTYPE_FP32;
}

int32_t to_int(int64_t x, const char* what) {
  if (x > INT32_MAX || x < INT32_MIN) refuse(what, " does not fit in 32 bits");
  return (int32_t)x;
}

gpt_paged_cache cache_of(const Place& at, PyObject* k_, PyObject* v_, PyObject* table_) {
  const at::Tensor &k = tensor(k_, "k_cache"), &v = tensor(v_, "v_cache"), &table = tensor(table_, "page_table");
  if (k.dim() != 4) refuse("k_cache must be [pages, page size, heads, head size]");
  if (table.dim() != 2) refuse("page_table must be [sequences, pages]");
  gpt_paged_cache c = {};
  c.dtype = type_code(k, "k_cache");
  c.k = data<void>(expect(at, k, "k_cache", k.scalar_type(), k.sizes()));
  c.v = data<void>(expect(at, v, "v_cache", k.scalar_type(), k.sizes()));
  c.page_table = data<int32_t>(expect(at, table, "page_table", at::kInt, table.sizes()));
  c.page_stride = stride(k, 0), c.slot_stride = stride(k, 1), c.head_stride = stride(k, 2);
  for (int i = 0; i < 3; ++i)
    if (stride(v, i) != stride(k, i)) refuse("k_cache and v_cache must have the same strides");
  c.table_stride = table.stride(0);
  c.n_pages = to_int(k.size(0), "the number of pages"), c.page_size = to_int(k.size(1), "page size");
  c.n_kv_head = to_int(k.size(2), "the number of heads"), c.head_dim = to_int(k.size(3), "head size");
  c.n_seq = to_int(table.size(0), "the number of sequences"), c.max_pages = to_int(table.size(1), "the width of page_table");
  return c;
}

#define ARGS(n) \
  if (count != (n)) { PyErr_SetString(PyExc_TypeError, "wrong number of arguments"); throw python_error(); }

// k, v, k_cache, v_cache, page_table, positions, seq, q, rope_dims, rope_base, q_out, status, stream
PyObject* kv_append(PyObject*, PyObject* const* o, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  ARGS(13)
  const at::Tensor &k = tensor(o[0], "k"), &v = tensor(o[1], "v");
  const Place at(k, "k", o[12]);
  const gpt_paged_cache c = cache_of(at, o[2], o[3], o[4]);
  const at::ScalarType type = THPVariable_Unpack(o[2]).scalar_type();
  if (k.dim() != 3) refuse("k must be [tokens, heads, head size]");
  const int64_t n = k.size(0);
  gpt_kv_append_args a = {};
  a.n_tokens = to_int(n, "the number of tokens");
  a.k = data<void>(expect(at, k, "k", type, {n, c.n_kv_head, c.head_dim}));
  a.v = data<void>(expect(at, v, "v", type, {n, c.n_kv_head, c.head_dim}));
  a.k_row = stride(k, 0), a.k_head = stride(k, 1), a.v_row = stride(v, 0), a.v_head = stride(v, 1);
  a.positions = data<int32_t>(expect(at, o[5], "positions", at::kInt, {n}));
  a.seq = data_or_null<int32_t>(at, o[6], "seq", at::kInt, {n});
  a.status = status_word(at, o[11]);
  const int64_t rope_dims = PyLong_AsLongLong(o[8]);
  if (PyErr_Occurred()) throw python_error();
  a.rope_dims = to_int(rope_dims, "rope_dims");
  a.rope_base = PyFloat_AsDouble(o[9]);
  if (PyErr_Occurred()) throw python_error();
  at::Tensor q_out;
  if (given(o[7])) {
    const at::Tensor& q = tensor(o[7], "q");
    if (q.dim() != 3) refuse("q must be [tokens, heads, head size]");
    a.n_head = to_int(q.size(1), "the number of heads");
    a.q = data<void>(expect(at, q, "q", type, {n, q.size(1), c.head_dim}));
    q_out = given(o[10]) ? tensor(o[10], "q_out") : at.empty({n, q.size(1), c.head_dim}, type);
    a.q_out = data<void>(expect(at, q_out, "q_out", type, {n, q.size(1), c.head_dim}));
    a.q_row = stride(q, 0), a.q_head = stride(q, 1), a.qo_row = stride(q_out, 0), a.qo_head = stride(q_out, 1);
  } else if (given(o[10])) {
    refuse("q_out goes with q");
  }
  check(f_kv_append(&c, &a, at.stream));
  written(o[2]), written(o[3]), written(o[10]), written(o[11]);
  if (!q_out.defined()) Py_RETURN_NONE;
  if (given(o[10])) { Py_INCREF(o[10]); return o[10]; }
  return THPVariable_Wrap(std::move(q_out));
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, page_table, lens, scale, out, status, stream
PyObject* decode_attention(PyObject*, PyObject* const* o, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  ARGS(9)
  const at::Tensor& q = tensor(o[0], "q");
  const Place at(q, "q", o[8]);
  const gpt_paged_cache c = cache_of(at, o[1], o[2], o[3]);
  const at::ScalarType type = THPVariable_Unpack(o[1]).scalar_type();
  if (q.dim() != 3) refuse("q must be [sequences, heads, head size]");
  const int64_t n = c.n_seq, heads = q.size(1), dim = c.head_dim;
  gpt_decode_attention_args a = {};
  a.n_head = to_int(heads, "the number of heads");
  a.q = data<void>(expect(at, q, "q", type, {n, heads, dim}));
  const at::Tensor out = given(o[6]) ? tensor(o[6], "out") : at.empty({n, heads, dim}, type);
  a.out = data<void>(expect(at, out, "out", type, {n, heads, dim}));
  a.q_row = stride(q, 0), a.q_head = stride(q, 1), a.out_row = stride(out, 0), a.out_head = stride(out, 1);
  a.lens = data<int32_t>(expect(at, o[4], "lens", at::kInt, {n}));
  a.status = status_word(at, o[7]);
  a.scale = (float)(given(o[5]) ? PyFloat_AsDouble(o[5]) : 1.0 / std::sqrt((double)dim));
  if (PyErr_Occurred()) throw python_error();
  at::Tensor lse = at.empty({n, heads}, at::kFloat), scratch;
  a.lse = data<float>(lse);
  a.workspace_bytes = f_workspace(&c, a.n_head);
  if (a.workspace_bytes) {
    scratch = at.empty({(int64_t)a.workspace_bytes}, at::kByte);
    a.workspace = scratch.data_ptr();
  }
  check(f_decode_attention(&c, &a, at.stream));
  written(o[6]), written(o[7]);
  PyObject* result = PyTuple_New(2);
  if (!result) throw python_error();
  if (given(o[6])) { Py_INCREF(o[6]); PyTuple_SET_ITEM(result, 0, o[6]); }
  else PyTuple_SET_ITEM(result, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(result, 1, THPVariable_Wrap(std::move(lse)));
  return result;
  END_HANDLE_TH_ERRORS
}

// logits, history, history_lens, prompt_lens, repetition, presence, frequency, bias_ids, bias_values, allowed, out, status, stream
PyObject* next_token(PyObject*, PyObject* const* o, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  ARGS(13)
  const at::Tensor& logits = tensor(o[0], "logits");
  const Place at(logits, "logits", o[12]);
  if (logits.dim() != 2) refuse("logits must be [rows, vocab]");
  const int64_t rows = logits.size(0), vocab = logits.size(1);
  gpt_next_token_args a = {};
  a.rows = to_int(rows, "the number of rows"), a.vocab = to_int(vocab, "vocab");
  a.dtype = type_code(logits, "logits");
  a.logits = data<void>(expect(at, logits, "logits", logits.scalar_type(), {rows, vocab}));
  a.logits_stride = logits.stride(0);
  if (given(o[1])) {
    const at::Tensor& history = tensor(o[1], "history");
    if (history.dim() != 2) refuse("history must be [rows, tokens]");
    a.max_history = to_int(history.size(1), "the width of history");
    a.history = data<int32_t>(expect(at, history, "history", at::kInt, {rows, history.size(1)}));
    a.history_stride = history.stride(0);
    const int32_t* lens = data_or_null<int32_t>(at, o[2], "history_lens", at::kInt, {rows});
    const int32_t* prompts = data_or_null<int32_t>(at, o[3], "prompt_lens", at::kInt, {rows});
    if (a.max_history) a.history_lens = lens, a.prompt_lens = prompts;  // a history of no columns has no memory
  } else if (given(o[2]) || given(o[3])) {
    refuse("history_lens and prompt_lens go with history");
  }
  a.repetition = data_or_null<float>(at, o[4], "repetition", at::kFloat, {rows});
  a.presence = data_or_null<float>(at, o[5], "presence", at::kFloat, {rows});
  a.frequency = data_or_null<float>(at, o[6], "frequency", at::kFloat, {rows});
  if (given(o[7]) != given(o[8])) refuse("bias_ids and bias_values go together");
  if (given(o[7])) {
    const at::Tensor &ids = tensor(o[7], "bias_ids"), &values = tensor(o[8], "bias_values");
    if (ids.dim() != 2) refuse("bias_ids must be [rows, entries]");
    a.n_bias = to_int(ids.size(1), "the width of bias_ids");
    a.bias_ids = data<int32_t>(expect(at, ids, "bias_ids", at::kInt, {rows, ids.size(1)}));
    a.bias_values = data<float>(expect(at, values, "bias_values", at::kFloat, {rows, ids.size(1)}));
    a.bias_stride = ids.stride(0);
    if (stride(ids, 0) != stride(values, 0)) refuse("bias_ids and bias_values must have the same strides");
  }
  if (given(o[9])) {
    const at::Tensor& allowed = expect(at, o[9], "allowed", at::kInt, {rows, (vocab + 31) / 32});
    a.allowed = data<uint32_t>(allowed), a.allowed_stride = allowed.stride(0);
  }
  a.status = status_word(at, o[11]);
  const at::Tensor out = given(o[10]) ? tensor(o[10], "out") : at.empty({rows, vocab}, at::kFloat);
  a.out = data<float>(expect(at, out, "out", at::kFloat, {rows, vocab}));
  a.out_stride = out.stride(0);
  at::Tensor token = at.empty({rows}, at::kInt), lse = at.empty({rows}, at::kFloat);
  a.token = data<int32_t>(token), a.lse = data<float>(lse);
  check(f_next_token(&a, at.stream));
  written(o[10]), written(o[11]);
  PyObject* result = PyTuple_New(3);
  if (!result) throw python_error();
  PyTuple_SET_ITEM(result, 0, THPVariable_Wrap(std::move(token)));
  if (given(o[10])) { Py_INCREF(o[10]); PyTuple_SET_ITEM(result, 1, o[10]); }
  else PyTuple_SET_ITEM(result, 1, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(result, 2, THPVariable_Wrap(std::move(lse)));
  return result;
  END_HANDLE_TH_ERRORS
}

// Addresses of gpt_kv_append, gpt_decode_attention, gpt_decode_attention_workspace, gpt_next_token, gpt_last_error; GptError
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long a, b, c, d, e;
  PyObject* error;
  if (!PyArg_ParseTuple(args, "KKKKKO", &a, &b, &c, &d, &e, &error)) return nullptr;
  f_kv_append = reinterpret_cast<decltype(f_kv_append)>(a);
  f_decode_attention = reinterpret_cast<decltype(f_decode_attention)>(b);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(c);
  f_next_token = reinterpret_cast<decltype(f_next_token)>(d);
  f_last_error = reinterpret_cast<decltype(f_last_error)>(e);
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"decode_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_attention)), METH_FASTCALL, nullptr},
    {"next_token", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(next_token)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() { return PyModule_Create(&module); }
