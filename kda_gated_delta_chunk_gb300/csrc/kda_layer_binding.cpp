// Marshalling of the full-attention layer's usual calls in C++: on small calls the checks and
// allocations of the Python binding take longer than the kernels.  A call that is usual -- plain
// tensors of the right types and shapes on the current device, caches and indexes contiguous,
// outputs left to the call, the current stream -- is checked, given its outputs and passed to the C
// entry point here.  Anything else returns None without having done anything, and the Python
// binding, which accepts more and names what is wrong, takes the call.
#include <Python.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kda.h"

namespace {

using at::ScalarType;
using at::Tensor;

decltype(&kda_add_rms_norm) norm_entry;
decltype(&kda_rope_append) append_entry;
decltype(&kda_cached_attention) attention_entry;

// (the entry points launch on the current device)
bool here(int64_t dev) { return dev == c10::cuda::current_device(); }

// The tensor behind an argument; null for anything but a plain one.
const Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const Tensor& t, int64_t dev, ScalarType type) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type;
}
bool dense(const Tensor* t, int64_t dev, ScalarType type, at::IntArrayRef sizes) {
  return t && on(*t, dev, type) && t->sizes() == sizes && t->is_contiguous();
}
// All dimensions but the first dense; `row`: the stride of the first.
bool rows(const Tensor* t, int64_t dev, ScalarType type, at::IntArrayRef sizes, int64_t* row) {
  if (!t || !on(*t, dev, type) || t->sizes() != sizes) return false;
  int64_t inner = 1;
  for (int64_t d = t->dim() - 1; d >= 1; --d) {
    if (t->stride(d) != inner && t->size(d) > 1) return false;
    inner *= t->size(d);
  }
  *row = t->size(0) != 1 ? t->stride(0) : t->numel();
  return true;
}
bool number(PyObject* o, float* x) {
  const double d = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : PyLong_Check(o) ? PyLong_AsDouble(o) : NAN;
  *x = (float)d;
  return !(PyErr_Occurred() ? (PyErr_Clear(), true) : false) && d == d;
}
bool integer(PyObject* o, int32_t* x) {
  int over = 0;
  const long v = PyLong_Check(o) ? PyLong_AsLongAndOverflow(o, &over) : LONG_MAX;
  *x = (int32_t)v;
  return !over && v == (long)*x;
}
bool bytes(const Tensor& t) {
  return t.scalar_type() == ScalarType::Float8_e4m3fn || t.scalar_type() == ScalarType::Byte;
}

// The six arguments of a cache from args[0]: a contiguous one.
bool cache_of(PyObject* const* args, int64_t dev, int64_t seqs, kda_kv_cache* c) {
  const Tensor *k = tensor(args[0]), *v = tensor(args[1]), *ks = tensor(args[2]), *vs = tensor(args[3]),
               *table = tensor(args[4]), *lens = tensor(args[5]);
  if (!k || !v || !table || k->dim() != 4 || table->dim() != 2) return false;
  if (!bytes(*k) || !bytes(*v) || k->size(3) != KDA_HEAD_DIM) return false;
  const int64_t pages = k->size(0), heads = k->size(1), page = k->size(2), blocks = table->size(1);
  if (pages > INT32_MAX || heads > INT32_MAX || page > INT32_MAX || blocks > INT32_MAX) return false;
  if (!dense(k, dev, k->scalar_type(), k->sizes()) || !dense(v, dev, v->scalar_type(), k->sizes()) ||
      !dense(ks, dev, ScalarType::Float, {pages, heads}) || !dense(vs, dev, ScalarType::Float, {pages, heads}) ||
      !dense(table, dev, ScalarType::Int, {seqs, blocks}) || !dense(lens, dev, ScalarType::Int, {seqs}))
    return false;
  std::memset(c, 0, sizeof(*c));
  c->k = k->data_ptr();
  c->v = v->data_ptr();
  c->k_scale = ks->data_ptr<float>();
  c->v_scale = vs->data_ptr<float>();
  c->token_stride = KDA_HEAD_DIM;
  c->head_stride = page * KDA_HEAD_DIM;
  c->page_stride = heads * c->head_stride;
  c->scale_stride = heads;
  c->num_pages = (int32_t)pages;
  c->page_size = (int32_t)page;
  c->kv_heads = (int32_t)heads;
  c->max_blocks = (int32_t)blocks;
  c->block_table = table->data_ptr<int32_t>();
  c->table_stride = blocks;
  c->kv_lens = lens->data_ptr<int32_t>();
  return true;
}
// cu_seqlens, and the number of sequences
const Tensor* lengths(PyObject* o, int64_t dev, int64_t* seqs) {
  const Tensor* cu = tensor(o);
  if (!cu || cu->dim() != 1 || cu->size(0) < 1 || cu->size(0) - 1 > INT32_MAX) return nullptr;
  *seqs = cu->size(0) - 1;
  return dense(cu, dev, ScalarType::Int, cu->sizes()) ? cu : nullptr;
}
Tensor make(at::IntArrayRef sizes, const Tensor& like, ScalarType type) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}
kda_stream_t stream_of(int64_t dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

#define UNUSUAL Py_RETURN_NONE

// (x, residual, weight, eps, want, group)
PyObject* add_rms_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *x = n == 6 ? tensor(args[0]) : nullptr, *w = n == 6 ? tensor(args[2]) : nullptr;
  if (!x || !w || !x->is_cuda() || x->dim() != 2) UNUSUAL;
  const int64_t dev = x->get_device(), T = x->size(0), C = x->size(1);
  int64_t ldx, ldr = C;
  float eps;
  int32_t group;
  if (C > INT32_MAX || !here(dev) || !rows(x, dev, ScalarType::BFloat16, x->sizes(), &ldx)) UNUSUAL;
  const ScalarType wt = w->scalar_type();
  if ((wt != ScalarType::BFloat16 && wt != ScalarType::Float) || !dense(w, dev, wt, {C})) UNUSUAL;
  if (!number(args[3], &eps) || !PyUnicode_Check(args[4]) || !integer(args[5], &group)) UNUSUAL;
  const bool only8 = PyUnicode_CompareWithASCIIString(args[4], "fp8") == 0;
  const bool both = PyUnicode_CompareWithASCIIString(args[4], "both") == 0;
  if (!only8 && !both && PyUnicode_CompareWithASCIIString(args[4], "bf16") != 0) UNUSUAL;
  const Tensor* r = nullptr;
  ScalarType rt = ScalarType::BFloat16;
  if (args[1] != Py_None) {
    r = tensor(args[1]);
    if (!r) UNUSUAL;
    rt = r->scalar_type();
    if ((rt != ScalarType::BFloat16 && rt != ScalarType::Float) || !rows(r, dev, rt, x->sizes(), &ldr)) UNUSUAL;
  }
  Tensor s, y, y8, scale;
  if (r) s = make(x->sizes(), *x, rt);
  if (!only8) y = make(x->sizes(), *x, ScalarType::BFloat16);
  if (only8 || both) {
    y8 = make(x->sizes(), *x, ScalarType::Float8_e4m3fn);
    scale = make({T, group == 128 ? (C + 127) / 128 : 1}, *x, ScalarType::Float);
  }
  auto at_ = [](const Tensor& t) -> void* { return t.defined() ? t.data_ptr() : nullptr; };
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = norm_entry(x->data_ptr(), ldx, r ? r->data_ptr() : nullptr, ldr,
                  rt == ScalarType::Float ? KDA_STATE_F32 : KDA_STATE_BF16, w->data_ptr(),
                  wt == ScalarType::Float ? KDA_STATE_F32 : KDA_STATE_BF16, eps, at_(s), C, at_(y), C, at_(y8), C,
                  static_cast<float*>(at_(scale)), group, T, (int32_t)C, stream_of(dev));
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  PyObject* out = PyTuple_New(4);
  if (!out) return nullptr;
  int i = 0;
  for (const Tensor* t : {&s, &y, &y8, &scale}) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(*t));
  return out;
  END_HANDLE_TH_ERRORS
}

// (q, k, v, rope, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, interleaved,
//  positions, workspace)
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) UNUSUAL;
  const Tensor *q = tensor(args[0]), *k = tensor(args[1]), *v = tensor(args[2]), *ws = tensor(args[13]);
  if (!q || !k || !v || !ws || !k->is_cuda() || k->dim() != 3 || q->dim() != 3) UNUSUAL;
  const int64_t dev = k->get_device(), T = k->size(0), heads = q->size(1);
  int64_t seqs, k_row, v_row, q_row, table_rows = 0, rot = 0;
  const Tensor* cu = lengths(args[10], dev, &seqs);
  kda_kv_cache c;
  if (!cu || !here(dev) || heads > INT32_MAX || k->size(2) != KDA_HEAD_DIM ||
      !rows(k, dev, ScalarType::BFloat16, k->sizes(), &k_row) ||
      !rows(v, dev, ScalarType::BFloat16, k->sizes(), &v_row) ||
      !rows(q, dev, ScalarType::BFloat16, {T, heads, KDA_HEAD_DIM}, &q_row) ||
      !dense(ws, dev, ScalarType::Byte, ws->sizes()) || !cache_of(args + 4, dev, seqs, &c) ||
      c.kv_heads != k->size(1) || !PyBool_Check(args[11]))
    UNUSUAL;
  const Tensor *rope = nullptr, *pos = nullptr;
  if (args[3] != Py_None) {
    rope = tensor(args[3]);
    if (!rope || rope->dim() != 2 || !dense(rope, dev, ScalarType::Float, rope->sizes())) UNUSUAL;
    table_rows = rope->size(0);
    rot = rope->size(1);
    if (rot > INT32_MAX) UNUSUAL;
  }
  if (args[12] != Py_None) {
    pos = tensor(args[12]);
    if (!dense(pos, dev, ScalarType::Int, {T})) UNUSUAL;
  }
  Tensor out = make(q->sizes(), *q, ScalarType::BFloat16);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = append_entry(q->data_ptr(), q_row, k->data_ptr(), k_row, v->data_ptr(), v_row,
                    rope ? rope->data_ptr<float>() : nullptr, table_rows, (int32_t)rot,
                    args[11] == Py_True, pos ? pos->data_ptr<int32_t>() : nullptr, out.data_ptr(),
                    heads * KDA_HEAD_DIM, &c, cu->data_ptr<int32_t>(), ws->data_ptr(), stream_of(dev), T,
                    (int32_t)seqs, (int32_t)heads, (size_t)ws->numel());
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, scale, max_q_len, softcap,
//  window, lse, workspace)
PyObject* cached_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 14) UNUSUAL;
  const Tensor *q = tensor(args[0]), *ws = tensor(args[13]);
  if (!q || !ws || !q->is_cuda() || q->dim() != 3 || q->size(2) != KDA_HEAD_DIM) UNUSUAL;
  const int64_t dev = q->get_device(), T = q->size(0), heads = q->size(1);
  int64_t seqs, q_row;
  const Tensor* cu = lengths(args[7], dev, &seqs);
  kda_kv_cache c;
  float scale, cap;
  int32_t max_q, window;
  if (!cu || !here(dev) || heads > INT32_MAX || !rows(q, dev, ScalarType::BFloat16, q->sizes(), &q_row) ||
      !dense(ws, dev, ScalarType::Byte, ws->sizes()) || !cache_of(args + 1, dev, seqs, &c) ||
      !number(args[8], &scale) || !integer(args[9], &max_q) || !number(args[10], &cap) ||
      !integer(args[11], &window) || !PyBool_Check(args[12]))
    UNUSUAL;
  Tensor out = make(q->sizes(), *q, ScalarType::BFloat16), lse;
  if (args[12] == Py_True) lse = make({T, heads}, *q, ScalarType::Float);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = attention_entry(q->data_ptr(), q_row, &c, cu->data_ptr<int32_t>(), scale, cap, window, out.data_ptr(),
                       heads * KDA_HEAD_DIM, lse.defined() ? lse.data_ptr<float>() : nullptr, ws->data_ptr(),
                       stream_of(dev), T, (int32_t)seqs, (int32_t)heads, max_q, (size_t)ws->numel());
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  PyObject* pair = PyTuple_New(2);
  if (!pair) return nullptr;
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
  return pair;
  END_HANDLE_TH_ERRORS
}

// (address of kda_add_rms_norm, of kda_rope_append, of kda_cached_attention), from the loaded library
PyObject* entries(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "three addresses");
    return nullptr;
  }
  void* p[3];
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  norm_entry = reinterpret_cast<decltype(norm_entry)>(p[0]);
  append_entry = reinterpret_cast<decltype(append_entry)>(p[1]);
  attention_entry = reinterpret_cast<decltype(attention_entry)>(p[2]);
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(add_rms_norm), METHOD(rope_append), METHOD(cached_attention), METHOD(entries),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer(void) { return PyModule_Create(&module); }
