// Marshalling of the layer operators' usual calls in C++: on small calls the checks and
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
decltype(&kda_tree_attention) tree_attention_entry;
decltype(&kda_tree_plan) plan_entry;
decltype(&kda_tree_recurrent_fwd) recurrent_entry;
decltype(&kda_tree_commit) commit_entry;
decltype(&kda_cache_accept) accept_entry;
decltype(&kda_pages_free) free_entry;
decltype(&kda_pages_reserve) reserve_entry;
decltype(&kda_pages_fork) fork_entry;
decltype(&kda_pages_copy) copy_entry;

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

// A cache's keys, values and scales from args[0]: contiguous ones.
bool pools_of(PyObject* const* args, int64_t dev, kda_kv_cache* c) {
  const Tensor *k = tensor(args[0]), *v = tensor(args[1]), *ks = tensor(args[2]), *vs = tensor(args[3]);
  if (!k || !v || k->dim() != 4) return false;
  if (!bytes(*k) || !bytes(*v) || k->size(3) != KDA_HEAD_DIM) return false;
  const int64_t pages = k->size(0), heads = k->size(1), page = k->size(2);
  if (pages > INT32_MAX || heads > INT32_MAX || page > INT32_MAX) return false;
  if (!dense(k, dev, k->scalar_type(), k->sizes()) || !dense(v, dev, v->scalar_type(), k->sizes()) ||
      !dense(ks, dev, ScalarType::Float, {pages, heads}) || !dense(vs, dev, ScalarType::Float, {pages, heads}))
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
  return true;
}
// The six arguments of a cache with its indexes.
bool cache_of(PyObject* const* args, int64_t dev, int64_t seqs, kda_kv_cache* c) {
  const Tensor *table = tensor(args[4]), *lens = tensor(args[5]);
  if (!table || table->dim() != 2 || table->size(1) > INT32_MAX) return false;
  const int64_t blocks = table->size(1);
  if (!dense(table, dev, ScalarType::Int, {seqs, blocks}) || !dense(lens, dev, ScalarType::Int, {seqs}) ||
      !pools_of(args, dev, c))
    return false;
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
//  window, lse, workspace[, mask])
PyObject* attention(PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const bool tree = n == 15;
  if (n != 14 && !tree) UNUSUAL;
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
  const Tensor* mask = tree ? tensor(args[14]) : nullptr;
  if (tree && !dense(mask, dev, ScalarType::Long, {T})) UNUSUAL;
  Tensor out = make(q->sizes(), *q, ScalarType::BFloat16), lse;
  if (args[12] == Py_True) lse = make({T, heads}, *q, ScalarType::Float);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  float* lse_ptr = lse.defined() ? lse.data_ptr<float>() : nullptr;
  rc = tree ? tree_attention_entry(q->data_ptr(), q_row, &c, cu->data_ptr<int32_t>(), mask->data_ptr(), scale, cap,
                                   window, out.data_ptr(), heads * KDA_HEAD_DIM, lse_ptr, ws->data_ptr(),
                                   stream_of(dev), T, (int32_t)seqs, (int32_t)heads, max_q, (size_t)ws->numel())
            : attention_entry(q->data_ptr(), q_row, &c, cu->data_ptr<int32_t>(), scale, cap, window,
                              out.data_ptr(), heads * KDA_HEAD_DIM, lse_ptr, ws->data_ptr(), stream_of(dev), T,
                              (int32_t)seqs, (int32_t)heads, max_q, (size_t)ws->numel());
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  PyObject* pair = PyTuple_New(2);
  if (!pair) return nullptr;
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
  return pair;
  END_HANDLE_TH_ERRORS
}

PyObject* cached_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 14) UNUSUAL;
  return attention(args, n);
}
PyObject* tree_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 15) UNUSUAL;
  return attention(args, n);
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* p = PyTuple_New(2);
  if (!p) return nullptr;
  PyTuple_SET_ITEM(p, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(p, 1, THPVariable_Wrap(b));
  return p;
}
// A dense int32 [n]
const int32_t* list(PyObject* o, int64_t dev, int64_t n) {
  const Tensor* t = tensor(o);
  return dense(t, dev, ScalarType::Int, {n}) ? t->data_ptr<int32_t>() : nullptr;
}
// (an empty tensor has no address: such calls are not usual)
const Tensor* status(PyObject* o, int64_t dev) {
  const Tensor* t = tensor(o);
  return t && dense(t, dev, ScalarType::Byte, t->sizes()) && t->numel() > 0 ? t : nullptr;
}

// (parents, cu_seqlens, kv_lens, max_q_len, workspace)
PyObject* tree_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor* parents = n == 5 ? tensor(args[0]) : nullptr;
  if (!parents || !parents->is_cuda() || parents->dim() != 1) UNUSUAL;
  const int64_t dev = parents->get_device(), T = parents->size(0);
  int64_t seqs;
  int32_t most;
  const Tensor* cu = lengths(args[1], dev, &seqs);
  if (!cu || !here(dev)) UNUSUAL;
  const int32_t *up = list(args[0], dev, T), *lens = list(args[2], dev, seqs);
  const Tensor* ws = status(args[4], dev);
  if (!up || !lens || !ws || !integer(args[3], &most)) UNUSUAL;
  Tensor mask = make({T}, *parents, ScalarType::Long), pos = make({T}, *parents, ScalarType::Int);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = plan_entry(up, cu->data_ptr<int32_t>(), lens, mask.data_ptr(), pos.data_ptr<int32_t>(), ws->data_ptr(),
                  stream_of(dev), T, (int32_t)seqs, most, (size_t)ws->numel());
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  return pair(mask, pos);
  END_HANDLE_TH_ERRORS
}

// What the recurrence's forward and commit have in common.
struct Recur {
  int64_t dev, T, heads, seqs, k_row, g_row;
  const Tensor *k, *g, *A_log, *dt, *state, *cu, *ws;
  const int32_t* parents;
  int32_t most;
  float lower;
  ScalarType type;      // the state's
};
bool recur_of(PyObject* k, PyObject* g, PyObject* A_log, PyObject* dt, PyObject* lower, PyObject* state,
              PyObject* cu, PyObject* parents, PyObject* most, PyObject* ws, Recur* r) {
  r->k = tensor(k);
  if (!r->k || !r->k->is_cuda() || r->k->dim() != 3 || r->k->size(2) != KDA_HEAD_DIM) return false;
  r->dev = r->k->get_device();
  r->T = r->k->size(0);
  r->heads = r->k->size(1);
  if (!here(r->dev) || r->heads > INT32_MAX || r->T == 0) return false;
  r->cu = lengths(cu, r->dev, &r->seqs);
  r->g = tensor(g);
  r->A_log = tensor(A_log);
  r->dt = tensor(dt);
  r->state = tensor(state);
  r->ws = status(ws, r->dev);
  r->parents = list(parents, r->dev, r->T);
  if (!r->cu || !r->state || !r->ws || !r->parents) return false;
  r->type = r->state->scalar_type();
  return (r->type == ScalarType::Float || r->type == ScalarType::BFloat16) &&
         dense(r->state, r->dev, r->type, {r->seqs, r->heads, KDA_HEAD_DIM, KDA_HEAD_DIM}) &&
         rows(r->k, r->dev, ScalarType::BFloat16, r->k->sizes(), &r->k_row) &&
         rows(r->g, r->dev, ScalarType::BFloat16, r->k->sizes(), &r->g_row) &&
         dense(r->A_log, r->dev, ScalarType::Float, {r->heads}) &&
         dense(r->dt, r->dev, ScalarType::Float, {r->heads, KDA_HEAD_DIM}) && number(lower, &r->lower) &&
         integer(most, &r->most);
}
int kind_of(ScalarType t) { return t == ScalarType::Float ? KDA_STATE_F32 : KDA_STATE_BF16; }

// (q, k, v, g, beta, A_log, dt_bias, lower_bound, scale, initial_state, cu_seqlens, parents, max_q_len, workspace)
PyObject* tree_recurrent_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Recur r;
  if (n != 14 || !recur_of(args[1], args[3], args[5], args[6], args[7], args[9], args[10], args[11], args[12],
                           args[13], &r))
    UNUSUAL;
  const Tensor *q = tensor(args[0]), *v = tensor(args[2]), *beta = tensor(args[4]);
  int64_t q_row, v_row, beta_row;
  float scale;
  if (!rows(q, r.dev, ScalarType::BFloat16, r.k->sizes(), &q_row) ||
      !rows(v, r.dev, ScalarType::BFloat16, r.k->sizes(), &v_row) ||
      !rows(beta, r.dev, ScalarType::BFloat16, {r.T, r.heads}, &beta_row) || !number(args[8], &scale))
    UNUSUAL;
  Tensor out = make(r.k->sizes(), *r.k, ScalarType::BFloat16), u = make(r.k->sizes(), *r.k, ScalarType::Float);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = recurrent_entry(q->data_ptr(), q_row, r.k->data_ptr(), r.k_row, v->data_ptr(), v_row, r.g->data_ptr(), r.g_row,
                       beta->data_ptr(), beta_row, r.A_log->data_ptr<float>(), r.dt->data_ptr<float>(), r.lower,
                       scale, r.state->data_ptr(), kind_of(r.type), r.cu->data_ptr<int32_t>(), r.parents,
                       out.data_ptr(), u.data_ptr<float>(), r.ws->data_ptr(), stream_of(r.dev), r.T,
                       (int32_t)r.seqs, (int32_t)r.heads, r.most, (size_t)r.ws->numel());
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  return pair(out, u);
  END_HANDLE_TH_ERRORS
}

// (k, g, A_log, dt_bias, lower_bound, initial_state, cu_seqlens, parents, u, accepted, max_q_len, final_state, workspace)
PyObject* tree_commit(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Recur r;
  if (n != 13 || !recur_of(args[0], args[1], args[2], args[3], args[4], args[5], args[6], args[7], args[10],
                           args[12], &r))
    UNUSUAL;
  const Tensor* u = tensor(args[8]);
  const int32_t* accepted = list(args[9], r.dev, r.seqs);
  if (!accepted || !dense(u, r.dev, ScalarType::Float, r.k->sizes())) UNUSUAL;
  Tensor made;
  const Tensor* fin = &made;
  if (args[11] == Py_None) {
    made = make(r.state->sizes(), *r.k, r.type);
  } else {
    fin = tensor(args[11]);
    if (!dense(fin, r.dev, r.type, r.state->sizes())) UNUSUAL;
  }
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = commit_entry(r.k->data_ptr(), r.k_row, r.g->data_ptr(), r.g_row, r.A_log->data_ptr<float>(),
                    r.dt->data_ptr<float>(), r.lower, r.state->data_ptr(), fin->data_ptr(), kind_of(r.type),
                    r.cu->data_ptr<int32_t>(), r.parents, u->data_ptr<float>(), accepted, r.ws->data_ptr(),
                    stream_of(r.dev), r.T, (int32_t)r.seqs, (int32_t)r.heads, r.most, (size_t)r.ws->numel());
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  if (fin != &made) {
    Py_INCREF(args[11]);
    return args[11];
  }
  return THPVariable_Wrap(made);
  END_HANDLE_TH_ERRORS
}

// (k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, parents, accepted, max_q_len, workspace)
PyObject* cache_accept(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *k = n == 11 ? tensor(args[0]) : nullptr, *parents = n == 11 ? tensor(args[7]) : nullptr;
  if (!k || !parents || !k->is_cuda() || parents->dim() != 1) UNUSUAL;
  const int64_t dev = k->get_device(), T = parents->size(0);
  int64_t seqs;
  int32_t most;
  const Tensor* cu = lengths(args[6], dev, &seqs);
  kda_kv_cache c;
  if (!cu || !here(dev) || !cache_of(args, dev, seqs, &c)) UNUSUAL;
  const int32_t *up = list(args[7], dev, T), *accepted = list(args[8], dev, seqs);
  const Tensor* ws = status(args[10], dev);
  if (!up || !accepted || !ws || !integer(args[9], &most)) UNUSUAL;
  Tensor lens = make({seqs}, *parents, ScalarType::Int);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = accept_entry(&c, cu->data_ptr<int32_t>(), up, accepted, lens.data_ptr<int32_t>(), ws->data_ptr(),
                    stream_of(dev), T, (int32_t)seqs, most, (size_t)ws->numel());
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  return THPVariable_Wrap(lens);
  END_HANDLE_TH_ERRORS
}

// A pool: (refs, block_table, kv_lens, page_size), dense, from args[0].
struct PoolArgs {
  int64_t dev;
  int32_t *refs, *table, *lens;
  int32_t pages, rows, blocks, page;
};
bool pool_of(PyObject* const* args, PyObject* page, PoolArgs* p) {
  const Tensor *refs = tensor(args[0]), *table = tensor(args[1]), *lens = tensor(args[2]);
  if (!refs || !table || !lens || !refs->is_cuda() || refs->dim() != 1 || table->dim() != 2) return false;
  p->dev = refs->get_device();
  const int64_t pages = refs->size(0), rows = table->size(0), blocks = table->size(1);
  if (!here(p->dev) || pages > INT32_MAX || rows > INT32_MAX || blocks > INT32_MAX) return false;
  if (!dense(refs, p->dev, ScalarType::Int, {pages}) || !dense(table, p->dev, ScalarType::Int, {rows, blocks}) ||
      !dense(lens, p->dev, ScalarType::Int, {rows}) || !integer(page, &p->page))
    return false;
  p->refs = refs->data_ptr<int32_t>();
  p->table = table->data_ptr<int32_t>();
  p->lens = lens->data_ptr<int32_t>();
  p->pages = (int32_t)pages;
  p->rows = (int32_t)rows;
  p->blocks = (int32_t)blocks;
  return true;
}
// A dense int32 list of any length that fits 32 bits
const int32_t* any_list(PyObject* o, int64_t dev, int64_t* n) {
  const Tensor* t = tensor(o);
  if (!t || t->dim() != 1 || t->size(0) < 1 || t->size(0) > INT32_MAX) return nullptr;
  *n = t->size(0);
  return list(o, dev, *n);
}
// True for done: None is for what is not usual.
PyObject* done(int rc) {
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  Py_RETURN_TRUE;
}

// (refs, block_table, kv_lens, page_size, rows, workspace)
PyObject* free_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  PoolArgs p;
  if (n != 6 || !pool_of(args, args[3], &p)) UNUSUAL;
  const Tensor* ws = status(args[5], p.dev);
  const int32_t* rows_ = nullptr;
  int64_t num = 0;
  if (!ws || (args[4] != Py_None && !(rows_ = any_list(args[4], p.dev, &num)))) UNUSUAL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = free_entry(p.refs, p.pages, p.table, p.blocks, p.rows, p.blocks, p.lens, p.page, rows_, (int32_t)num,
                  ws->data_ptr(), (size_t)ws->numel(), stream_of(p.dev));
  Py_END_ALLOW_THREADS
  return done(rc);
  END_HANDLE_TH_ERRORS
}

// (refs, block_table, kv_lens, new_tokens, page_size, workspace)
PyObject* reserve_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  PoolArgs p;
  if (n != 6 || !pool_of(args, args[4], &p)) UNUSUAL;
  const Tensor* ws = status(args[5], p.dev);
  const int32_t* add = list(args[3], p.dev, p.rows);
  if (!ws || !add) UNUSUAL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = reserve_entry(p.refs, p.pages, p.table, p.blocks, p.rows, p.blocks, p.lens, p.page, add, ws->data_ptr(),
                     (size_t)ws->numel(), stream_of(p.dev));
  Py_END_ALLOW_THREADS
  return done(rc);
  END_HANDLE_TH_ERRORS
}

// (refs, block_table, kv_lens, src, dst, page_size, workspace)
PyObject* fork_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  PoolArgs p;
  if (n != 7 || !pool_of(args, args[5], &p)) UNUSUAL;
  const Tensor* ws = status(args[6], p.dev);
  int64_t num = 0;
  const int32_t* src = any_list(args[3], p.dev, &num);
  const int32_t* dst = src ? list(args[4], p.dev, num) : nullptr;
  if (!ws || !dst) UNUSUAL;
  const Tensor* like = tensor(args[0]);
  Tensor from = make({num}, *like, ScalarType::Int), to = make({num}, *like, ScalarType::Int);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = fork_entry(p.refs, p.pages, p.table, p.blocks, p.rows, p.blocks, p.lens, p.page, src, dst, (int32_t)num,
                  from.data_ptr<int32_t>(), to.data_ptr<int32_t>(), ws->data_ptr(), (size_t)ws->numel(),
                  stream_of(p.dev));
  Py_END_ALLOW_THREADS
  if (rc != KDA_OK) return PyLong_FromLong(rc);
  return pair(from, to);
  END_HANDLE_TH_ERRORS
}

// (k_cache, v_cache, k_scale, v_scale, from_pages, to_pages, workspace)
PyObject* copy_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor* k = n == 7 ? tensor(args[0]) : nullptr;
  if (!k || !k->is_cuda()) UNUSUAL;
  const int64_t dev = k->get_device();
  int64_t num = 0;
  kda_kv_cache c;
  if (!here(dev) || !pools_of(args, dev, &c)) UNUSUAL;
  const int32_t* from = any_list(args[4], dev, &num);
  const int32_t* to = from ? list(args[5], dev, num) : nullptr;
  const Tensor* ws = status(args[6], dev);
  if (!to || !ws) UNUSUAL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = copy_entry(&c, from, to, num, ws->data_ptr(), (size_t)ws->numel(), stream_of(dev));
  Py_END_ALLOW_THREADS
  return done(rc);
  END_HANDLE_TH_ERRORS
}

// The entry points' addresses from the loaded library, in the order below.
template <class F>
void take(F& entry, PyObject* o) { entry = reinterpret_cast<F>(PyLong_AsVoidPtr(o)); }
PyObject* entries(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 12) {
    PyErr_SetString(PyExc_TypeError, "twelve addresses");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i)
    if (!PyLong_AsVoidPtr(args[i])) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  take(norm_entry, args[0]);
  take(append_entry, args[1]);
  take(attention_entry, args[2]);
  take(tree_attention_entry, args[3]);
  take(plan_entry, args[4]);
  take(recurrent_entry, args[5]);
  take(commit_entry, args[6]);
  take(accept_entry, args[7]);
  take(free_entry, args[8]);
  take(reserve_entry, args[9]);
  take(fork_entry, args[10]);
  take(copy_entry, args[11]);
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(add_rms_norm), METHOD(rope_append), METHOD(cached_attention),
                         METHOD(tree_attention), METHOD(tree_plan), METHOD(tree_recurrent_fwd),
                         METHOD(tree_commit), METHOD(cache_accept), METHOD(free_pages), METHOD(reserve_pages),
                         METHOD(fork_pages), METHOD(copy_pages), METHOD(entries), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer(void) { return PyModule_Create(&module); }
