// The attention operators' calls on torch tensors (a Python extension module): argument tests, results and scratch, and
// the C entries of include/moe_attention.h. attention.py documents the operators and says what is wrong with arguments
// that are not taken here: a function returns None for those (also when the tensors' device is not the current one, or
// where gradients are asked for), the status for a call that the library refuses, and the results otherwise. Tensors that
// a call changes have their version counted up, as autograd expects of changes in place.
//
// A decode step is a few kernels of a few microseconds each, so what a call costs on the host counts: the same tests,
// allocations and marshalling written in Python took 9 us of a prefill call and 11 us of a decode call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <utility>

#include "../../include/moe_attention.h"

namespace {

using at::Tensor;

// arg as a tensor, or nullptr
const Tensor* tensor(PyObject* arg) { return THPVariable_Check(arg) ? &THPVariable_Unpack(arg) : nullptr; }

// an optional tensor: false when it is neither None nor a tensor
bool optional(PyObject* arg, const Tensor*& t) {
  t = nullptr;
  if (arg == Py_None) return true;
  t = tensor(arg);
  return t != nullptr;
}

bool scale_of(PyObject* arg, int64_t dim, float& scale) {
  if (arg == Py_None) {
    scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim)));
    return true;
  }
  const double v = PyFloat_AsDouble(arg);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  scale = static_cast<float>(v);
  return true;
}

bool int_of(PyObject* arg, int32_t& v) {
  const long x = PyLong_AsLong(arg);
  if (x == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  if (x < 0 || x > INT32_MAX) return false;
  v = static_cast<int32_t>(x);
  return true;
}

int dtype_of(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? MOE_ATTN_BF16 : t.scalar_type() == at::kHalf ? MOE_ATTN_F16 : -1;
}

// [tokens][heads][dim] with dense rows
bool is_rows(const Tensor* t, const Tensor& like) {
  return t && t->dim() == 3 && t->scalar_type() == like.scalar_type() && t->get_device() == like.get_device() &&
         t->stride(2) == 1;
}
bool is_ints(const Tensor* t, int dim, at::ScalarType type, int device) {
  return t && t->dim() == dim && t->scalar_type() == type && t->get_device() == device &&
         (t->stride(dim - 1) == 1 || t->size(dim - 1) < 2);
}
// the stride of a dimension of one is never walked, so it is given any valid value
int64_t token_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2); }
int64_t head_stride(const Tensor& t) { return t.size(1) > 1 ? t.stride(1) : t.size(2); }

bool here(const Tensor& t) { return t.is_cuda() && t.get_device() == c10::cuda::current_device(); }
void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }
bool fits(int64_t v) { return v <= INT32_MAX; }
// The allocation without at::empty's way through the dispatcher (five results: 9.8 us a call of assign, now 8.0).
Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

bool wants_grad(const Tensor& t) { return t.requires_grad() && at::GradMode::is_enabled(); }
void changed(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

struct Cache {
  const Tensor *k, *v, *ks, *vs;
};
bool is_cache(PyObject* arg, const Tensor& like, Cache& c) {
  if (!PyTuple_Check(arg) || PyTuple_GET_SIZE(arg) != 4) return false;
  c.k = tensor(PyTuple_GET_ITEM(arg, 0)), c.v = tensor(PyTuple_GET_ITEM(arg, 1));
  c.ks = tensor(PyTuple_GET_ITEM(arg, 2)), c.vs = tensor(PyTuple_GET_ITEM(arg, 3));
  if (!c.k || !c.v || !c.ks || !c.vs) return false;
  const at::ScalarType type = c.k->scalar_type();
  const int dev = like.get_device();
  return (type == at::kFloat8_e4m3fn || type == at::kByte) && c.v->scalar_type() == type && c.k->dim() == 4 &&
         c.v->sizes() == c.k->sizes() && c.ks->scalar_type() == at::kFloat && c.vs->scalar_type() == at::kFloat &&
         c.ks->dim() == 2 && c.ks->sizes() == c.k->sizes().slice(0, 2) && c.vs->sizes() == c.ks->sizes() &&
         c.k->is_contiguous() && c.v->is_contiguous() && c.ks->is_contiguous() && c.vs->is_contiguous() &&
         c.k->get_device() == dev && c.v->get_device() == dev && c.ks->get_device() == dev && c.vs->get_device() == dev &&
         fits(c.k->size(0)) && fits(c.k->size(1)) && fits(c.k->size(2));
}

PyObject* none() { Py_RETURN_NONE; }

// (q, k, v, cu_q, cu_k, scale, out, lse) -> (out, lse)
PyObject* prefill(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return none();
  const Tensor *q = tensor(arg[0]), *k = tensor(arg[1]), *v = tensor(arg[2]), *cq = tensor(arg[3]), *ck = tensor(arg[4]);
  const Tensor *out_given, *lse_given;
  moe_attn_prefill_args a = {};
  if (!q || !is_rows(q, *q) || (a.dtype = dtype_of(*q)) < 0 || !here(*q) || !is_rows(k, *q) || !is_rows(v, *q) ||
      v->sizes() != k->sizes() || k->size(2) != q->size(2) || !is_ints(cq, 1, at::kInt, q->get_device()) ||
      !is_ints(ck, 1, at::kInt, q->get_device()) || cq->size(0) < 1 || ck->size(0) != cq->size(0) ||
      !scale_of(arg[5], q->size(2), a.scale) || !optional(arg[6], out_given) || !optional(arg[7], lse_given) ||
      !fits(q->size(0)) || !fits(k->size(0)) || !fits(cq->size(0)) || !fits(q->size(1)) || !fits(k->size(1)) ||
      wants_grad(*q) || wants_grad(*k) || wants_grad(*v))
    return none();
  if (out_given && (!is_rows(out_given, *q) || out_given->sizes() != q->sizes())) return none();
  if (lse_given && (lse_given->scalar_type() != at::kFloat || lse_given->dim() != 2 ||
                    lse_given->size(0) != q->size(1) || lse_given->size(1) != q->size(0) ||
                    !lse_given->is_contiguous() || lse_given->get_device() != q->get_device()))
    return none();
  const Tensor out = out_given ? *out_given : empty(q->sizes(), q->scalar_type(), *q);
  const Tensor lse = lse_given ? *lse_given : empty({q->size(1), q->size(0)}, at::kFloat, *q);
  a.q = q->data_ptr(), a.k = k->data_ptr(), a.v = v->data_ptr(), a.out = out.data_ptr();
  a.lse = static_cast<float*>(lse.data_ptr());
  a.cu_q = static_cast<const int32_t*>(cq->data_ptr()), a.cu_k = static_cast<const int32_t*>(ck->data_ptr());
  a.q_token = token_stride(*q), a.q_head = head_stride(*q), a.k_token = token_stride(*k), a.k_head = head_stride(*k);
  a.v_token = token_stride(*v), a.v_head = head_stride(*v);
  a.out_token = token_stride(out), a.out_head = head_stride(out);
  a.n_seqs = static_cast<int32_t>(cq->size(0) - 1);
  a.total_q = static_cast<int32_t>(q->size(0)), a.total_k = static_cast<int32_t>(k->size(0));
  a.n_heads = static_cast<int32_t>(q->size(1)), a.n_kv_heads = static_cast<int32_t>(k->size(1));
  a.head_dim = static_cast<int32_t>(q->size(2));
  const moe_status st = moe_attn_prefill(&a, stream_of(*q));
  if (st != MOE_OK) return PyLong_FromLong(st);
  if (out_given) changed(out);
  if (lse_given) changed(lse);
  return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

// (ctx_lens, new_lens, free_blocks, block_table, block_size, max_tokens) -> (cu_new, kv_lens, slot_map, positions, used)
PyObject* assign(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) return none();
  const Tensor *ctx = tensor(arg[0]), *fresh = tensor(arg[1]), *free = tensor(arg[2]), *table = tensor(arg[3]);
  moe_kv_assign_args a = {};
  if (!ctx || !here(*ctx) || !is_ints(ctx, 1, at::kInt, ctx->get_device()) ||
      !is_ints(fresh, 1, at::kInt, ctx->get_device()) || !is_ints(free, 1, at::kInt, ctx->get_device()) ||
      !is_ints(table, 2, at::kInt, ctx->get_device()) || fresh->size(0) != ctx->size(0) ||
      table->size(0) != ctx->size(0) || !int_of(arg[4], a.block_size) || !int_of(arg[5], a.max_tokens) ||
      !fits(ctx->size(0)) || !fits(free->size(0)) || !fits(table->size(1)))
    return none();
  const int64_t reqs = ctx->size(0);
  // five allocations: they take less time than views of one
  const Tensor cu_new = empty({reqs + 1}, at::kInt, *ctx), kv_lens = empty({reqs}, at::kInt, *ctx);
  const Tensor used = empty({1}, at::kInt, *ctx), positions = empty({a.max_tokens}, at::kInt, *ctx);
  const Tensor slots = empty({a.max_tokens}, at::kLong, *ctx);
  a.ctx_lens = static_cast<const int32_t*>(ctx->data_ptr()), a.new_lens = static_cast<const int32_t*>(fresh->data_ptr());
  a.free_blocks = static_cast<const int32_t*>(free->data_ptr());
  a.block_table = static_cast<int32_t*>(table->data_ptr());
  a.cu_new = static_cast<int32_t*>(cu_new.data_ptr()), a.kv_lens = static_cast<int32_t*>(kv_lens.data_ptr());
  a.used = static_cast<int32_t*>(used.data_ptr()), a.positions = static_cast<int32_t*>(positions.data_ptr());
  a.slot_map = static_cast<int64_t*>(slots.data_ptr());
  a.table_stride = reqs > 1 ? table->stride(0) : table->size(1);
  a.n_requests = static_cast<int32_t>(reqs), a.n_free = static_cast<int32_t>(free->size(0));
  a.max_blocks = static_cast<int32_t>(table->size(1));
  const moe_status st = moe_kv_assign(&a, stream_of(*ctx));
  if (st != MOE_OK) return PyLong_FromLong(st);
  changed(*table);
  return Py_BuildValue("(NNNNN)", THPVariable_Wrap(cu_new), THPVariable_Wrap(kv_lens), THPVariable_Wrap(slots),
                       THPVariable_Wrap(positions), THPVariable_Wrap(used));
  END_HANDLE_TH_ERRORS
}

// (k, v, slot_map, cache) -> True
PyObject* append(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return none();
  const Tensor *k = tensor(arg[0]), *v = tensor(arg[1]), *slots = tensor(arg[2]);
  moe_kv_append_args a = {};
  Cache c;
  if (!k || !is_rows(k, *k) || (a.dtype = dtype_of(*k)) < 0 || !here(*k) || !is_rows(v, *k) ||
      v->sizes() != k->sizes() || !is_ints(slots, 1, at::kLong, k->get_device()) || slots->size(0) < k->size(0) ||
      !is_cache(arg[3], *k, c) || c.k->size(1) != k->size(1) || c.k->size(3) != k->size(2) || !fits(k->size(0)))
    return none();
  a.k = k->data_ptr(), a.v = v->data_ptr(), a.slot_map = static_cast<const int64_t*>(slots->data_ptr());
  a.k_codes = c.k->data_ptr(), a.v_codes = c.v->data_ptr();
  a.k_scale = static_cast<float*>(c.ks->data_ptr()), a.v_scale = static_cast<float*>(c.vs->data_ptr());
  a.k_token = token_stride(*k), a.k_head = head_stride(*k), a.v_token = token_stride(*v), a.v_head = head_stride(*v);
  a.n_tokens = static_cast<int32_t>(k->size(0)), a.n_kv_heads = static_cast<int32_t>(k->size(1));
  a.head_dim = static_cast<int32_t>(k->size(2));
  a.block_size = static_cast<int32_t>(c.k->size(2)), a.num_blocks = static_cast<int32_t>(c.k->size(0));
  const moe_status st = moe_kv_append(&a, stream_of(*k));
  if (st != MOE_OK) return PyLong_FromLong(st);
  for (const Tensor* t : {c.k, c.v, c.ks, c.vs}) changed(*t);
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// Scratch of a stream's calls, which run one after the other; calls under capture get their own, as a graph may run
// beside them later. Kept for the process's life (the GIL guards the map).
Tensor workspace_of(const Tensor& q, void* stream, int64_t need) {
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
    return empty({need}, at::kByte, q);
  static auto* kept = new std::map<std::pair<int, void*>, Tensor>;
  Tensor& w = (*kept)[{q.get_device(), stream}];
  if (!w.defined() || w.numel() < need) w = empty({need}, at::kByte, q);
  return w;
}

// (q, cache, block_table, kv_lens, scale, out, lse, workspace) -> (out, lse)
PyObject* decode(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return none();
  const Tensor *q = tensor(arg[0]), *table = tensor(arg[2]), *lens = tensor(arg[3]);
  const Tensor *out_given, *lse_given, *ws_given;
  moe_attn_decode_args a = {};
  Cache c;
  if (!q || !is_rows(q, *q) || (a.dtype = dtype_of(*q)) < 0 || !here(*q) || !is_cache(arg[1], *q, c) ||
      c.k->size(3) != q->size(2) || !is_ints(table, 2, at::kInt, q->get_device()) ||
      !is_ints(lens, 1, at::kInt, q->get_device()) || table->size(0) != q->size(0) || lens->size(0) != q->size(0) ||
      !scale_of(arg[4], q->size(2), a.scale) || !optional(arg[5], out_given) || !optional(arg[6], lse_given) ||
      !optional(arg[7], ws_given) || !fits(q->size(0)) || !fits(q->size(1)) || !fits(table->size(1)) ||
      wants_grad(*q))
    return none();
  if (out_given && (!is_rows(out_given, *q) || out_given->sizes() != q->sizes())) return none();
  if (lse_given && (lse_given->scalar_type() != at::kFloat || lse_given->sizes() != q->sizes().slice(0, 2) ||
                    !lse_given->is_contiguous() || lse_given->get_device() != q->get_device()))
    return none();
  if (ws_given && (ws_given->scalar_type() != at::kByte || !ws_given->is_contiguous() ||
                   ws_given->get_device() != q->get_device()))
    return none();
  a.n_requests = static_cast<int32_t>(q->size(0)), a.n_heads = static_cast<int32_t>(q->size(1));
  a.n_kv_heads = static_cast<int32_t>(c.k->size(1)), a.head_dim = static_cast<int32_t>(q->size(2));
  void* stream = stream_of(*q);
  const size_t need = moe_attn_decode_workspace(a.n_requests, a.n_heads, a.n_kv_heads, a.head_dim);
  if (need == 0) return PyLong_FromLong(moe_attn_decode(&a, stream));  // refused for its heads or head_dim
  const Tensor out = out_given ? *out_given : empty(q->sizes(), q->scalar_type(), *q);
  const Tensor lse = lse_given ? *lse_given : empty(q->sizes().slice(0, 2), at::kFloat, *q);
  const Tensor ws = ws_given ? *ws_given : workspace_of(*q, stream, static_cast<int64_t>(need));
  a.q = q->data_ptr(), a.k_codes = c.k->data_ptr(), a.v_codes = c.v->data_ptr();
  a.k_scale = static_cast<const float*>(c.ks->data_ptr()), a.v_scale = static_cast<const float*>(c.vs->data_ptr());
  a.block_table = static_cast<const int32_t*>(table->data_ptr());
  a.kv_lens = static_cast<const int32_t*>(lens->data_ptr());
  a.out = out.data_ptr(), a.lse = static_cast<float*>(lse.data_ptr());
  a.workspace = ws.data_ptr(), a.workspace_bytes = static_cast<size_t>(ws.numel());
  a.q_token = token_stride(*q), a.q_head = head_stride(*q), a.out_token = token_stride(out), a.out_head = head_stride(out);
  a.table_stride = a.n_requests > 1 ? table->stride(0) : table->size(1);
  a.block_size = static_cast<int32_t>(c.k->size(2)), a.num_blocks = static_cast<int32_t>(c.k->size(0));
  a.max_blocks = static_cast<int32_t>(table->size(1));
  const moe_status st = moe_attn_decode(&a, stream);
  if (st != MOE_OK) return PyLong_FromLong(st);
  if (out_given) changed(out);
  if (lse_given) changed(lse);
  return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<prefill>("prefill"), method<assign>("assign"), method<append>("append"),
                         method<decode>("decode"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "attention_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attention_py() { return PyModule_Create(&module); }
