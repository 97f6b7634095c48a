// Short way from Python to libq4's fused calls and its cache, for small layers, where the
// time of a call is the time of its Python (7 of 11 us for a 512 x 512 row).
//
// Each function takes the Python function's arguments by position, checks that
// the call is an ordinary one (contiguous device tensors of the current device
// with the right shapes and types, none of them part of a gradient), allocates what it returns, and calls the
// C entry point, whose address it was given.  It returns None for any other
// call and for any status but OK (a refused call has launched nothing): the
// Python function then takes its own full way, with its own errors.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "q4.h"

namespace {

decltype(&q4_linear) p_linear;
decltype(&q4_linear_workspace_size) p_linear_ws;
decltype(&q4_route) p_route;
decltype(&q4_route_plan) p_route_plan;
decltype(&q4_route_plan_size) p_plan_size;
decltype(&q4_experts) p_experts;
decltype(&q4_experts_workspace_size) p_experts_ws;
decltype(&q4_moe) p_moe;
decltype(&q4_moe_workspace_size) p_moe_ws;
decltype(&q4_cache_write) p_cache_write;
decltype(&q4_cache_read) p_cache_read;
decltype(&q4_attention) p_attention;
decltype(&q4_attention_workspace_size) p_attention_ws;

// The arguments of one call: the first tensor names the device, and every check
// that fails is remembered.
struct Call {
  PyObject* const* args;
  bool grad = at::GradMode::is_enabled();
  bool ok = true;
  int device = -1;

  // Argument i as a tensor of the call's device, or nullptr for None.  strided: one
  // that need not be contiguous.
  const at::Tensor* tensor(int i, bool strided = false) {
    PyObject* o = args[i];
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || (!strided && !t.is_contiguous()) || (grad && t.requires_grad()) || t._fw_grad(0).defined()) {
      ok = false;
      return nullptr;
    }
    const int d = t.device().index();
    if (device < 0) device = d;
    if (d != device) ok = false;
    return &t;
  }
  const at::Tensor* needed(int i, bool strided = false) {
    const at::Tensor* t = tensor(i, strided);
    if (t == nullptr) ok = false;
    return t;
  }
  int64_t integer(int i) {
    const long long v = PyLong_Check(args[i]) ? PyLong_AsLongLong(args[i]) : -1;
    if (v == -1) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  bool truth(int i) {
    if (args[i] == Py_True) return true;
    if (args[i] != Py_False) ok = false;
    return false;
  }
  int dtype(const at::Tensor& t) {
    switch (t.scalar_type()) {
      case at::kFloat: return Q4_F32;
      case at::kHalf: return Q4_F16;
      case at::kBFloat16: return Q4_BF16;
      default: ok = false; return -1;
    }
  }
  void want(bool condition) { ok = ok && condition; }
  void shape(const at::Tensor* t, at::IntArrayRef s) { want(t == nullptr || t->sizes() == s); }
  // Last: the call's device is the current one.
  bool ready() { return ok && device >= 0 && c10::hip::current_device() == device; }
  q4_stream_t stream() {
    return reinterpret_cast<q4_stream_t>(c10::hip::getCurrentHIPStream(device).stream());
  }
};

const void* data(const at::Tensor* t) { return t == nullptr ? nullptr : t->const_data_ptr(); }

at::Tensor bytes(const at::Tensor& like, size_t n) {
  return at::empty({static_cast<int64_t>(n)}, like.options().dtype(at::kByte));
}

// Runs f (a call's body); a C++ exception becomes None: the Python way reports it.
template <typename F>
PyObject* guarded(F f) {
  try {
    PyObject* r = f();
    if (r != nullptr) return r;
  } catch (...) {
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

q4_epilogue epilogue(Call& c, const at::Tensor* bias, int64_t act, bool gated, const at::Tensor* residual) {
  return q4_epilogue{data(bias), bias ? c.dtype(*bias) : 0, static_cast<int>(act), gated ? 1 : 0, data(residual)};
}

// x, packed, bias, activation code, gated, residual
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) return nullptr;
    Call c{args};
    const at::Tensor *x = c.needed(0), *w = c.needed(1), *bias = c.tensor(2), *res = c.tensor(5);
    const int64_t act = c.integer(3);
    const bool gated = c.truth(4);
    if (!c.ok || x->dim() != 2 || w->dim() != 2 || w->scalar_type() != at::kByte) return nullptr;
    const int64_t rows = w->size(0), k = w->size(1) / Q4_BLOCK_BYTES * Q4_QK, m = x->size(0);
    c.want(w->size(1) % Q4_BLOCK_BYTES == 0 && x->size(1) == k && (!gated || rows % 2 == 0));
    c.shape(bias, {rows});
    const int64_t nout = gated ? rows / 2 : rows;
    c.shape(res, {m, nout});
    const int xd = c.dtype(*x);
    c.want(res == nullptr || res->scalar_type() == x->scalar_type());
    const q4_epilogue ep = epilogue(c, bias, act, gated, res);
    if (!c.ready()) return nullptr;
    at::Tensor y = at::empty({m, nout}, x->options()), ws;
    const size_t need = p_linear_ws(m, rows, k, xd, ep.gated);
    if (need > 0) ws = bytes(*x, need);
    if (p_linear(x->const_data_ptr(), xd, w->const_data_ptr(), &ep, y.mutable_data_ptr(), xd, m, rows, k,
                 need > 0 ? ws.mutable_data_ptr() : nullptr, need, c.stream()) != Q4_OK)
      return nullptr;
    return THPVariable_Wrap(y);
  });
}

bool routing(Call& c, int at, const at::Tensor* bias, int64_t experts, q4_routing* r) {
  // score, groups, group_topk, group_score, renormalise, scale from args[at]
  r->score = static_cast<int>(c.integer(at));
  r->groups = static_cast<int>(c.integer(at + 1));
  r->group_topk = static_cast<int>(c.integer(at + 2));
  r->group_score = static_cast<int>(c.integer(at + 3));
  r->renormalise = c.truth(at + 4) ? 1 : 0;
  c.want(PyFloat_Check(c.args[at + 5]));
  if (!c.ok) return false;
  r->scale = static_cast<float>(PyFloat_AS_DOUBLE(c.args[at + 5]));
  c.want(bias == nullptr || bias->scalar_type() == at::kFloat);
  c.shape(bias, {experts});
  r->bias = static_cast<const float*>(data(bias));
  return c.ok;
}

// logits, topk, bias, then a routing -> (ids, weights, plan words)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) return nullptr;
    Call c{args};
    const at::Tensor *l = c.needed(0), *bias = c.tensor(2);
    const int64_t topk = c.integer(1);
    if (!c.ok || l->dim() != 2) return nullptr;
    const int64_t m = l->size(0), experts = l->size(1);
    q4_routing r;
    if (!routing(c, 3, bias, experts, &r)) return nullptr;
    const int ld = c.dtype(*l);
    const size_t size = p_plan_size(m, topk, experts);
    c.want(size > 0);
    if (!c.ready()) return nullptr;
    const auto ints = l->options().dtype(at::kInt);
    at::Tensor ids = at::empty({m, topk}, ints), weights = at::empty({m, topk}, l->options().dtype(at::kFloat));
    at::Tensor plan = at::empty({static_cast<int64_t>(size / 4)}, ints);
    if (p_route(l->const_data_ptr(), ld, m, experts, topk, &r, static_cast<int32_t*>(ids.mutable_data_ptr()),
                static_cast<float*>(weights.mutable_data_ptr()), plan.mutable_data_ptr(), c.stream()) != Q4_OK)
      return nullptr;
    PyObject* t = PyTuple_New(3);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(ids));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(weights));
    PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(plan));
    return t;
  });
}

// ids, experts -> plan words
PyObject* route_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 2) return nullptr;
    Call c{args};
    const at::Tensor* ids = c.needed(0);
    const int64_t experts = c.integer(1);
    if (!c.ok || ids->dim() != 2 || ids->scalar_type() != at::kInt) return nullptr;
    const int64_t m = ids->size(0), topk = ids->size(1);
    const size_t size = p_plan_size(m, topk, experts);
    c.want(size > 0);
    if (!c.ready()) return nullptr;
    at::Tensor plan = at::empty({static_cast<int64_t>(size / 4)}, ids->options());
    if (p_route_plan(static_cast<const int32_t*>(ids->const_data_ptr()), m, topk, experts, plan.mutable_data_ptr(),
                     c.stream()) != Q4_OK)
      return nullptr;
    return THPVariable_Wrap(plan);
  });
}

// Experts, rows and k of packed [experts, rows, k / 32 * 18].
bool expert_shape(Call& c, const at::Tensor& w, int64_t* e, int64_t* rows, int64_t* k) {
  c.want(w.dim() == 3 && w.scalar_type() == at::kByte && w.size(2) % Q4_BLOCK_BYTES == 0);
  if (!c.ok) return false;
  *e = w.size(0);
  *rows = w.size(1);
  *k = w.size(2) / Q4_BLOCK_BYTES * Q4_QK;
  return true;
}

// x, packed, plan words, m, topk, experts, bias, activation code, gated, weights, residual
PyObject* experts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11) return nullptr;
    Call c{args};
    const at::Tensor *x = c.needed(0), *w = c.needed(1), *plan = c.needed(2), *bias = c.tensor(6);
    const at::Tensor *weights = c.tensor(9), *res = c.tensor(10);
    const int64_t m = c.integer(3), topk = c.integer(4), ne = c.integer(5), act = c.integer(7);
    const bool gated = c.truth(8);
    int64_t e, rows, k;
    if (!c.ok || x->dim() != 2 || !expert_shape(c, *w, &e, &rows, &k)) return nullptr;
    const int64_t xr = x->size(0), nout = gated ? rows / 2 : rows, yr = weights ? m : m * topk;
    c.want(e == ne && x->size(1) == k && (xr == m || xr == m * topk) && (!gated || rows % 2 == 0));
    c.want(plan->scalar_type() == at::kInt &&
           static_cast<size_t>(plan->numel()) * 4 == p_plan_size(m, topk, ne));
    c.shape(bias, {e, rows});
    c.shape(weights, {m, topk});
    c.want(weights == nullptr || weights->scalar_type() == at::kFloat);
    c.shape(res, {yr, nout});
    c.want(res == nullptr || res->scalar_type() == x->scalar_type());
    const int xd = c.dtype(*x);
    const q4_epilogue ep = epilogue(c, bias, act, gated, res);
    if (!c.ready()) return nullptr;
    at::Tensor y = at::empty({yr, nout}, x->options()), ws;
    const size_t need = p_experts_ws(m, topk, e, rows, k, xr, xd, ep.gated, weights != nullptr);
    if (need > 0) ws = bytes(*x, need);
    if (p_experts(x->const_data_ptr(), xd, xr, w->const_data_ptr(), &ep, plan->const_data_ptr(),
                  static_cast<const float*>(data(weights)), y.mutable_data_ptr(), xd, m, topk, e, rows, k,
                  need > 0 ? ws.mutable_data_ptr() : nullptr, need, c.stream()) != Q4_OK)
      return nullptr;
    return THPVariable_Wrap(y);
  });
}

// x, logits, up, down, topk, activation code, gated, up_bias, down_bias, residual, route_bias, then a routing
PyObject* moe(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 17) return nullptr;
    Call c{args};
    const at::Tensor *x = c.needed(0), *l = c.needed(1), *up = c.needed(2), *down = c.needed(3);
    const int64_t topk = c.integer(4), act = c.integer(5);
    const bool gated = c.truth(6);
    const at::Tensor *ub = c.tensor(7), *db = c.tensor(8), *res = c.tensor(9), *rb = c.tensor(10);
    int64_t e, nup, hidden, e2, n2, inter;
    if (!c.ok || x->dim() != 2 || l->dim() != 2 || !expert_shape(c, *up, &e, &nup, &hidden) ||
        !expert_shape(c, *down, &e2, &n2, &inter))
      return nullptr;
    const int64_t m = x->size(0);
    c.want(e2 == e && n2 == hidden && nup == (gated ? 2 * inter : inter) && x->size(1) == hidden);
    c.shape(l, {m, e});
    c.shape(ub, {e, nup});
    c.shape(db, {e, hidden});
    c.shape(res, {m, hidden});
    c.want(res == nullptr || res->scalar_type() == x->scalar_type());
    q4_routing r;
    if (!c.ok || !routing(c, 11, rb, e, &r)) return nullptr;
    const int xd = c.dtype(*x), ld = c.dtype(*l);
    const q4_epilogue uep = epilogue(c, ub, act, gated, nullptr), dep = epilogue(c, db, Q4_ACT_NONE, false, res);
    const size_t need = c.ok ? p_moe_ws(m, topk, e, hidden, inter, xd, uep.gated) : 0;
    c.want(need > 0);
    if (!c.ready()) return nullptr;
    at::Tensor y = at::empty({m, hidden}, x->options()), ws = bytes(*x, need);
    if (p_moe(x->const_data_ptr(), xd, l->const_data_ptr(), ld, &r, up->const_data_ptr(), &uep,
              down->const_data_ptr(), &dep, y.mutable_data_ptr(), xd, m, topk, e, hidden, inter, nullptr, nullptr,
              ws.mutable_data_ptr(), need, c.stream()) != Q4_OK)
      return nullptr;
    return THPVariable_Wrap(y);
  });
}

// A cache [pages, kv heads, 2, page size / 16, 9 d] and a batch over it, from args[at]:
// cache, tables, lengths, offsets (or None).
struct CacheCall {
  q4_cache cache;
  q4_batch batch;
  const at::Tensor* data;
  bool take(Call& c, int at, int64_t tokens) {
    data = c.needed(at);
    const at::Tensor *tables = c.needed(at + 1), *lengths = c.needed(at + 2), *offsets = c.tensor(at + 3);
    if (!c.ok) return false;
    c.want(data->dim() == 5 && data->scalar_type() == at::kByte && tables->dim() == 2 && lengths->dim() == 1);
    if (!c.ok) return false;
    c.want(data->size(2) == 2 && data->size(4) % (9 * Q4_QK) == 0 && tables->scalar_type() == at::kInt &&
           lengths->scalar_type() == at::kInt && lengths->size(0) == tables->size(0));
    const int64_t seqs = tables->size(0);
    c.want(offsets ? offsets->dim() == 1 && offsets->scalar_type() == at::kInt && offsets->size(0) == seqs + 1
                   : tokens < 0 || tokens == seqs);
    if (!c.ok) return false;
    cache = q4_cache{const_cast<void*>(data->const_data_ptr()), data->size(0), data->size(3) * Q4_CACHE_GRANULE,
                     data->size(1), data->size(4) / 9};
    batch = q4_batch{seqs, tokens < 0 ? seqs : tokens, tables->size(1),
                     static_cast<const int32_t*>(tables->const_data_ptr()),
                     static_cast<const int32_t*>(lengths->const_data_ptr()),
                     offsets ? static_cast<const int32_t*>(offsets->const_data_ptr()) : nullptr};
    return true;
  }
  // Elements between the rows of t [tokens, heads, d], whose heads lie together.
  int64_t stride(Call& c, const at::Tensor& t) {
    const int64_t width = t.size(1) * cache.head_dim;
    c.want(t.size(2) == cache.head_dim && t.stride(2) == 1 && (t.size(1) == 1 || t.stride(1) == cache.head_dim));
    return t.size(0) > 1 ? t.stride(0) : width;  // (of one row it says nothing)
  }
};

// k, v, then a cache call -> True
PyObject* cache_write(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) return nullptr;
    Call c{args};
    const at::Tensor *k = c.needed(0, true), *v = c.needed(1, true);
    if (!c.ok || k->dim() != 3 || v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type()) return nullptr;
    CacheCall cc;
    if (!cc.take(c, 2, k->size(0))) return nullptr;
    c.want(k->size(1) == cc.cache.kv_heads);
    const int64_t ks = cc.stride(c, *k), vs = cc.stride(c, *v);
    const int dt = c.dtype(*k);
    cc.cache.data = cc.data->mutable_data_ptr();
    if (!c.ready() || p_cache_write(&cc.cache, &cc.batch, k->const_data_ptr(), ks, v->const_data_ptr(), vs, dt,
                                    c.stream()) != Q4_OK)
      return nullptr;
    Py_RETURN_TRUE;
  });
}

// A cache call, tokens (None: one a sequence), dtype (0, 1, 2 as in q4_dtype) -> (k, v)
PyObject* cache_read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) return nullptr;
    Call c{args};
    const bool each = args[4] == Py_None;
    const int64_t tokens = each ? -1 : c.integer(4), dt = c.integer(5);
    c.want(each ? args[3] == Py_None : tokens >= 1);
    CacheCall cc;
    if (!c.ok || dt < 0 || dt > 2 || !cc.take(c, 0, tokens) || !c.ready()) return nullptr;
    const auto options =
        cc.data->options().dtype(dt == Q4_F32 ? at::kFloat : dt == Q4_F16 ? at::kHalf : at::kBFloat16);
    at::Tensor k = at::empty({cc.batch.tokens, cc.cache.kv_heads, cc.cache.head_dim}, options), v = at::empty_like(k);
    if (p_cache_read(&cc.cache, &cc.batch, k.mutable_data_ptr(), v.mutable_data_ptr(), static_cast<int>(dt),
                     c.stream()) != Q4_OK)
      return nullptr;
    PyObject* t = PyTuple_New(2);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(v));
    return t;
  });
}

// q, then a cache call, scale (or None), causal, window, softcap, whether lse is asked -> y or (y, lse)
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10) return nullptr;
    Call c{args};
    const at::Tensor* q = c.needed(0, true);
    if (!c.ok || q->dim() != 3) return nullptr;
    CacheCall cc;
    if (!cc.take(c, 1, q->size(0))) return nullptr;
    const int64_t qs = cc.stride(c, *q), window = c.integer(7), heads = q->size(1), tokens = q->size(0);
    const bool causal = c.truth(6), with_lse = c.truth(9);
    c.want((args[5] == Py_None || PyFloat_Check(args[5])) && PyFloat_Check(args[8]));
    const int qd = c.dtype(*q);
    if (!c.ready()) return nullptr;
    const q4_attention_options options{
        static_cast<float>(args[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(cc.cache.head_dim))
                                              : PyFloat_AS_DOUBLE(args[5])),
        causal ? 1 : 0, window, static_cast<float>(PyFloat_AS_DOUBLE(args[8]))};
    at::Tensor y = at::empty({tokens, heads, cc.cache.head_dim}, q->options()), lse, ws;
    if (with_lse) lse = at::empty({tokens, heads}, q->options().dtype(at::kFloat));
    const size_t need = p_attention_ws(cc.batch.seqs, tokens, heads, cc.cache.kv_heads, cc.cache.head_dim, qd,
                                       cc.batch.offsets != nullptr);
    if (need > 0) ws = bytes(y, need);
    if (p_attention(&cc.cache, &cc.batch, &options, q->const_data_ptr(), qs, qd, heads, y.mutable_data_ptr(), qd,
                    with_lse ? static_cast<float*>(lse.mutable_data_ptr()) : nullptr,
                    need > 0 ? ws.mutable_data_ptr() : nullptr, need, c.stream()) != Q4_OK)
      return nullptr;
    if (!with_lse) return THPVariable_Wrap(y);
    PyObject* t = PyTuple_New(2);
    if (t == nullptr) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(y));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(lse));
    return t;
  });
}

// Addresses of the library's entry points, in this order.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int kAddresses = 13;
  void* p[kAddresses];
  if (n != kAddresses) {
    PyErr_SetString(PyExc_TypeError, "bind takes thirteen addresses");
    return nullptr;
  }
  for (int i = 0; i < kAddresses; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
  }
  p_linear = reinterpret_cast<decltype(p_linear)>(p[0]);
  p_linear_ws = reinterpret_cast<decltype(p_linear_ws)>(p[1]);
  p_route = reinterpret_cast<decltype(p_route)>(p[2]);
  p_route_plan = reinterpret_cast<decltype(p_route_plan)>(p[3]);
  p_plan_size = reinterpret_cast<decltype(p_plan_size)>(p[4]);
  p_experts = reinterpret_cast<decltype(p_experts)>(p[5]);
  p_experts_ws = reinterpret_cast<decltype(p_experts_ws)>(p[6]);
  p_moe = reinterpret_cast<decltype(p_moe)>(p[7]);
  p_moe_ws = reinterpret_cast<decltype(p_moe_ws)>(p[8]);
  p_cache_write = reinterpret_cast<decltype(p_cache_write)>(p[9]);
  p_cache_read = reinterpret_cast<decltype(p_cache_read)>(p[10]);
  p_attention = reinterpret_cast<decltype(p_attention)>(p[11]);
  p_attention_ws = reinterpret_cast<decltype(p_attention_ws)>(p[12]);
  Py_RETURN_NONE;
}

#define Q4_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {Q4_FAST(bind), Q4_FAST(linear), Q4_FAST(route), Q4_FAST(route_plan),
                         Q4_FAST(experts), Q4_FAST(moe), Q4_FAST(cache_write),
                         Q4_FAST(cache_read), Q4_FAST(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q4_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__q4_torch() { return PyModule_Create(&module); }
