// serve_bind.cpp -- torch argument marshalling of the serving entry points.
//
// The serving kernels take a few microseconds and are called in a generation
// loop, where reading a dozen tensors' shapes and strides through the
// interpreter takes longer than the kernel.  This module does what the ctypes
// binding does for the attention calls -- check tensors, fill the C ABI's
// descriptors, allocate outputs that were not given, call the entry point on
// the current stream, raise on a status -- in C++.  All arithmetic is in the
// library.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <stdexcept>
#include <string>

#include "sdpa_serve.h"

namespace {

// Python's ValueError, TypeError or SdpaError (status >= 0).
struct Refusal {
  std::string text;
  int status = -1;
};

[[noreturn]] void refuse(const std::string& text) { throw Refusal{text}; }

void check(sdpa_status_t st, const char* where) {
  if (st != SDPA_OK) throw Refusal{where, static_cast<int>(st)};
}

// One argument as a tensor; null where it is None.
const at::Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& need(PyObject* o, const char* name) {
  const at::Tensor* t = opt(o, name);
  if (!t) refuse(std::string(name) + " must be a tensor");
  return *t;
}
int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  return v;
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return v;
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a bool");
  }
  return v != 0;
}

// Every tensor on one GPU, the current one; its current stream.
void* stream_of(std::initializer_list<const at::Tensor*> ts) {
  int dev = -1;
  for (const at::Tensor* t : ts) {
    if (!t) continue;
    if (!t->is_cuda()) refuse("tensors must be on a CUDA device");
    if (dev < 0) dev = t->get_device();
    else if (dev != t->get_device()) refuse("tensors are on different CUDA devices");
  }
  if (dev != c10::cuda::current_device())
    refuse("tensors are on cuda:" + std::to_string(dev) + ", which is not the current CUDA device");
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

// The stride of dimension i; 8 where it is never stepped along (any number
// would do, and the library asks for a multiple of 8).
int64_t step(const at::Tensor& t, int64_t i) { return t.size(i) == 1 ? 8 : t.stride(i); }

void rows(const at::Tensor& t, const char* name, int64_t dims) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != dims || (t.stride(dims - 1) != 1 && t.size(dims - 1) != 1))
    refuse(std::string(name) + " must be bf16 with " + std::to_string(dims) +
           " dimensions and a contiguous head_dim");
}
void shaped(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) refuse(std::string(name) + " has a wrong shape");
}
// As the tensor it goes with, strides included (where they matter).
void alike(const at::Tensor& t, const char* name, const at::Tensor& ref) {
  rows(t, name, ref.dim());
  shaped(t, name, ref.sizes());
  for (int64_t i = 0; i < ref.dim(); ++i)
    if (step(t, i) != step(ref, i)) refuse(std::string(name) + " must have the strides of its partner");
}
template <typename T>
T* vec(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
    refuse(std::string(name) + " must be contiguous, of the type and shape that the call asks for");
  return static_cast<T*>(t.data_ptr());
}

// An output of a call whose arguments are on the GPU (straight from the
// allocator: the dispatcher would take as long as a kernel's launch).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), at::MemoryFormat::Contiguous);
}

struct Cache {
  const at::Tensor *k, *v, *ks, *vs;
  sdpa_kv_cache c{};
  // args: k_cache, v_cache, k_scale, v_scale
  explicit Cache(PyObject* const* a)
      : k(&need(a[0], "k_cache")), v(&need(a[1], "v_cache")), ks(opt(a[2], "k_scale")), vs(opt(a[3], "v_scale")) {
    const at::ScalarType dt = k->scalar_type();
    const bool e4m3 = dt == at::kFloat8_e4m3fn;
    if (!e4m3 && dt != at::kBFloat16) refuse("a cache is bf16 or float8_e4m3fn");
    if (k->dim() != 4 || v->sizes() != k->sizes() || v->scalar_type() != dt || v->strides() != k->strides() ||
        k->stride(3) != 1)
      refuse("k_cache and v_cache must be [num_pages, Hkv, page_size, d] alike in type, shape and strides, "
             "with a contiguous head_dim");
    c.k = k->data_ptr();
    c.v = v->data_ptr();
    c.format = e4m3 ? SDPA_CACHE_E4M3 : SDPA_CACHE_BF16;
    c.num_pages = k->size(0);
    c.Hkv = k->size(1);
    c.page_size = k->size(2);
    c.d = k->size(3);
    // (16: as `step`, for a dimension of one)
    c.stride_page = k->size(0) == 1 ? 16 : k->stride(0);
    c.stride_head = k->size(1) == 1 ? 16 : k->stride(1);
    c.stride_row = k->size(2) == 1 ? 16 : k->stride(2);
    if (e4m3) {
      if (!ks || !vs) refuse("an e4m3 cache needs k_scale and v_scale");
      const auto sh = k->sizes().slice(0, 3);
      if (ks->scalar_type() != at::kByte || vs->scalar_type() != at::kByte || ks->sizes() != sh || vs->sizes() != sh ||
          ks->stride(2) != 1 || vs->strides() != ks->strides())
        refuse("k_scale and v_scale must be uint8 [num_pages, Hkv, page_size] alike in strides, with contiguous rows");
      c.k_scale = ks->data_ptr<uint8_t>();
      c.v_scale = vs->data_ptr<uint8_t>();
      c.scale_stride_page = ks->size(0) == 1 ? 16 : ks->stride(0);
      c.scale_stride_head = ks->size(1) == 1 ? 16 : ks->stride(1);
    } else if (ks || vs) {
      refuse("a bf16 cache has no scales");
    }
  }
};

struct Table {
  const at::Tensor& t;
  int64_t width, step_b;
  Table(PyObject* o, int64_t B) : t(need(o, "page_table")) {
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != B || (t.size(1) > 1 && t.stride(1) != 1))
      refuse("page_table must be int32 [B, pages] with contiguous rows");
    width = t.size(1);
    step_b = B > 1 ? t.stride(0) : width;
  }
  const int32_t* data() const { return t.data_ptr<int32_t>(); }
};

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = Py_None;
    if (t.defined()) o = THPVariable_Wrap(t);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// q, k, freqs, positions, out_q, out_k, offset, interleaved, inverse, amplitude
PyObject* rope(PyObject* const* a) {
  const at::Tensor& q = need(a[0], "q");
  const at::Tensor* k = opt(a[1], "k");
  const at::Tensor& freqs = need(a[2], "freqs");
  const at::Tensor* pos = opt(a[3], "positions");
  const at::Tensor *gq = opt(a[4], "out_q"), *gk = opt(a[5], "out_k");
  const int64_t dims = q.dim();
  if (dims != 3 && dims != 4) refuse("q must be [B, L, Hq, d] or [T, Hq, d]");
  void* stream = stream_of({&q, k, &freqs, pos, gq, gk});
  rows(q, "q", dims);
  const bool packed = dims == 3;
  sdpa_rope_desc r{};
  r.B = packed ? 1 : q.size(0);
  r.L = q.size(dims - 3);
  r.Hq = q.size(dims - 2);
  r.d = q.size(dims - 1);
  if (freqs.scalar_type() != at::kDouble || freqs.dim() != 1 || !freqs.is_contiguous())
    refuse("freqs must be a contiguous float64 vector");
  if (pos) {
    if (pos->scalar_type() != at::kInt || pos->sizes() != q.sizes().slice(0, dims - 2))
      refuse("positions must be int32 [B, L] (packed: [T])");
    if (r.L > 1 && pos->stride(dims - 3) != 1) refuse("positions must be contiguous along the sequence");
    r.positions = pos->data_ptr<int32_t>();
  }
  r.pos_b = pos && r.B > 1 ? pos->stride(0) : r.L;
  const at::Tensor oq = gq ? *gq : fresh(q.sizes(), at::kBFloat16, q);
  rows(oq, "out_q", dims);
  shaped(oq, "out_q", q.sizes());
  auto strides = [&](const at::Tensor& t, int64_t& b, int64_t& l, int64_t& h) {
    b = packed ? 8 : step(t, 0);
    l = step(t, dims - 3);
    h = step(t, dims - 2);
  };
  strides(q, r.q_b, r.q_l, r.q_h);
  strides(oq, r.qo_b, r.qo_l, r.qo_h);
  at::Tensor ok;
  if (k) {
    rows(*k, "k", dims);
    for (int64_t i = 0; i < dims; ++i)
      if (i != dims - 2 && k->size(i) != q.size(i)) refuse("k's shape does not match q's");
    ok = gk ? *gk : fresh(k->sizes(), at::kBFloat16, q);
    rows(ok, "out_k", dims);
    shaped(ok, "out_k", k->sizes());
    strides(*k, r.k_b, r.k_l, r.k_h);
    strides(ok, r.ko_b, r.ko_l, r.ko_h);
    r.Hkv = k->size(dims - 2);
  }
  if (r.B != 0 && r.L != 0) {
    r.offset = integer(a[6], "offset");
    r.freqs = freqs.data_ptr<double>();
    r.rot = static_cast<int32_t>(std::min<int64_t>(2 * freqs.numel(), 1 << 20));
    r.interleaved = truth(a[7], "interleaved");
    r.inverse = truth(a[8], "inverse");
    r.amplitude = static_cast<float>(number(a[9], "amplitude"));
    check(sdpa_rope(&r, q.data_ptr(), k ? k->data_ptr() : nullptr, oq.data_ptr(), k ? ok.data_ptr() : nullptr, stream),
          "sdpa_rope");
  }
  return tuple({oq, ok});
}

// k_cache, v_cache, k_scale, v_scale, k, v, slots
PyObject* append(PyObject* const* a) {
  const Cache cache(a);
  const at::Tensor &k = need(a[4], "k"), &v = need(a[5], "v"), &slots = need(a[6], "slots");
  void* stream = stream_of({cache.k, cache.v, cache.ks, cache.vs, &k, &v, &slots});
  rows(k, "k", 3);
  rows(v, "v", 3);
  shaped(v, "v", k.sizes());
  const int64_t T = k.size(0);
  if (k.size(1) != cache.c.Hkv || k.size(2) != cache.c.d) refuse("k does not fit the cache's heads");
  const int64_t* at = vec<int64_t>(slots, "slots", at::kLong, {T});
  const bool alike = step(k, 0) == step(v, 0) && step(k, 1) == step(v, 1);
  // (two calls: what the second would refuse is refused before the first)
  if (!alike && (reinterpret_cast<uintptr_t>(v.data_ptr()) % 16 || step(v, 0) <= 0 || step(v, 0) % 8 ||
                 step(v, 1) <= 0 || step(v, 1) % 8))
    check(SDPA_ERR_INVALID_ARG, "sdpa_cache_append");
  check(sdpa_cache_append(&cache.c, k.data_ptr(), alike ? v.data_ptr() : nullptr, T, step(k, 0), step(k, 1), at, stream),
        "sdpa_cache_append");
  if (!alike) {  // V by itself, as the K of its part of the cache
    sdpa_kv_cache values = cache.c;
    values.k = cache.c.v;
    values.k_scale = cache.c.v_scale;
    check(sdpa_cache_append(&values, v.data_ptr(), nullptr, T, step(v, 0), step(v, 1), at, stream), "sdpa_cache_append");
  }
  Py_RETURN_NONE;
}

// k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens, total, k, v
PyObject* gather(PyObject* const* a) {
  const Cache cache(a);
  const at::Tensor& cu = need(a[5], "cu_seqlens");
  const at::Tensor *gk = opt(a[7], "k"), *gv = opt(a[8], "v");
  const int64_t B = cu.numel() - 1;
  const Table table(a[4], B);
  void* stream = stream_of({cache.k, cache.v, cache.ks, cache.vs, &table.t, &cu, gk, gv});
  const int32_t* cup = vec<int32_t>(cu, "cu_seqlens", at::kInt, {B + 1});
  const int64_t total = integer(a[6], "total");
  if (total < 0) refuse("total must not be negative");
  const int64_t shape[] = {total, cache.c.Hkv, cache.c.d};
  const at::Tensor k = gk ? *gk : fresh(shape, at::kBFloat16, *cache.k);
  const at::Tensor v = gv ? *gv : fresh(shape, at::kBFloat16, *cache.k);
  rows(k, "k", 3);
  shaped(k, "k", shape);
  alike(v, "v", k);
  check(sdpa_cache_gather(&cache.c, B, table.data(), table.width, table.step_b, cup, total, k.data_ptr(), v.data_ptr(),
                          step(k, 0), step(k, 1), stream),
        "sdpa_cache_gather");
  return tuple({k, v});
}

// k_cache, v_cache, k_scale, v_scale, q, page_table, ctx_lens, cu_nodes,
// max_nodes, tree_mask, window_left, t5_table, t5_num_buckets,
// t5_max_distance, t5_bidirectional, alibi_slopes, scale, out, lse, workspace,
// size_only
PyObject* tree(PyObject* const* a) {
  const Cache cache(a);
  const at::Tensor &q = need(a[4], "q"), &ctx = need(a[6], "ctx_lens"), &cu = need(a[7], "cu_nodes");
  const at::Tensor *mask = opt(a[9], "tree_mask"), *t5 = opt(a[11], "t5_table"), *slopes = opt(a[15], "alibi_slopes");
  const at::Tensor *go = opt(a[17], "out"), *gl = opt(a[18], "lse"), *gw = opt(a[19], "workspace");
  const int64_t B = ctx.numel();
  const Table table(a[5], B);
  void* stream =
      stream_of({cache.k, cache.v, cache.ks, cache.vs, &q, &table.t, &ctx, &cu, mask, t5, slopes, go, gl, gw});
  rows(q, "q", 3);
  sdpa_tree t{};
  t.B = B;
  t.T = q.size(0);
  t.Hq = q.size(1);
  if (q.size(2) != cache.c.d) refuse("q and the cache differ in head_dim");
  t.max_nodes = integer(a[8], "max_nodes");
  t.cu_nodes = vec<int32_t>(cu, "cu_nodes", at::kInt, {B + 1});
  t.ctx_lens = vec<int32_t>(ctx, "ctx_lens", at::kInt, {B});
  t.page_table = table.data();
  t.table_width = table.width;
  t.table_b = table.step_b;
  if (mask) t.tree_mask = vec<int64_t>(*mask, "tree_mask", at::kLong, {t.T});
  t.window_left = integer(a[10], "window_left");
  t.q_t = step(q, 0);
  t.q_h = step(q, 1);
  if (a[20] == Py_True) {
    t.o_t = t.q_t;
    t.o_h = t.q_h;
    return PyLong_FromSize_t(sdpa_tree_fwd_workspace_size(&t, &cache.c));
  }
  const at::Tensor o = go ? *go : fresh(q.sizes(), at::kBFloat16, q);
  rows(o, "out", 3);
  shaped(o, "out", q.sizes());
  t.o_t = step(o, 0);
  t.o_h = step(o, 1);
  const at::Tensor lse = gl ? *gl : fresh({t.Hq, t.T}, at::kFloat, q);
  float* lp = vec<float>(lse, "lse", at::kFloat, {t.Hq, t.T});
  sdpa_bias_desc bias{};
  if (t5 && slopes) refuse("give one of a T5 table and ALiBi slopes");
  if (t5) {
    bias.kind = SDPA_BIAS_T5;
    const int64_t nb = integer(a[12], "t5_num_buckets");
    bias.ptr = vec<float>(*t5, "t5_table", at::kFloat, {nb, t.Hq});
    bias.num_buckets = static_cast<int32_t>(nb);
    bias.max_distance = static_cast<int32_t>(std::clamp<int64_t>(integer(a[13], "t5_max_distance"), 0, 1 << 30));
    bias.bidirectional = truth(a[14], "t5_bidirectional");
  } else if (slopes) {
    bias.kind = SDPA_BIAS_ALIBI;
    bias.ptr = vec<float>(*slopes, "alibi_slopes", at::kFloat, {t.Hq});
  }
  const at::Tensor ws = gw ? *gw
                           : fresh({static_cast<int64_t>(sdpa_tree_fwd_workspace_size(&t, &cache.c))}, at::kByte, q);
  const double scale = a[16] == Py_None ? 1.0 / std::sqrt(static_cast<double>(cache.c.d)) : number(a[16], "scale");
  check(sdpa_tree_fwd(&t, &cache.c, q.data_ptr(), &bias, static_cast<float>(scale), o.data_ptr(), lp, ws.data_ptr(),
                      ws.nbytes(), stream),
        "sdpa_tree_fwd");
  return tuple({o, lse});
}

// target, draft, tokens, parents, u_accept, u_sample
PyObject* verify(PyObject* const* a) {
  const at::Tensor& target = need(a[0], "target");
  const at::Tensor *draft = opt(a[1], "draft"), *tokens = opt(a[2], "tokens"), *parents = opt(a[3], "parents");
  const at::Tensor* ua = opt(a[4], "u_accept");
  const at::Tensor& us = need(a[5], "u_sample");
  void* stream = stream_of({&target, draft, tokens, parents, ua, &us});
  auto dist = [&](const at::Tensor& t, const char* name) {
    if (t.scalar_type() != at::kFloat || t.dim() != 3 || (t.stride(2) != 1 && t.size(2) != 1))
      refuse(std::string(name) + " must be float32 [B, N, V] with a contiguous vocabulary");
  };
  dist(target, "target");
  sdpa_verify s{};
  s.B = target.size(0);
  s.N = target.size(1);
  s.V = target.size(2);
  s.target = target.data_ptr<float>();
  s.target_b = target.stride(0);
  s.target_n = target.stride(1);
  if (draft) {
    dist(*draft, "draft");
    shaped(*draft, "draft", target.sizes());
    s.draft = draft->data_ptr<float>();
    s.draft_b = draft->stride(0);
    s.draft_n = draft->stride(1);
  }
  if (s.N > 1) {
    if (!draft || !tokens || !ua) refuse("draft, tokens and u_accept are needed when there are drafted nodes");
    s.tokens = vec<int32_t>(*tokens, "tokens", at::kInt, {s.B, s.N});
    s.u_accept = vec<float>(*ua, "u_accept", at::kFloat, {s.B, s.N});
    if (parents) s.parents = vec<int32_t>(*parents, "parents", at::kInt, {s.B, s.N});
  }
  s.u_sample = vec<float>(us, "u_sample", at::kFloat, {s.B});
  const at::Tensor path = fresh({s.B, s.N}, at::kInt, target), accepted = fresh({s.B}, at::kInt, target),
                   token = fresh({s.B}, at::kInt, target);
  check(sdpa_spec_verify(&s, path.data_ptr<int32_t>(), accepted.data_ptr<int32_t>(), token.data_ptr<int32_t>(), stream),
        "sdpa_spec_verify");
  return tuple({path, accepted, token});
}

// What a status raises, (status, where) its arguments, and what a failed
// allocation raises.
PyObject* g_error = nullptr;
PyObject* g_memory = nullptr;

PyObject* set_error(PyObject*, PyObject* classes) {
  PyObject *e, *m;
  if (!PyArg_ParseTuple(classes, "OO", &e, &m)) return nullptr;
  Py_INCREF(e);
  Py_INCREF(m);
  Py_XDECREF(g_error);
  Py_XDECREF(g_memory);
  g_error = e;
  g_memory = m;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refusal& r) {
    if (r.status < 0) {
      PyErr_SetString(PyExc_ValueError, r.text.c_str());
    } else if (PyObject* v = Py_BuildValue("(is)", r.status, r.text.c_str())) {
      PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, v);
      Py_DECREF(v);
    }
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory ? g_memory : PyExc_MemoryError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define SERVE_ENTRY(name, f, n) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {SERVE_ENTRY("rope", rope, 10),     SERVE_ENTRY("append", append, 7),
                           SERVE_ENTRY("gather", gather, 9),  SERVE_ENTRY("tree", tree, 21),
                           SERVE_ENTRY("verify", verify, 6),  {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__serve() { return PyModule_Create(&g_module); }
