// Native marshalling of the 8-bit serving calls for Python: the checks that
// the C ABI cannot make (it sees pointers, not tensors), the outputs, the
// scratch buffer of the stream, and the call. The calls
// take a few microseconds on the GPU; in Python this part alone took longer
// (13.5 us for a product that takes 8, 20 us for append and read).
//
// group_wise_affine_amd/qmm.py holds the functions that users call and their
// documentation.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <sstream>
#include <stdexcept>

#include "../../include/libqmm.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {   // -> ValueError
  using std::runtime_error::runtime_error;
};
struct Failed {};                       // a Python exception is set

PyObject* g_fail = nullptr;   // fail(status, message) raises the binding's error
PyObject* g_grow = nullptr;   // grow(bytes, device, stream, number of its capture or 0)
                              // -> scratch, counters zero

template <class... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream o;
  (o << ... << a);
  throw Refused(o.str());
}

[[noreturn]] void fail(int status, const char* msg) {
  PyObject* r = PyObject_CallFunction(g_fail, "is", status, msg);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, msg);
  throw Failed();
}
void check(qmm_status st) {
  if (st != QMM_OK) fail(st, qmm_last_error());
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name, int dims) {
  const Tensor& t = tensor(o, name);
  if (t.dim() != dims)
    refuse(name, " must have ", dims, " dimensions, got shape ", t.sizes());
  return t;
}
// shape, element type, packed
const Tensor& exact(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dt) {
  if (t.sizes() != shape) refuse(name, " has shape ", t.sizes(), ", expected ", shape);
  if (t.scalar_type() != dt) refuse(name, " has dtype ", t.scalar_type(), ", expected ", dt);
  if (!t.is_contiguous()) refuse(name, " must be contiguous");
  return t;
}
const Tensor& exact(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt) {
  return exact(tensor(o, name), name, shape, dt);
}
// stride of the first dimension of a tensor whose others are packed
int64_t rows(const Tensor& t, const char* name) {
  int64_t width = 1;
  for (int i = (int)t.dim() - 1; i > 0; i--) {
    if (t.size(i) != 1 && t.stride(i) != width)
      refuse(name, ": all dimensions but the first must be packed");
    width *= t.size(i);
  }
  return t.size(0) > 1 ? t.stride(0) : width;   // (one row has no next one)
}
qmm_dtype element(at::ScalarType t) {
  if (t == at::kHalf) return QMM_F16;
  if (t == at::kBFloat16) return QMM_BF16;
  fail(QMM_E_DTYPE, "only float16 and bfloat16 are supported");
}

// the device that every tensor is on (it must be the current one), and the
// stream to launch on
struct Place {
  int dev;
  hipStream_t st;
};
void on_gpu(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(name, " must be on a ROCm device, got ", t.device());
}
Place place(PyObject* stream, std::initializer_list<std::pair<const Tensor*, const char*>> ts) {
  for (auto& [t, name] : ts)
    if (t) on_gpu(*t, name);
  Place p{-1, nullptr};
  if (hipGetDevice(&p.dev) != hipSuccess) refuse("no current ROCm device");
  for (auto& [t, name] : ts)
    if (t && t->get_device() != p.dev)
      refuse(name, " is on ", t->device(), " but the current device is cuda:", p.dev);
  p.st = static_cast<hipStream_t>(PyLong_AsVoidPtr(stream));
  if (PyErr_Occurred()) throw Failed();
  return p;
}

// Scratch for calls on one stream, kept and reused as a program's workspace
// is. (The interpreter's lock is held from here until a call's launches are
// queued, so that calls of two threads on one stream do not mix.) A graph
// under capture gets its own, cleared in the graph, which goes back to the
// graph's pool in the order of the stream when the call returns.
struct Scratch {
  void* p = nullptr;
  int64_t bytes = 0;
};
Scratch scratch(int64_t need, const Place& at) {
  if (need <= 0) return {};
  // never destroyed: the allocator may be gone when the process ends
  static auto& held = *new std::map<std::pair<int, hipStream_t>, Tensor>;
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  unsigned long long id = 0;
  const bool capturing = hipStreamGetCaptureInfo(at.st, &cs, &id) == hipSuccess && cs != hipStreamCaptureStatusNone;
  Tensor* t = nullptr;
  if (!capturing) {
    t = &held[{at.dev, at.st}];
    if (t->defined() && t->numel() >= need) return {t->data_ptr(), t->numel()};
  }
  PyObject* r = PyObject_CallFunction(g_grow, "LiLK", (long long)need, at.dev,
                                      (long long)(intptr_t)at.st, capturing ? id + 1 : 0ull);
  if (!r) throw Failed();
  const Tensor fresh = THPVariable_Unpack(r);
  Py_DECREF(r);
  if (t) *t = fresh;
  return {fresh.data_ptr(), fresh.numel()};
}

// a tuple that takes over its items' references
template <class... T>
PyObject* tuple(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (!r) throw Failed();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t)), ...);
  return r;
}

bool none(PyObject* o) { return o == Py_None; }

// ------------------------------------------------------------ int8 products
// i8_quantize(x, out | None, stream)
PyObject* i8_quantize(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x", 2);
  const int64_t M = x.size(0), K = x.size(1), ld = rows(x, "x");
  const qmm_dtype dt = element(x.scalar_type());
  Tensor c, s;
  if (none(a[1])) {
    on_gpu(x, "x");
    c = at::empty({M, K}, x.options().dtype(at::kChar));
    s = at::empty({M}, x.options().dtype(at::kFloat));
  } else {
    if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 2) refuse("out must be (codes, scales)");
    c = exact(PyTuple_GET_ITEM(a[1], 0), "codes", {M, K}, at::kChar);
    s = exact(PyTuple_GET_ITEM(a[1], 1), "scales", {M}, at::kFloat);
  }
  const Place p = place(a[2], {{&x, "x"}, {&c, "codes"}, {&s, "scales"}});
  check(qmm_i8_quantize(x.data_ptr(), ld, dt, M, K, static_cast<int8_t*>(c.data_ptr()),
                        static_cast<float*>(s.data_ptr()), p.st));
  return tuple(c, s);
}

// weight side of both products: wq, sw, bias | None, out | None
struct Layer {
  const Tensor *wq, *sw, *bias;
  Tensor out;
  int64_t N;
};
Layer layer(const Tensor& x, int64_t M, int64_t K, at::ScalarType dt, PyObject* wq, PyObject* sw,
            PyObject* bias, PyObject* out) {
  Layer l{};
  l.wq = &tensor(wq, "wq", 2);
  l.N = l.wq->size(0);
  exact(*l.wq, "wq", {l.N, K}, at::kChar);
  l.sw = &exact(sw, "sw", {l.N}, at::kFloat);
  if (!none(bias)) l.bias = &exact(bias, "bias", {l.N}, dt);
  if (none(out)) {
    on_gpu(x, "x");
    l.out = at::empty({M, l.N}, x.options().dtype(dt));
  } else {
    l.out = exact(out, "out", {M, l.N}, dt);
  }
  return l;
}
const float* floats(const Tensor& t) { return static_cast<const float*>(t.data_ptr()); }
const int8_t* codes(const Tensor& t) { return static_cast<const int8_t*>(t.data_ptr()); }
const int32_t* ints(const Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
int32_t* ints_out(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// i8_t(xq, sx, wq, sw, bias | None, bf16, out | None, stream)
PyObject* i8_t(PyObject* const* a) {
  const Tensor& xq = tensor(a[0], "xq", 2);
  const int64_t M = xq.size(0), K = xq.size(1);
  exact(xq, "xq", {M, K}, at::kChar);
  const Tensor& sx = exact(a[1], "sx", {M}, at::kFloat);
  const at::ScalarType st = PyObject_IsTrue(a[5]) ? at::kBFloat16 : at::kHalf;
  const Layer l = layer(xq, M, K, st, a[2], a[3], a[4], a[6]);
  const Place p = place(a[7], {{&xq, "xq"}, {&sx, "sx"}, {l.wq, "wq"}, {l.sw, "sw"}, {l.bias, "bias"}, {&l.out, "out"}});
  const Scratch w = scratch(qmm_i8_t_work(M, l.N, K), p);
  check(qmm_i8_t(codes(xq), floats(sx), codes(*l.wq), floats(*l.sw), l.bias ? l.bias->data_ptr() : nullptr,
                 element(st), M, l.N, K, l.out.data_ptr(), w.p, w.bytes, p.st));
  return THPVariable_Wrap(l.out);
}

// i8_linear(x, wq, sw, bias | None, out | None, stream)
PyObject* i8_linear(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x", 2);
  const int64_t M = x.size(0), K = x.size(1), ld = rows(x, "x");
  const qmm_dtype dt = element(x.scalar_type());
  const Layer l = layer(x, M, K, x.scalar_type(), a[1], a[2], a[3], a[4]);
  const Place p = place(a[5], {{&x, "x"}, {l.wq, "wq"}, {l.sw, "sw"}, {l.bias, "bias"}, {&l.out, "out"}});
  const Scratch w = scratch(qmm_i8_linear_work(M, l.N, K), p);
  check(qmm_i8_linear(x.data_ptr(), ld, codes(*l.wq), floats(*l.sw), l.bias ? l.bias->data_ptr() : nullptr, dt, M,
                      l.N, K, l.out.data_ptr(), w.p, w.bytes, p.st));
  return THPVariable_Wrap(l.out);
}

// -------------------------------------------------------------- 8-bit cache
// A cache arrives as the address of its C structure and the tuple of its four
// tensors; the Python object that owns both checked their shapes once. That
// they still lie where the structure says (a tensor can be given other memory
// in place) is checked at each call.
struct Cache {
  const qmm_kv8_cache* c;
  const Tensor* k;
};
Cache cache(PyObject* at, PyObject* held) {
  Cache c;
  c.c = static_cast<const qmm_kv8_cache*>(PyLong_AsVoidPtr(at));
  if (PyErr_Occurred()) throw Failed();
  if (!PyTuple_Check(held) || PyTuple_GET_SIZE(held) != 4) refuse("a cache has four tensors");
  const std::pair<const void*, const char*> parts[4] = {
      {c.c->k, "k"}, {c.c->v, "v"}, {c.c->k_scales, "k_scales"}, {c.c->v_scales, "v_scales"}};
  const int64_t blocks = c.c->pages * c.c->heads;
  const int64_t codes = blocks * c.c->page_tokens * c.c->head_dim;
  for (int i = 0; i < 4; i++) {
    const Tensor& t = tensor(PyTuple_GET_ITEM(held, i), parts[i].second);
    if (t.numel() != (i < 2 ? codes : blocks) || t.data_ptr() != parts[i].first)
      refuse("the cache's ", parts[i].second, " was given other memory: make a cache of the new tensors");
  }
  c.k = &tensor(PyTuple_GET_ITEM(held, 0), "cache");
  return c;
}
struct Batch {
  const Tensor *table, *lens, *cu;
  int64_t S, W;
};
Batch batch(PyObject* table, PyObject* lens, PyObject* cu) {
  Batch b{};
  b.table = &tensor(table, "table", 2);
  b.S = b.table->size(0);
  b.W = b.table->size(1);
  exact(*b.table, "table", {b.S, b.W}, at::kInt);
  if (lens) b.lens = &exact(lens, "lens", {b.S}, at::kInt);
  if (cu) b.cu = &exact(cu, "cu", {b.S + 1}, at::kInt);
  return b;
}
const Tensor& new_rows(PyObject* o, const char* name, int64_t heads, int64_t dim) {
  const Tensor& t = tensor(o, name, 3);
  if (t.size(2) != dim || (heads > 0 && t.size(1) != heads))
    refuse(name, " has shape ", t.sizes(), ", expected [tokens, ", heads > 0 ? heads : t.size(1), ", ", dim, "]");
  return t;
}

// kv8_append(cache, its tensors, k, v, table, lens, cu, stream)
PyObject* kv8_append(PyObject* const* a) {
  const Cache c = cache(a[0], a[1]);
  const Tensor& k = new_rows(a[2], "k", c.c->heads, c.c->head_dim);
  const Tensor& v = new_rows(a[3], "v", c.c->heads, c.c->head_dim);
  if (k.size(0) != v.size(0) || k.scalar_type() != v.scalar_type())
    refuse("k and v must have one shape and dtype");
  const int64_t ldk = rows(k, "k"), ldv = rows(v, "v");
  const qmm_dtype dt = element(k.scalar_type());
  const Batch b = batch(a[4], a[5], a[6]);
  const Place p = place(a[7], {{c.k, "cache"}, {&k, "k"}, {&v, "v"}, {b.table, "table"}, {b.lens, "lens"}, {b.cu, "cu"}});
  check(qmm_kv8_append(c.c, k.data_ptr(), ldk, v.data_ptr(), ldv, dt, k.size(0), ints(*b.table), ints(*b.lens),
                       ints(*b.cu), b.S, b.W, p.st));
  Py_RETURN_NONE;
}

// kv8_read(cache, its tensors, pages, bf16, stream)
PyObject* kv8_read(PyObject* const* a) {
  const Cache c = cache(a[0], a[1]);
  const Tensor& pages = tensor(a[2], "pages", 1);
  const int64_t n = pages.size(0);
  exact(pages, "pages", {n}, at::kInt);
  on_gpu(pages, "pages");
  const at::ScalarType st = PyObject_IsTrue(a[3]) ? at::kBFloat16 : at::kHalf;
  const auto options = pages.options().dtype(st);
  const Tensor k = at::empty({n, c.c->heads, c.c->page_tokens, c.c->head_dim}, options);
  const Tensor v = at::empty({n, c.c->heads, c.c->page_tokens, c.c->head_dim}, options);
  const Place p = place(a[4], {{c.k, "cache"}, {&pages, "pages"}});
  check(qmm_kv8_read(c.c, ints(pages), n, element(st), k.data_ptr(), v.data_ptr(), p.st));
  return tuple(k, v);
}

// What the calls of the attention have in common: arguments (cache, its tensors,
// q, table, lens, cu, the mask's own, scale | None, out | None, lse wanted, stream),
// of which `rest` are those from the scale on. work() says the scratch bytes, go()
// makes the call.
struct Queries {
  Cache c;
  const Tensor& q;
  int64_t T, H, ld;
  qmm_dtype dt;
  Batch b;
};
Queries queries(PyObject* const* a) {
  const Cache c = cache(a[0], a[1]);
  const Tensor& q = new_rows(a[2], "q", 0, c.c->head_dim);
  const int64_t ld = rows(q, "q");
  return {c, q, q.size(0), q.size(1), ld, element(q.scalar_type()), batch(a[3], a[4], a[5])};
}
template <class Work, class Go>
PyObject* attention(const Queries& x, PyObject* const* rest, const Tensor* parent, Work work, Go go) {
  const int64_t D = x.q.size(2);
  double scale = 1.0 / std::sqrt((double)D);
  if (!none(rest[0])) {
    scale = PyFloat_AsDouble(rest[0]);
    if (PyErr_Occurred()) throw Failed();
  }
  Tensor out, lse;
  if (none(rest[1])) {
    on_gpu(x.q, "q");
    out = at::empty({x.T, x.H, D}, x.q.options());
  } else {
    out = exact(rest[1], "out", {x.T, x.H, D}, x.q.scalar_type());
  }
  const bool want = PyObject_IsTrue(rest[2]);
  const Place p = place(rest[3], {{x.c.k, "cache"}, {&x.q, "q"}, {x.b.table, "table"}, {x.b.lens, "lens"}, {x.b.cu, "cu"}, {parent, "parent"}, {&out, "out"}});
  if (want) lse = at::empty({x.T, x.H}, x.q.options().dtype(at::kFloat));
  const Scratch w = scratch(work(), p);
  check(go((float)scale, out.data_ptr(), want ? static_cast<float*>(lse.data_ptr()) : nullptr, w, p.st));
  if (!want) return THPVariable_Wrap(out);
  return tuple(out, lse);
}

// kv8_attention(cache, its tensors, q, table, lens, cu, scale | None, out | None, lse wanted, stream)
PyObject* kv8_attention(PyObject* const* a) {
  const Queries x = queries(a);
  return attention(
      x, a + 6, nullptr, [&] { return qmm_kv8_attention_work(x.c.c, x.T, x.H, x.b.S, x.b.W); },
      [&](float scale, void* out, float* lse, const Scratch& w, hipStream_t st) {
        return qmm_kv8_attention(x.c.c, x.q.data_ptr(), x.ld, x.dt, x.T, x.H, ints(*x.b.table), ints(*x.b.lens),
                                 ints(*x.b.cu), x.b.S, x.b.W, scale, out, lse, w.p, w.bytes, st);
      });
}

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) throw Failed();
  return v;
}

// kv8_attention_window(cache, its tensors, q, table, lens, cu, window, sinks, scale | None, out | None, lse wanted, stream)
PyObject* kv8_attention_window(PyObject* const* a) {
  const Queries x = queries(a);
  const int64_t window = whole(a[6]), sinks = whole(a[7]);
  return attention(
      x, a + 8, nullptr,
      [&] { return qmm_kv8_attention_window_work(x.c.c, x.T, x.H, x.b.S, x.b.W, window, sinks); },
      [&](float scale, void* out, float* lse, const Scratch& w, hipStream_t st) {
        return qmm_kv8_attention_window(x.c.c, x.q.data_ptr(), x.ld, x.dt, x.T, x.H, ints(*x.b.table),
                                        ints(*x.b.lens), ints(*x.b.cu), x.b.S, x.b.W, window, sinks, scale, out, lse,
                                        w.p, w.bytes, st);
      });
}

// kv8_attention_tree(cache, its tensors, q, table, lens, cu, parent, scale | None, out | None, lse wanted, stream)
PyObject* kv8_attention_tree(PyObject* const* a) {
  const Queries x = queries(a);
  const Tensor& parent = exact(a[6], "parent", {x.T}, at::kInt);
  return attention(
      x, a + 7, &parent, [&] { return qmm_kv8_attention_tree_work(x.c.c, x.T, x.H, x.b.S, x.b.W); },
      [&](float scale, void* out, float* lse, const Scratch& w, hipStream_t st) {
        return qmm_kv8_attention_tree(x.c.c, x.q.data_ptr(), x.ld, x.dt, x.T, x.H, ints(*x.b.table), ints(*x.b.lens),
                                      ints(*x.b.cu), x.b.S, x.b.W, ints(parent), scale, out, lse, w.p, w.bytes, st);
      });
}

// --------------------------------------- queries, keys and tokens of a step
// qk_norm_rope(q, k, positions, inv_freq, q_weight | None, k_weight | None, eps, interleaved, out | None, stream)
PyObject* qk_norm_rope(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q", 3);
  const Tensor& k = tensor(a[1], "k", 3);
  const int64_t T = q.size(0), D = q.size(2), Hq = q.size(1), Hk = k.size(1);
  if (k.size(0) != T || k.size(2) != D || k.scalar_type() != q.scalar_type())
    refuse("q and k must have the same tokens, head size and dtype, got ", q.sizes(), " and ", k.sizes());
  const int64_t ldq = rows(q, "q"), ldk = rows(k, "k");
  const qmm_dtype dt = element(q.scalar_type());
  const Tensor& pos = exact(a[2], "positions", {T}, at::kInt);
  const Tensor& freq = tensor(a[3], "inv_freq", 1);
  exact(freq, "inv_freq", {freq.size(0)}, at::kFloat);
  const Tensor* wq = none(a[4]) ? nullptr : &exact(a[4], "q_weight", {D}, q.scalar_type());
  const Tensor* wk = none(a[5]) ? nullptr : &exact(a[5], "k_weight", {D}, q.scalar_type());
  const double eps = PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred()) throw Failed();
  Tensor qo, ko;
  if (none(a[8])) {
    on_gpu(q, "q");
    on_gpu(k, "k");
    qo = at::empty({T, Hq, D}, q.options());
    ko = at::empty({T, Hk, D}, k.options());
  } else {
    if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 2) refuse("out must be (q, k)");
    qo = tensor(PyTuple_GET_ITEM(a[8], 0), "out[0]", 3);
    ko = tensor(PyTuple_GET_ITEM(a[8], 1), "out[1]", 3);
    if (qo.sizes() != q.sizes() || ko.sizes() != k.sizes() || qo.scalar_type() != q.scalar_type() ||
        ko.scalar_type() != q.scalar_type())
      refuse("out must have the shapes and the dtype of q and k");
  }
  const int64_t ldqo = rows(qo, "out[0]"), ldko = rows(ko, "out[1]");
  const Place p = place(a[9], {{&q, "q"}, {&k, "k"}, {&pos, "positions"}, {&freq, "inv_freq"}, {wq, "q_weight"}, {wk, "k_weight"}, {&qo, "out[0]"}, {&ko, "out[1]"}});
  check(qmm_qk_norm_rope(q.data_ptr(), ldq, k.data_ptr(), ldk, dt, T, Hq, Hk, D, ints(pos), floats(freq),
                         2 * freq.size(0), PyObject_IsTrue(a[7]), wq ? wq->data_ptr() : nullptr,
                         wk ? wk->data_ptr() : nullptr, (float)eps, qo.data_ptr(), ldqo, ko.data_ptr(), ldko, p.st));
  return tuple(qo, ko);
}

// logprobs(logits, tokens, top, stream)
PyObject* logprobs(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "logits", 2);
  const int64_t M = x.size(0), V = x.size(1), ld = rows(x, "logits"), top = whole(a[2]);
  const qmm_dtype dt = x.scalar_type() == at::kFloat ? QMM_F32 : element(x.scalar_type());
  const Tensor& tokens = exact(a[1], "tokens", {M}, at::kInt);
  if (top < 0 || top > V) refuse("top must be in [0, ", V, "], got ", top);
  on_gpu(x, "logits");
  const Place p = place(a[3], {{&x, "logits"}, {&tokens, "tokens"}});
  const auto f32 = x.options().dtype(at::kFloat);
  const Tensor lp = at::empty({M}, f32), h = at::empty({M}, f32), top_lp = at::empty({M, top}, f32);
  const Tensor ids = at::empty({M, top}, tokens.options());
  const Scratch w = scratch(qmm_logprobs_work(dt, M, V, top), p);
  check(qmm_logprobs(x.data_ptr(), ld, dt, M, V, ints(tokens), top, static_cast<float*>(lp.data_ptr()),
                     static_cast<float*>(h.data_ptr()), ints_out(ids), static_cast<float*>(top_lp.data_ptr()), w.p,
                     w.bytes, p.st));
  return tuple(lp, h, ids, top_lp);
}

// kv8_update(cache, its tensors, ref, table, lens, parent, new_lens, stream)
PyObject* kv8_update(PyObject* const* a) {
  const Cache c = cache(a[0], a[1]);
  const Batch b = batch(a[3], a[4], nullptr);
  const Tensor& ref = exact(a[2], "ref", {c.c->pages}, at::kInt);
  const Tensor& parent = exact(a[5], "parent", {b.S}, at::kInt);
  const Tensor& new_lens = exact(a[6], "new_lens", {b.S}, at::kInt);
  const Place p = place(a[7], {{c.k, "cache"}, {&ref, "ref"}, {b.table, "table"}, {b.lens, "lens"}, {&parent, "parent"}, {&new_lens, "new_lens"}});
  const Tensor ref_out = at::empty({c.c->pages}, ref.options());
  const Tensor table_out = at::empty({b.S, b.W}, ref.options());
  const Tensor shortage = at::empty({1}, ref.options());
  const Scratch w = scratch(qmm_kv8_pages_work(c.c->pages), p);
  check(qmm_kv8_update(c.c, ints(ref), ints(*b.table), ints(*b.lens), ints(parent), ints(new_lens), b.S, b.W,
                       ints_out(ref_out), ints_out(table_out), ints_out(shortage), w.p, w.bytes, p.st));
  return tuple(ref_out, table_out, shortage);
}

// kv8_compact(cache, its tensors, ref, table, stream)
PyObject* kv8_compact(PyObject* const* a) {
  const Cache c = cache(a[0], a[1]);
  const Batch b = batch(a[3], nullptr, nullptr);
  const Tensor& ref = exact(a[2], "ref", {c.c->pages}, at::kInt);
  const Place p = place(a[4], {{c.k, "cache"}, {&ref, "ref"}, {b.table, "table"}});
  const Tensor ref_out = at::empty({c.c->pages}, ref.options()), remap = at::empty({c.c->pages}, ref.options());
  const Tensor table_out = at::empty({b.S, b.W}, ref.options()), used = at::empty({1}, ref.options());
  const Scratch w = scratch(qmm_kv8_pages_work(c.c->pages), p);
  check(qmm_kv8_compact(c.c, ints(ref), ints(*b.table), b.S, b.W, ints_out(ref_out), ints_out(table_out),
                        ints_out(remap), ints_out(used), w.p, w.bytes, p.st));
  return tuple(ref_out, table_out, remap, used);
}

// kv8_copy(to, its tensors, dst, source, its tensors, src, stream)
PyObject* kv8_copy(PyObject* const* a) {
  const Cache to = cache(a[0], a[1]), from = cache(a[3], a[4]);
  const Tensor& dst = tensor(a[2], "dst", 1);
  const int64_t n = dst.size(0);
  exact(dst, "dst", {n}, at::kInt);
  const Tensor& src = exact(a[5], "src", {n}, at::kInt);
  const Place p = place(a[6], {{to.k, "to"}, {from.k, "source"}, {&dst, "dst"}, {&src, "src"}});
  check(qmm_kv8_copy(to.c, ints(dst), from.c, ints(src), n, p.st));
  Py_RETURN_NONE;
}

// set_hooks(fail, grow)
PyObject* set_hooks(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  g_fail = a[0];
  g_grow = a[1];
  Py_RETURN_NONE;
}

// no C++ exception leaves the module
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %d", N, (int)n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Failed&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
#define QMM_ENTRY(f, n) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    QMM_ENTRY(set_hooks, 2),  QMM_ENTRY(i8_quantize, 3),   QMM_ENTRY(i8_t, 8),
    QMM_ENTRY(i8_linear, 6),  QMM_ENTRY(kv8_append, 8),    QMM_ENTRY(kv8_read, 5),
    QMM_ENTRY(kv8_attention, 10), QMM_ENTRY(kv8_update, 8), QMM_ENTRY(kv8_compact, 5),
    QMM_ENTRY(kv8_copy, 7),   QMM_ENTRY(kv8_attention_window, 12),
    QMM_ENTRY(kv8_attention_tree, 11), QMM_ENTRY(qk_norm_rope, 10), QMM_ENTRY(logprobs, 4),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
