// Native argument checks of the step operators' Python calls.
//
// One function per operator: it checks every tensor's type, GPU, shape and
// layout, takes their addresses and the stream, and calls the C ABI.  The
// checks read the tensors' metadata directly (about 20 ns a tensor, where the
// same checks in Python took 0.4 us, 7 of the 10 us of a call with eleven
// tensors).  Functions return the number of launches, or minus the
// spec_status code; a bad argument raises ValueError.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/spec_verify.h"

namespace {

using Shape = std::initializer_list<int64_t>;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": a tensor is wanted");
  return THPVariable_Unpack(o);
}

// The GPU of a call's first tensor.
int device_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) throw Refused(std::string(name) + " must live on the GPU");
  return t.get_device();
}

std::string text(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

void check(const at::Tensor& t, const char* name, at::ScalarType dtype, int device, Shape shape) {
  if (t.scalar_type() != dtype)
    throw Refused(std::string(name) + ": " + c10::toString(dtype) + " is wanted, not " +
                  c10::toString(t.scalar_type()));
  if (!t.is_cuda() || t.get_device() != device)
    throw Refused(std::string(name) + " lives on " + t.device().str() + ", not on cuda:" +
                  std::to_string(device));
  const c10::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want)
    throw Refused(std::string(name) + ": shape " + text(want) + " is wanted, not " + text(t.sizes()));
}

// Address of a dense tensor of this type and shape.
void* dense(PyObject* o, const char* name, at::ScalarType dtype, int device, Shape shape) {
  const at::Tensor& t = tensor(o, name);
  check(t, name, dtype, device, shape);
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  return t.data_ptr();
}
void* dense_or_none(PyObject* o, const char* name, at::ScalarType dtype, int device, Shape shape) {
  return o == Py_None ? nullptr : dense(o, name, dtype, device, shape);
}
template <typename T>
T* as(void* p) {
  return static_cast<T*>(p);
}

// Address and row stride of [rows, heads, D] with dense heads.
void* rows_of(PyObject* o, const char* name, at::ScalarType dtype, int device, int64_t rows,
              int64_t heads, int64_t D, int64_t* stride) {
  const at::Tensor& t = tensor(o, name);
  check(t, name, dtype, device, {rows, heads, D});
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D))
    throw Refused(std::string(name) + ": heads must be dense");
  *stride = rows > 1 ? t.stride(0) : heads * D;
  return t.data_ptr();
}

spec_dims dims_of(PyObject* o) {
  Py_buffer v;
  if (PyObject_GetBuffer(o, &v, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    throw Refused("dims: a SpecDims is wanted");
  }
  spec_dims d{};
  const bool ok = v.len == (Py_ssize_t)sizeof(d);
  if (ok) d = *static_cast<const spec_dims*>(v.buf);
  PyBuffer_Release(&v);
  if (!ok) throw Refused("dims: a SpecDims is wanted");
  return d;
}
at::ScalarType kv_type(const spec_dims& d) {
  return d.kv_dtype == SPEC_BF16 ? at::kBFloat16 : at::kFloat;
}

void* workspace(PyObject* o, int device, size_t* bytes) {
  const at::Tensor& t = tensor(o, "ws");
  *bytes = (size_t)t.numel();
  return dense(o, "ws", at::kByte, device, {t.numel()});
}

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused("");
  if (v < INT32_MIN || v > INT32_MAX) throw Refused("a 32-bit whole number is wanted");
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused("");
  return v;
}

// Runs `call(stream)` on the device and the given stream (an address, or None
// for the device's current one).  The call runs without the interpreter's lock:
// it may call the C ABI alone, and touches no tensor (which could throw).
template <typename F>
PyObject* launch(int device, PyObject* stream, F call) {
  void* st;
  if (stream == Py_None) {
    st = c10::cuda::getCurrentCUDAStream(device).stream();
  } else {
    st = PyLong_AsVoidPtr(stream);
    if (st == nullptr && PyErr_Occurred()) throw Refused("");
  }
  int code = 0, launches = 0;
  {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    Py_BEGIN_ALLOW_THREADS;
    code = call(st);
    launches = spec_last_launch_count();
    Py_END_ALLOW_THREADS;
  }
  return PyLong_FromLong(code == SPEC_OK ? launches : -code);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, not %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The tensors that the forms of the verify attention share.
struct AttnTensors {
  int dev;
  spec_dims d;
  void *q, *kn, *vn, *kc, *vc, *bt, *ctx, *par, *out, *lse, *ws;
  size_t bytes;
};
// q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, parent, out, lse,
// dims, ws
AttnTensors attn_tensors(PyObject* const* a) {
  AttnTensors t;
  t.dev = device_of(a[0], "q");
  t.d = dims_of(a[10]);
  const spec_dims& d = t.d;
  const auto kv = kv_type(d);
  const int64_t B = d.B, M = d.M, Hq = d.Hq, Hkv = d.Hkv, D = d.D;
  const Shape cache = {d.num_blocks, Hkv, d.block, D};
  t.q = dense(a[0], "q", kv, t.dev, {B, M, Hq, D});
  t.kn = dense(a[1], "k_new", kv, t.dev, {B, M, Hkv, D});
  t.vn = dense(a[2], "v_new", kv, t.dev, {B, M, Hkv, D});
  t.kc = dense(a[3], "k_cache", kv, t.dev, cache);
  t.vc = dense(a[4], "v_cache", kv, t.dev, cache);
  t.bt = dense(a[5], "block_table", at::kInt, t.dev, {B, d.max_blocks});
  t.ctx = dense(a[6], "ctx_lens", at::kInt, t.dev, {B});
  t.par = dense_or_none(a[7], "parent", at::kInt, t.dev, {B, M});
  t.out = dense(a[8], "out", kv, t.dev, {B, M, Hq, D});
  t.lse = dense_or_none(a[9], "lse", at::kFloat, t.dev, {B, M, Hq});
  t.ws = workspace(a[11], t.dev, &t.bytes);
  return t;
}

// the tensors of the verify attention, window, sinks, stream
PyObject* verify_attn_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const AttnTensors t = attn_tensors(a);
    const int32_t window = (int32_t)whole(a[12]), sinks = (int32_t)whole(a[13]);
    return launch(t.dev, a[14], [&](void* st) {
      return spec_verify_attn_window(t.q, t.kn, t.vn, t.kc, t.vc, as<int32_t>(t.bt),
                                     as<int32_t>(t.ctx), as<int32_t>(t.par), window, sinks, t.out,
                                     as<float>(t.lse), &t.d, t.ws, t.bytes, st);
    });
  });
}

// the tensors of the verify attention, prefix, stream
PyObject* verify_attn_prefix(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const AttnTensors t = attn_tensors(a);
    const int64_t pages = tensor(a[12], "prefix").numel();
    void* prefix = dense(a[12], "prefix", at::kInt, t.dev, {pages});
    if (pages > INT32_MAX / 16) throw Refused("prefix: too many pages");
    return launch(t.dev, a[13], [&](void* st) {
      return spec_verify_attn_prefix(t.q, t.kn, t.vn, t.kc, t.vc, as<int32_t>(t.bt),
                                     as<int32_t>(t.ctx), as<int32_t>(t.par), as<int32_t>(prefix),
                                     (int32_t)(16 * pages), t.out, as<float>(t.lse), &t.d, t.ws,
                                     t.bytes, st);
    });
  });
}

// Pages per KV head of a selection [B, Hkv, n].
int64_t selected(PyObject* o) {
  const at::Tensor& t = tensor(o, "pages");
  if (t.dim() != 3) throw Refused("pages: [B, Hkv, n] is wanted");
  if (t.size(2) > INT32_MAX) throw Refused("pages: too many");
  return t.size(2);
}

// the tensors of the verify attention, pages, page_counts, stream
PyObject* verify_attn_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const AttnTensors t = attn_tensors(a);
    const int64_t np = selected(a[12]);
    void* pages = dense(a[12], "pages", at::kInt, t.dev, {t.d.B, t.d.Hkv, np});
    void* counts = dense(a[13], "page_counts", at::kInt, t.dev, {t.d.B});
    return launch(t.dev, a[14], [&](void* st) {
      return spec_verify_attn_pages(t.q, t.kn, t.vn, t.kc, t.vc, as<int32_t>(t.bt),
                                    as<int32_t>(t.ctx), as<int32_t>(t.par), as<int32_t>(pages),
                                    as<int32_t>(counts), (int32_t)np, t.out, as<float>(t.lse), &t.d,
                                    t.ws, t.bytes, st);
    });
  });
}

// k_cache, block_table, from_lens, ctx_lens, bounds, dims, ws, stream
PyObject* page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const int dev = device_of(a[0], "k_cache");
    const spec_dims d = dims_of(a[5]);
    const auto kv = kv_type(d);
    void* kc = dense(a[0], "k_cache", kv, dev, {d.num_blocks, d.Hkv, d.block, d.D});
    void* bt = dense(a[1], "block_table", at::kInt, dev, {d.B, d.max_blocks});
    void* from = dense_or_none(a[2], "from_lens", at::kInt, dev, {d.B});
    void* ctx = dense(a[3], "ctx_lens", at::kInt, dev, {d.B});
    void* bounds = dense(a[4], "bounds", kv, dev, {d.num_blocks, d.Hkv, 2, d.D});
    size_t bytes;
    void* ws = workspace(a[6], dev, &bytes);
    return launch(dev, a[7], [&](void* st) {
      return spec_page_bounds(kc, as<int32_t>(bt), as<int32_t>(from), as<int32_t>(ctx), bounds, &d,
                              ws, bytes, st);
    });
  });
}

// q, bounds, block_table, ctx_lens, scores, dims, ws, stream
PyObject* page_score(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const int dev = device_of(a[0], "q");
    const spec_dims d = dims_of(a[5]);
    const auto kv = kv_type(d);
    void* q = dense(a[0], "q", kv, dev, {d.B, d.M, d.Hq, d.D});
    void* bounds = dense(a[1], "bounds", kv, dev, {d.num_blocks, d.Hkv, 2, d.D});
    void* bt = dense(a[2], "block_table", at::kInt, dev, {d.B, d.max_blocks});
    void* ctx = dense(a[3], "ctx_lens", at::kInt, dev, {d.B});
    void* scores = dense(a[4], "scores", at::kFloat, dev, {d.B, d.Hkv, d.max_blocks});
    size_t bytes;
    void* ws = workspace(a[6], dev, &bytes);
    return launch(dev, a[7], [&](void* st) {
      return spec_page_score(q, bounds, as<int32_t>(bt), as<int32_t>(ctx), as<float>(scores), &d, ws,
                             bytes, st);
    });
  });
}

// scores, ctx_lens, pages, page_counts, dims, ws, first, last, stream
PyObject* page_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const int dev = device_of(a[0], "scores");
    const spec_dims d = dims_of(a[4]);
    const int64_t np = selected(a[2]);
    void* scores = dense(a[0], "scores", at::kFloat, dev, {d.B, d.Hkv, d.max_blocks});
    void* ctx = dense(a[1], "ctx_lens", at::kInt, dev, {d.B});
    void* pages = dense(a[2], "pages", at::kInt, dev, {d.B, d.Hkv, np});
    void* counts = dense(a[3], "page_counts", at::kInt, dev, {d.B});
    size_t bytes;
    void* ws = workspace(a[5], dev, &bytes);
    const int32_t first = (int32_t)whole(a[6]), last = (int32_t)whole(a[7]);
    return launch(dev, a[8], [&](void* st) {
      return spec_page_select(as<float>(scores), as<int32_t>(ctx), (int32_t)np, first, last,
                              as<int32_t>(pages), as<int32_t>(counts), &d, ws, bytes, st);
    });
  });
}

// ctx_lens, row_start, parent, block_table, span, pool, pool_state, slots,
// positions, ok, dims, ws, window, sinks, stream
PyObject* block_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const int dev = device_of(a[0], "ctx_lens");
    const spec_dims d = dims_of(a[10]);
    const int64_t B = d.B, rows = tensor(a[7], "slots").numel();
    void* ctx = dense(a[0], "ctx_lens", at::kInt, dev, {B});
    void* start = dense_or_none(a[1], "row_start", at::kInt, dev, {B + 1});
    void* par = dense_or_none(a[2], "parent", at::kInt, dev, {B, d.M});
    void* bt = dense(a[3], "block_table", at::kInt, dev, {B, d.max_blocks});
    void* span = dense(a[4], "span", at::kInt, dev, {B, 2});
    void* pool = dense(a[5], "pool", at::kInt, dev, {d.num_blocks});
    void* state = dense(a[6], "pool_state", at::kInt, dev, {2});
    void* slots = dense(a[7], "slots", at::kLong, dev, {rows});
    void* pos = dense(a[8], "positions", at::kInt, dev, {rows});
    void* ok = dense_or_none(a[9], "ok", at::kInt, dev, {B});
    size_t bytes;
    void* ws = workspace(a[11], dev, &bytes);
    const int32_t window = (int32_t)whole(a[12]), sinks = (int32_t)whole(a[13]);
    if (rows > INT32_MAX) throw Refused("slots: at most 2^31 - 1 rows");
    return launch(dev, a[14], [&](void* st) {
      return spec_block_tables(as<int32_t>(ctx), as<int32_t>(start), as<int32_t>(par), (int32_t)rows,
                               window, sinks, as<int32_t>(bt), as<int32_t>(span), as<int32_t>(pool),
                               as<int32_t>(state), as<int64_t>(slots), as<int32_t>(pos),
                               as<int32_t>(ok), &d, ws, bytes, st);
    });
  });
}

// q, k, v, q_weight, k_weight, positions, inv_freq, q_out, k_out, dims, ws, eps,
// interleaved, slots, k_cache, v_cache, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    const int dev = device_of(a[0], "q");
    const spec_dims d = dims_of(a[9]);
    const auto kv = kv_type(d);
    const int64_t rows = tensor(a[5], "positions").numel(), Hq = d.Hq, Hkv = d.Hkv, D = d.D;
    const bool cached = a[13] != Py_None;
    int64_t qs = 0, ks = 0, vs = 0;
    void* q = rows_of(a[0], "q", kv, dev, rows, Hq, D, &qs);
    void* k = rows_of(a[1], "k", kv, dev, rows, Hkv, D, &ks);
    void* v = cached ? rows_of(a[2], "v", kv, dev, rows, Hkv, D, &vs) : nullptr;
    void* wq = dense_or_none(a[3], "q_weight", kv, dev, {D});
    void* wk = dense_or_none(a[4], "k_weight", kv, dev, {D});
    void* pos = dense(a[5], "positions", at::kInt, dev, {rows});
    const int64_t half = a[6] == Py_None ? 0 : tensor(a[6], "inv_freq").numel();
    void* f = dense_or_none(a[6], "inv_freq", at::kDouble, dev, {half});
    void* qo = dense(a[7], "q_out", kv, dev, {rows, Hq, D});
    void* ko = cached ? dense_or_none(a[8], "k_out", kv, dev, {rows, Hkv, D})
                      : dense(a[8], "k_out", kv, dev, {rows, Hkv, D});
    void *slots = nullptr, *kc = nullptr, *vc = nullptr;
    if (cached) {
      const Shape cache = {d.num_blocks, Hkv, d.block, D};
      slots = dense(a[13], "slots", at::kLong, dev, {rows});
      kc = dense(a[14], "k_cache", kv, dev, cache);
      vc = dense(a[15], "v_cache", kv, dev, cache);
    }
    size_t bytes;
    void* ws = workspace(a[10], dev, &bytes);
    const float eps = (float)real(a[11]);
    const int inter = PyObject_IsTrue(a[12]);
    if (inter < 0) throw Refused("");
    if (rows > INT32_MAX || half > INT32_MAX / 2) throw Refused("positions: too many rows");
    return launch(dev, a[16], [&](void* st) {
      return spec_qk_norm_rope(q, k, v, qs, ks, vs, wq, wk, eps, as<int32_t>(pos), as<double>(f),
                               (int32_t)(2 * half), inter, (int32_t)rows, qo, ko, as<int64_t>(slots),
                               kc, vc, &d, ws, bytes, st);
    });
  });
}

// logits, temperature, uniform, out_tokens, out_prob, ws, top_k, top_p, min_p,
// stream
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const int dev = device_of(a[0], "logits");
    const at::Tensor& x = tensor(a[0], "logits");
    if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
      throw Refused("logits: [rows, V] with dense rows is wanted");
    const auto type = x.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat)
      throw Refused(std::string("logits: unsupported dtype ") + c10::toString(type));
    const int64_t rows = x.size(0), V = x.size(1);
    const int64_t stride = rows > 1 ? x.stride(0) : V;
    const void* logits = x.data_ptr();
    void* T = dense(a[1], "temperature", at::kFloat, dev, {rows});
    void* u = dense(a[2], "uniform", at::kFloat, dev, {rows});
    void* tok = dense(a[3], "out_tokens", at::kInt, dev, {rows});
    void* prob = dense_or_none(a[4], "out_prob", at::kFloat, dev, {rows});
    size_t bytes;
    void* ws = workspace(a[5], dev, &bytes);
    void* k = dense_or_none(a[6], "top_k", at::kInt, dev, {rows});
    void* p = dense_or_none(a[7], "top_p", at::kFloat, dev, {rows});
    void* mp = dense_or_none(a[8], "min_p", at::kFloat, dev, {rows});
    if (rows > INT32_MAX || V > INT32_MAX) throw Refused("logits: too large");
    return launch(dev, a[9], [&](void* st) {
      return spec_sample(logits, stride, (int32_t)rows, (int32_t)V,
                         type == at::kBFloat16 ? SPEC_BF16 : SPEC_F32, as<float>(T), as<int32_t>(k),
                         as<float>(p), as<float>(mp), as<float>(u), as<int32_t>(tok),
                         as<float>(prob), ws, bytes, st);
    });
  });
}

#define SPECV_FN(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SPECV_FN(verify_attn_window), SPECV_FN(verify_attn_prefix),
                         SPECV_FN(verify_attn_pages),  SPECV_FN(block_tables),
                         SPECV_FN(qk_norm_rope),       SPECV_FN(page_bounds),
                         SPECV_FN(page_score),         SPECV_FN(page_select),
                         SPECV_FN(sample),             {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_specbind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__specbind() { return PyModule_Create(&module); }
