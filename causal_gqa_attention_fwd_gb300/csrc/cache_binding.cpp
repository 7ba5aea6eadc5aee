// cache_binding.cpp -- CPython module _cache_ext: the cache operators' argument
// checks, output allocation and C calls on PyTorch tensors, for _cache.py.
//
// A decode step's calls take 2 to 10 microseconds each on the GPU.  Checking a
// call's ten or so tensors one attribute at a time from Python and converting
// the arguments with ctypes took 13 (rotary rows) to 25 microseconds (cache
// plan) on the host of a GB300, so these entry points are native.  The C
// functions are not linked: bind() gets their addresses from the ctypes handle
// of the library that _binding has loaded.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <c10/util/accumulate.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "gqa_attn.h"

namespace {

// What a call is refused with.
struct Refused : std::runtime_error {
  PyObject* type;
  Refused(PyObject* t, const std::string& m) : std::runtime_error(m), type(t) {}
};
// A Python exception is set already.
struct Raised {};

[[noreturn]] void type_error(const std::string& m) { throw Refused(PyExc_TypeError, m); }
[[noreturn]] void value_error(const std::string& m) { throw Refused(PyExc_ValueError, m); }

struct Fns {
  decltype(&attn_cache_plan) plan;
  decltype(&attn_rope_table) rope_table;
  decltype(&attn_rope) rope, rope_bwd;
  decltype(&attn_cache_append) append;
  decltype(&attn_cache_append_fp8) append_fp8;
  decltype(&attn_cache_append_q4) append_q4;
  decltype(&attn_cache_gather_q4) gather_q4;
  decltype(&attn_decode_q4_workspace_size) decode_ws;
  decltype(&attn_decode_q4_fwd) decode;
  decltype(&attn_decode_paged_q4_fwd) decode_paged;
  decltype(&attn_cache_weights) weights;
  decltype(&attn_cache_weights_fp8) weights_fp8;
  decltype(&attn_cache_weights_q4) weights_q4;
  decltype(&attn_cache_evict) evict;
  decltype(&attn_decode_prefix_workspace_size) prefix_ws;
  decltype(&attn_decode_prefix_fwd) prefix;
  decltype(&attn_decode_paged_prefix_fwd) prefix_paged;
} g_fn{};
PyObject* g_check = nullptr;    // _binding._check(status, name)
PyObject* g_stream = nullptr;   // the device's current stream's handle

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    default: return "torch.uint8";
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// A tensor of the call, or one that does not exist (None).
at::Tensor optional(PyObject* o, const char* name) { return o == Py_None ? at::Tensor() : tensor(o, name); }

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
  return t.device().index();
}

void* address(const at::Tensor& t, const char* name, at::ScalarType type, int dev, bool contiguous = true) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + dtype_name(type) + ", got " + c10::toString(t.scalar_type()));
  if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
  if (t.device().index() != dev)
    value_error(std::string(name) + " is on cuda:" + std::to_string((int)t.device().index()) +
                ", the call's first tensor on cuda:" + std::to_string(dev));
  if (contiguous && !t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t.numel() ? t.mutable_data_ptr() : nullptr;
}
template <typename T>
T* address_of(const at::Tensor& t, const char* name, at::ScalarType type, int dev) {
  return static_cast<T*>(address(t, name, type, dev));
}

int to_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return (int)v;
}
int int_arg(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return to_int(v, name);
}
double float_arg(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int bool_arg(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}
int dim(const at::Tensor& t, int i, const char* name) { return to_int(t.size(i), name); }

// The device's current stream (a call on another one makes it current first, so
// that what it allocates is that stream's).
void* stream_of(int dev) {
  PyObject* d = PyLong_FromLong(dev);
  PyObject* h = d ? PyObject_CallOneArg(g_stream, d) : nullptr;
  Py_XDECREF(d);
  if (!h) throw Raised{};
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw Raised{};
  return p;
}

void check(attn_status st, const char* name) {
  if (st == ATTN_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, name);
  Py_XDECREF(r);
  if (!r) throw Raised{};
  throw Refused(PyExc_RuntimeError, std::string(name) + " failed");
}

at::TensorOptions on(const at::Tensor& like, at::ScalarType t) { return like.options().dtype(t).memory_format(c10::nullopt); }

// A contiguous part of `all` from an entry on, not through the dispatcher (five of them took 6 us).
at::Tensor part(const at::Tensor& all, int64_t entry, at::IntArrayRef sizes) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(entry);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}
// bf16 outputs that are missing.  Two small ones (1 MB in all) share an allocation: gathering 64 slots takes the host
// 4.2 us so, and 4.9 with two; large ones do not, so that either can be freed by itself.
void allocate(at::Tensor& a, at::IntArrayRef a_sizes, at::Tensor& b, at::IntArrayRef b_sizes, const at::Tensor& like) {
  const int64_t na = c10::multiply_integers(a_sizes), nb = c10::multiply_integers(b_sizes);
  if (!a.defined() && !b.defined() && na % 8 == 0 && na + nb <= 1 << 19) {
    const at::Tensor all = at::empty({na + nb}, on(like, at::kBFloat16));
    a = part(all, 0, a_sizes);
    b = part(all, na, b_sizes);
    return;
  }
  if (!a.defined()) a = at::empty(a_sizes, on(like, at::kBFloat16));
  if (!b.defined()) b = at::empty(b_sizes, on(like, at::kBFloat16));
}

// (B, T, H, D) of a [total, H, D] or [B, H, T, D] tensor, and its batch, token
// and head strides in elements; those of single entries are 0.
struct Tokens {
  int B, T, H, D;
};
Tokens tokens_of(const at::Tensor& x, const char* name) {
  if (x.dim() == 3) return {1, dim(x, 0, name), dim(x, 1, name), dim(x, 2, name)};
  if (x.dim() == 4) return {dim(x, 0, name), dim(x, 2, name), dim(x, 1, name), dim(x, 3, name)};
  value_error(std::string(name) + " must be [total, H, D] or [B, H, T, D]");
}
void strides_of(const at::Tensor& x, const char* name, long long* s, bool out = false) {
  const int n = (int)x.dim();
  if (x.size(n - 1) > 1 && x.stride(n - 1) != 1) value_error(std::string(name) + " must be contiguous in its last dimension");
  if (out)
    for (int i = 0; i < n; ++i)
      if (x.stride(i) == 0 && x.size(i) > 1) value_error(std::string(name) + " must not repeat its memory");
  auto of = [&](int i) { return x.size(i) > 1 ? (long long)x.stride(i) : 0LL; };
  s[0] = n == 4 ? of(0) : 0;
  s[1] = n == 4 ? of(2) : of(0);
  s[2] = of(1);
}

struct Table {
  const float* p = nullptr;
  int n = 0, R = 0;
};
Table table_arg(PyObject* o, int dev) {
  Table t;
  if (o == Py_None) return t;
  const at::Tensor& x = tensor(o, "rope_cos_sin");
  if (x.dim() != 2) value_error("rope_cos_sin must be [positions, rotary_dim]");
  t.p = address_of<const float>(x, "rope_cos_sin", at::kFloat, dev);
  t.n = dim(x, 0, "rope_cos_sin");
  t.R = dim(x, 1, "rope_cos_sin");
  if (t.n == 0) value_error("rope_cos_sin holds no position");   // its NULL would mean: no rotation
  return t;
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("wrong number of arguments");
}

PyObject* wrap2(at::Tensor a, at::Tensor b) {
  PyObject* r = PyTuple_New(2);
  if (!r) throw Raised{};
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(a)));
  PyObject* second = Py_None;
  if (b.defined()) second = THPVariable_Wrap(std::move(b));
  else Py_INCREF(second);
  PyTuple_SET_ITEM(r, 1, second);
  return r;
}

// (cache_lens, new_lens, block_table, page_size, free_pages, cursor, total_tokens, slots, positions, cu_seqlens,
//  lens_out, cursor_out)
PyObject* plan(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 12);
  const at::Tensor &lens = tensor(a[0], "cache_lens"), &add = tensor(a[1], "new_lens"), &bt = tensor(a[2], "block_table"),
                   &pages = tensor(a[4], "free_pages");
  const int dev = device_of(lens, "cache_lens");
  const int B = to_int(lens.numel(), "cache_lens");
  if (bt.dim() != 2 || bt.size(0) != B || add.numel() != B)
    value_error("cache_lens and new_lens must be [B], block_table [B, max_pages]");
  const at::Tensor cursor = optional(a[5], "cursor");
  if (cursor.defined() && cursor.numel() != 1) value_error("cursor must have one entry");
  int total;
  if (a[6] != Py_None) {
    total = int_arg(a[6], "total_tokens");
  } else {
    if (a[7] == Py_None) value_error("total_tokens (or slots) is needed: the lengths are not read on the host");
    total = to_int(tensor(a[7], "slots").numel(), "slots");
  }
  if (total < 0) value_error("total_tokens must not be negative");
  static const char* names[5] = {"slots", "positions", "cu_seqlens", "lens_out", "cursor_out"};
  const int64_t sizes[5] = {total, total, (int64_t)B + 1, B, 1};
  at::Tensor out[5];
  int* p[5];
  bool missing = false;
  for (int i = 0; i < 5; ++i) {
    out[i] = optional(a[7 + i], names[i]);
    missing |= !out[i].defined();
  }
  if (missing) {
    const at::Tensor all = at::empty({2 * (int64_t)total + 2 * (int64_t)B + 2}, on(lens, at::kInt));
    int64_t entry = 0;
    for (int i = 0; i < 5; entry += sizes[i++])
      if (!out[i].defined()) out[i] = part(all, entry, at::IntArrayRef(sizes + i, 1));
  }
  for (int i = 0; i < 5; ++i) {
    if (out[i].numel() != sizes[i])
      value_error(std::string(names[i]) + " must have " + std::to_string(sizes[i]) + " entries, got " +
                  std::to_string(out[i].numel()));
    p[i] = address_of<int>(out[i], names[i], at::kInt, dev);
  }
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  check(g_fn.plan(address_of<const int>(lens, "cache_lens", at::kInt, dev),
                  address_of<const int>(add, "new_lens", at::kInt, dev), address_of<int>(bt, "block_table", at::kInt, dev),
                  address_of<const int>(pages, "free_pages", at::kInt, dev),
                  cursor.defined() ? address_of<const int>(cursor, "cursor", at::kInt, dev) : nullptr, p[0], p[1], p[2],
                  p[3], p[4], B, int_arg(a[3], "page_size"), dim(bt, 1, "block_table"), to_int(pages.numel(), "free_pages"),
                  total, stream_of(dev)),
        "attn_cache_plan");
  PyObject* r = PyTuple_New(5);
  if (!r) throw Raised{};
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(out[i])));
  return r;
}

// (out, n, rotary_dim, base, factor, original_positions, low_turns, high_turns, mscale)
PyObject* rope_table(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  const at::Tensor& out = tensor(a[0], "out");
  const int dev = device_of(out, "out"), rows = int_arg(a[1], "n"), R = int_arg(a[2], "rotary_dim");
  if (out.dim() != 2 || out.size(0) != rows || out.size(1) != R)
    value_error("out must be [" + std::to_string(rows) + ", " + std::to_string(R) + "]");
  float* p = address_of<float>(out, "out", at::kFloat, dev);
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  check(g_fn.rope_table(p, rows, R, float_arg(a[3]), float_arg(a[4]), int_arg(a[5], "original_positions"), float_arg(a[6]),
                        float_arg(a[7]), float_arg(a[8]), stream_of(dev)),
        "attn_rope_table");
  Py_INCREF(a[0]);
  return a[0];
}

// (backward, q, k, positions, rope_cos_sin, interleaved, q_out, k_out)
PyObject* rope(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 8);
  const bool bwd = bool_arg(a[0]);
  const at::Tensor& q = tensor(a[1], "q");
  const int dev = device_of(q, "q");
  const Tokens t = tokens_of(q, "q");
  const at::Tensor k = optional(a[2], "k");
  at::Tensor qo = optional(a[6], "q_out"), ko = optional(a[7], "k_out");
  long long s[12] = {};
  int Hkv = 0;
  if (k.defined()) {
    if (k.dim() != q.dim()) value_error("k must have q's tokens and head dimension");
    const Tokens u = tokens_of(k, "k");
    if (u.B != t.B || u.T != t.T || u.D != t.D) value_error("k must have q's tokens and head dimension");
    Hkv = u.H;
    allocate(qo, q.sizes(), ko, k.sizes(), q);
    if (ko.sizes() != k.sizes()) value_error("k_out must have k's shape");
    strides_of(k, "k", s + 3);
    strides_of(ko, "k_out", s + 9, true);
  } else if (ko.defined()) {
    value_error("k_out without k");
  }
  if (!qo.defined()) qo = at::empty(q.sizes(), on(q, q.scalar_type()));
  if (qo.sizes() != q.sizes()) value_error("q_out must have q's shape");
  strides_of(q, "q", s);
  strides_of(qo, "q_out", s + 6, true);
  const at::Tensor& pos = tensor(a[3], "positions");
  int pos_stride;
  if (pos.numel() == (int64_t)t.B * t.T && (pos.dim() == 1 || (pos.dim() == 2 && pos.size(0) == t.B))) pos_stride = t.T;
  else if (pos.dim() == 1 && pos.size(0) == t.T) pos_stride = 0;
  else value_error("positions must hold one entry a token ([total], [B, T], or [T] for every batch row)");
  if (a[4] == Py_None) type_error("rope_cos_sin must be a torch.Tensor");
  const Table tab = table_arg(a[4], dev);
  const auto bf = at::kBFloat16;
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  check((bwd ? g_fn.rope_bwd : g_fn.rope)(
            address(q, "q", bf, dev, false), Hkv ? address(k, "k", bf, dev, false) : nullptr,
            address(qo, "q_out", bf, dev, false), Hkv ? address(ko, "k_out", bf, dev, false) : nullptr,
            address_of<const int>(pos, "positions", at::kInt, dev), pos_stride, tab.p, tab.n, t.B, t.T, t.H, Hkv, t.D, tab.R,
            bool_arg(a[5]), s, stream_of(dev)),
        bwd ? "attn_rope_bwd" : "attn_rope");
  return wrap2(std::move(qo), std::move(ko));
}

// (k, v, slots, caches, scales, positions, rope_cos_sin, interleaved): two caches for bf16 (no scales) and
// E4M3, four for 4 bits
PyObject* append(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 8);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots");
  const int dev = device_of(k, "k");
  const Tokens t = tokens_of(k, "k");
  if (v.sizes() != k.sizes()) value_error("v must have k's shape");
  const int nc = (int)PyTuple_GET_SIZE(a[3]);
  const bool q4 = nc == 4, bf16 = PyTuple_GET_SIZE(a[4]) == 0;
  static const char* names[3][4] = {{"k_cache", "v_cache"}, {"k8", "v8"}, {"k4", "k4_sf", "v4", "v4_sf"}};
  const char** nm = names[q4 ? 2 : bf16 ? 0 : 1];
  void* c[4];
  int pages = 0, page_size = 0;
  for (int i = 0; i < nc; ++i) {
    const at::Tensor& x = tensor(PyTuple_GET_ITEM(a[3], i), nm[i]);
    const int w = q4 ? t.D / (i & 1 ? 16 : 2) : t.D;
    if (x.dim() != 4) value_error(std::string(nm[i]) + " must be [pages, Hkv, page_size, ...]");
    if (i == 0) pages = dim(x, 0, nm[0]), page_size = dim(x, 2, nm[0]);
    if (x.size(0) != pages || x.size(1) != t.H || x.size(2) != page_size || x.size(3) != w)
      value_error(std::string(nm[i]) + " must be [pages, Hkv, page_size, " + std::to_string(w) + "] with k's heads");
    c[i] = address(x, nm[i], bf16 ? at::kBFloat16 : at::kByte, dev);
  }
  if (slots.numel() != (int64_t)t.B * t.T) value_error("slots must hold one entry a token");
  const Table tab = table_arg(a[6], dev);
  const int* pos = nullptr;
  if (a[6] != Py_None) {
    if (a[5] == Py_None) value_error("positions must hold one entry a token");
    const at::Tensor& x = tensor(a[5], "positions");
    if (x.numel() != (int64_t)t.B * t.T) value_error("positions must hold one entry a token");
    pos = address_of<const int>(x, "positions", at::kInt, dev);
  } else if (a[5] != Py_None) {
    value_error("positions without rope_cos_sin");
  }
  long long s[6];
  strides_of(k, "k", s);
  strides_of(v, "v", s + 3);
  const void *kp = address(k, "k", at::kBFloat16, dev, false), *vp = address(v, "v", at::kBFloat16, dev, false);
  const int* sl = address_of<const int>(slots, "slots", at::kInt, dev);
  const int inter = bool_arg(a[7]);
  float ks = 1.f, vs = 1.f;
  if (!bf16) ks = (float)float_arg(PyTuple_GET_ITEM(a[4], 0)), vs = (float)float_arg(PyTuple_GET_ITEM(a[4], 1));
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  void* st = stream_of(dev);
  if (q4)
    check(g_fn.append_q4(kp, vp, sl, pos, tab.p, tab.n, tab.R, inter, c[0], c[1], c[2], c[3], ks, vs, t.B, t.T, t.H, t.D,
                         page_size, pages, s, st),
          "attn_cache_append_q4");
  else if (bf16)
    check(g_fn.append(kp, vp, sl, pos, tab.p, tab.n, tab.R, inter, c[0], c[1], t.B, t.T, t.H, t.D, page_size, pages, s, st),
          "attn_cache_append");
  else
    check(g_fn.append_fp8(kp, vp, sl, pos, tab.p, tab.n, tab.R, inter, c[0], c[1], ks, vs, t.B, t.T, t.H, t.D, page_size,
                          pages, s, st),
          "attn_cache_append_fp8");
  Py_RETURN_NONE;
}

// The tensors of a 4-bit cache, checked against the codes of k.
struct Q4Cache {
  const void* p[4];
  int pages, H, page_size, D;
};
Q4Cache q4_cache(PyObject* const* a, int dev, bool paged) {
  static const char* names[2][4] = {{"k4", "k4_sf", "v4", "v4_sf"}, {"k4_pages", "k4_sf_pages", "v4_pages", "v4_sf_pages"}};
  const char** nm = names[paged];
  const at::Tensor *x[4];
  for (int i = 0; i < 4; ++i) x[i] = &tensor(a[i], nm[i]);
  if (x[0]->dim() != 4) value_error(std::string(nm[0]) + " must be [pages, Hkv, page_size, D/2]");
  const auto s = x[0]->sizes();
  if (x[2]->sizes() != s || x[1]->dim() != 4 || x[1]->size(0) != s[0] || x[1]->size(1) != s[1] || x[1]->size(2) != s[2] ||
      x[1]->size(3) != s[3] / 8 || x[3]->sizes() != x[1]->sizes())
    value_error(std::string(nm[0]) + " and " + nm[2] + " must be [pages, Hkv, page_size, D/2], " + nm[1] + " and " + nm[3] +
                " [pages, Hkv, page_size, D/16]");
  Q4Cache c;
  for (int i = 0; i < 4; ++i) c.p[i] = address(*x[i], nm[i], at::kByte, dev);
  c.pages = dim(*x[0], 0, nm[0]);
  c.H = dim(*x[0], 1, nm[0]);
  c.page_size = dim(*x[0], 2, nm[0]);
  c.D = to_int(2 * s[3], nm[0]);
  return c;
}

// (slots, k4, k4_sf, v4, v4_sf, k_scale, v_scale, k, v)
PyObject* gather(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  const at::Tensor& slots = tensor(a[0], "slots");
  const int dev = device_of(slots, "slots");
  const Q4Cache c = q4_cache(a + 1, dev, false);
  const int tokens = to_int(slots.numel(), "slots");
  at::Tensor out[2] = {optional(a[7], "k"), optional(a[8], "v")};
  const int64_t shape[3] = {tokens, c.H, c.D};
  const at::IntArrayRef sizes(shape, 3);
  allocate(out[0], sizes, out[1], sizes, slots);
  if (out[0].sizes() != sizes || out[1].sizes() != sizes) value_error("k, v must be [tokens, Hkv, D]");
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  check(g_fn.gather_q4(address_of<const int>(slots, "slots", at::kInt, dev), c.p[0], c.p[1], c.p[2], c.p[3],
                       (float)float_arg(a[5]), (float)float_arg(a[6]), address(out[0], "k", at::kBFloat16, dev),
                       address(out[1], "v", at::kBFloat16, dev), tokens, c.H, c.D, c.page_size, c.pages,
                       stream_of(dev)),
        "attn_cache_gather_q4");
  return wrap2(std::move(out[0]), std::move(out[1]));
}

// (q, k4, k4_sf, v4, v4_sf, k_scale, v_scale, block_table, cache_lens, scale, o, lse, workspace, rope_cos_sin);
// block_table None: contiguous caches
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 14);
  const at::Tensor &q = tensor(a[0], "q"), &lens = tensor(a[8], "cache_lens");
  const at::Tensor bt = optional(a[7], "block_table");
  const int dev = device_of(q, "q");
  if (q.dim() != 4) value_error("q must be [B, Hq, Tq, D]");
  const bool paged = bt.defined();
  const Q4Cache c = q4_cache(a + 1, dev, paged);
  const int B = dim(q, 0, "q"), Hq = dim(q, 1, "q"), Tq = dim(q, 2, "q"), D = dim(q, 3, "q");
  int S = c.page_size, max_pages = 0;
  if (paged) {
    if (c.D != D || bt.dim() != 2 || bt.size(0) != B)
      value_error("k4_pages must match q's head dimension, block_table be [B, max_pages]");
    max_pages = dim(bt, 1, "block_table");
    S = to_int((int64_t)max_pages * c.page_size, "max_pages * page_size");
  } else if (c.pages != B || c.D != D) {
    value_error("k4, v4 must be [B, Hkv, S, D/2] matching q");
  }
  if (lens.dim() != 1 || lens.size(0) != B) value_error("cache_lens must be [B]");
  at::Tensor o = optional(a[10], "o"), lse = optional(a[11], "lse");
  if (!o.defined()) o = at::empty(q.sizes(), on(q, q.scalar_type()));
  if (!lse.defined()) lse = at::empty(q.sizes().slice(0, 3), on(q, at::kFloat));
  if (o.sizes() != q.sizes() || lse.sizes() != q.sizes().slice(0, 3))
    value_error("o must be [B, Hq, Tq, D], lse [B, Hq, Tq]");
  const Table tab = table_arg(a[13], dev);
  if (a[13] != Py_None && tab.R != D) value_error("rope_cos_sin must be [positions, D]");
  at::Tensor ws = optional(a[12], "workspace");
  if (!ws.defined()) {
    const int64_t bytes = (int64_t)g_fn.decode_ws(B, Hq, c.H, Tq, S, D);
    if (bytes > 0) ws = at::empty({bytes}, on(q, at::kByte));
  }
  void* wp = ws.defined() ? address(ws, "workspace", at::kByte, dev) : nullptr;
  const size_t wn = ws.defined() ? (size_t)ws.numel() : 0;
  const void* qp = address(q, "q", at::kBFloat16, dev);
  const int* ln = address_of<const int>(lens, "cache_lens", at::kInt, dev);
  void* op = address(o, "o", at::kBFloat16, dev);
  float* lp = address_of<float>(lse, "lse", at::kFloat, dev);
  const float ks = (float)float_arg(a[5]), vs = (float)float_arg(a[6]);
  const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)float_arg(a[9]);
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  void* st = stream_of(dev);
  if (paged)
    check(g_fn.decode_paged(qp, c.p[0], c.p[1], c.p[2], c.p[3], ks, vs,
                            address_of<const int>(bt, "block_table", at::kInt, dev), ln, op, lp, wp, wn, B, Hq, c.H, Tq,
                            c.page_size, c.pages, max_pages, D, scale, tab.p, tab.n, st),
          "attn_decode_paged_q4_fwd");
  else
    check(g_fn.decode(qp, c.p[0], c.p[1], c.p[2], c.p[3], ks, vs, ln, op, lp, wp, wn, B, Hq, c.H, Tq, S, D, scale, tab.p,
                      tab.n, st),
          "attn_decode_q4_fwd");
  return wrap2(std::move(o), std::move(lse));
}

// A block table of B rows, or none: its pointer and its width.
struct Blocks {
  const int* p = nullptr;
  int max_pages = 0;
};
Blocks blocks_arg(const at::Tensor& t, const char* name, int rows, int dev) {
  Blocks b;
  if (!t.defined()) return b;
  if (t.dim() != 2 || t.size(0) != rows) value_error(std::string(name) + " must be [" + std::to_string(rows) + ", max_pages]");
  b.p = address_of<const int>(t, name, at::kInt, dev);
  b.max_pages = dim(t, 1, name);
  return b;
}

const int* lens_arg(const at::Tensor& t, const char* name, int n, int dev) {
  if (t.dim() != 1 || t.size(0) != n) value_error(std::string(name) + " must be [" + std::to_string(n) + "]");
  return address_of<const int>(t, name, at::kInt, dev);
}

// (q, keys, k_scale, lse, cache_lens, weights, block_table, scale); keys: a cache of bf16 (k_scale None) or E4M3 keys,
// or the codes and block scales of 4-bit ones
PyObject* weights(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 8);
  const at::Tensor &q = tensor(a[0], "q"), &lse = tensor(a[3], "lse"), &lens = tensor(a[4], "cache_lens"),
                   &w = tensor(a[5], "weights");
  const at::Tensor bt = optional(a[6], "block_table");
  const int dev = device_of(q, "q");
  if (q.dim() != 4) value_error("q must be [B, Hq, Tq, D]");
  const bool q4 = PyTuple_GET_SIZE(a[1]) == 2, bf16 = a[2] == Py_None;
  const char* kn = bf16 ? "k_cache" : q4 ? "k4" : "k8";
  const char* name = bf16 ? "attn_cache_weights" : q4 ? "attn_cache_weights_q4" : "attn_cache_weights_fp8";
  const at::Tensor& k = tensor(PyTuple_GET_ITEM(a[1], 0), kn);
  const int B = dim(q, 0, "q"), Hq = dim(q, 1, "q"), Tq = dim(q, 2, "q"), D = dim(q, 3, "q");
  const int64_t wide = q4 ? D / 2 : D;
  if (k.dim() != 4 || k.size(3) != wide)
    value_error(std::string(kn) + " must be [pages, Hkv, page_size, " + std::to_string(wide) + "] matching q");
  if (!bt.defined() && k.size(0) != B)
    value_error(std::string(kn) + " must hold a row for each of q's (or come with a block_table)");
  const void *kp = address(k, kn, bf16 ? at::kBFloat16 : at::kByte, dev), *sf = nullptr;
  if (q4) {
    const at::Tensor& x = tensor(PyTuple_GET_ITEM(a[1], 1), "k4_sf");
    if (x.dim() != 4 || x.sizes().slice(0, 3) != k.sizes().slice(0, 3) || x.size(3) != D / 16)
      value_error("k4_sf must be [pages, Hkv, page_size, D/16]");
    sf = address(x, "k4_sf", at::kByte, dev);
  }
  if (w.sizes() != k.sizes().slice(0, 3)) value_error("weights must be [pages, Hkv, page_size], an entry for each key");
  if (lse.sizes() != q.sizes().slice(0, 3)) value_error("lse must be [B, Hq, Tq]");
  const Blocks blocks = blocks_arg(bt, "block_table", B, dev);
  if (bt.defined() && blocks.max_pages == 0) {     // no position: its NULL would mean contiguous caches
    Py_INCREF(a[5]);
    return a[5];
  }
  const void* qp = address(q, "q", at::kBFloat16, dev);
  const float* lp = address_of<const float>(lse, "lse", at::kFloat, dev);
  const int* ln = lens_arg(lens, "cache_lens", B, dev);
  float* wp = address_of<float>(w, "weights", at::kFloat, dev);
  const int pages = dim(k, 0, kn), H = dim(k, 1, kn), page_size = dim(k, 2, kn);
  const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)float_arg(a[7]);
  const float ks = bf16 ? 1.f : (float)float_arg(a[2]);
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  void* st = stream_of(dev);
  if (bf16)
    check(g_fn.weights(qp, kp, lp, blocks.p, ln, wp, B, Hq, H, Tq, page_size, pages, blocks.max_pages, D, scale, st), name);
  else if (q4)
    check(g_fn.weights_q4(qp, kp, sf, ks, lp, blocks.p, ln, wp, B, Hq, H, Tq, page_size, pages, blocks.max_pages, D, scale,
                          st),
          name);
  else
    check(g_fn.weights_fp8(qp, kp, ks, lp, blocks.p, ln, wp, B, Hq, H, Tq, page_size, pages, blocks.max_pages, D, scale,
                           st),
          name);
  Py_INCREF(a[5]);
  return a[5];
}

// (weights, caches, cache_lens, budget, recent, first, block_table, kept, lens_out)
PyObject* evict(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  const at::Tensor &w = tensor(a[0], "weights"), &lens = tensor(a[2], "cache_lens");
  const at::Tensor bt = optional(a[6], "block_table");
  const int dev = device_of(w, "weights");
  if (w.dim() != 3) value_error("weights must be [pages, Hkv, page_size]");
  if (lens.dim() != 1) value_error("cache_lens must be [B]");
  const int B = dim(lens, 0, "cache_lens"), pages = dim(w, 0, "weights"), H = dim(w, 1, "weights");
  const int page_size = dim(w, 2, "weights");
  if (!bt.defined() && pages != B) value_error("weights must hold a row for each length (or come with a block_table)");
  const int budget = int_arg(a[3], "budget"), recent = int_arg(a[4], "recent"), first = int_arg(a[5], "first");
  if (budget < 1) value_error("budget must be at least 1");
  const Py_ssize_t np = PyTuple_GET_SIZE(a[1]);
  if (np > 8) value_error("caches: at most 8 planes");
  void* planes[8];
  int rows[8];
  for (Py_ssize_t i = 0; i < np; ++i) {
    const std::string name = "caches[" + std::to_string(i) + "]";
    const at::Tensor& x = tensor(PyTuple_GET_ITEM(a[1], i), name.c_str());
    if (x.dim() != 4 || x.sizes().slice(0, 3) != w.sizes())
      value_error(name + " must be [pages, Hkv, page_size, width] as weights");
    planes[i] = address(x, name.c_str(), x.scalar_type(), dev);
    rows[i] = to_int(x.size(3) * (int64_t)x.element_size(), name.c_str());
  }
  const Blocks blocks = blocks_arg(bt, "block_table", B, dev);
  at::Tensor kept = optional(a[7], "kept"), out = optional(a[8], "lens_out");
  if (!kept.defined()) kept = at::empty({B, H, budget}, on(w, at::kInt));
  if (!out.defined()) out = at::empty({B}, on(w, at::kInt));
  if (kept.dim() != 3 || kept.size(0) != B || kept.size(1) != H || kept.size(2) != budget || out.dim() != 1 || out.size(0) != B)
    value_error("kept must be [B, Hkv, budget], lens_out [B]");
  const int* ln = lens_arg(lens, "cache_lens", B, dev);
  float* wp = address_of<float>(w, "weights", at::kFloat, dev);
  int *kp = address_of<int>(kept, "kept", at::kInt, dev), *op = address_of<int>(out, "lens_out", at::kInt, dev);
  if (bt.defined() && blocks.max_pages == 0) value_error("block_table holds no page");
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  check(g_fn.evict(wp, planes, rows, (int)np, blocks.p, ln, budget, recent, first, kp, op, B, H, page_size, pages,
                   blocks.max_pages, stream_of(dev)),
        "attn_cache_evict");
  return wrap2(std::move(kept), std::move(out));
}

// (q, k_prefix, v_prefix, prefix_table, prefix_lens, k, v, block_table, cache_lens, scale, o, lse, workspace);
// k_prefix, v_prefix None: the prefixes are in k, v's pages too, through prefix_table
PyObject* prefix(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 13);
  const at::Tensor &q = tensor(a[0], "q"), &pl = tensor(a[4], "prefix_lens"), &lens = tensor(a[8], "cache_lens");
  const bool paged = a[1] == Py_None;
  const char *kn = paged ? "k_pages" : "k_cache", *vn = paged ? "v_pages" : "v_cache";
  const at::Tensor &k = tensor(a[5], kn), &v = tensor(a[6], vn);
  const int dev = device_of(q, "q");
  if (q.dim() != 4) value_error("q must be [B, Hq, Tq, D]");
  if (pl.dim() != 1) value_error("prefix_lens must be [P]");
  const int B = dim(q, 0, "q"), Hq = dim(q, 1, "q"), Tq = dim(q, 2, "q"), D = dim(q, 3, "q"), P = dim(pl, 0, "prefix_lens");
  if (P < 1 || B % P)
    value_error("the rows must be a multiple of the prefixes: " + std::to_string(B) + " rows, " + std::to_string(P) +
                " prefixes");
  if (k.dim() != 4 || k.size(3) != D || v.sizes() != k.sizes() || (!paged && k.size(0) != B))
    value_error(std::string(kn) + ", " + vn +
                (paged ? " must be [num_pages, Hkv, page_size, D] matching q" : " must be [B, Hkv, S, D] matching q"));
  const int N = dim(k, 0, kn), H = dim(k, 1, kn), per = dim(k, 2, kn);
  int Sp, S = per;
  Blocks pt, bt;
  const void *kp = nullptr, *vp = nullptr;
  if (paged) {
    pt = blocks_arg(tensor(a[3], "prefix_table"), "prefix_table", P, dev);
    bt = blocks_arg(tensor(a[7], "block_table"), "block_table", B, dev);
    Sp = to_int((int64_t)pt.max_pages * per, "prefix_table's positions");
    S = to_int((int64_t)bt.max_pages * per, "block_table's positions");
  } else {
    const at::Tensor &x = tensor(a[1], "k_prefix"), &y = tensor(a[2], "v_prefix");
    if (x.dim() != 4 || x.size(0) != P || x.size(1) != H || x.size(3) != D || y.sizes() != x.sizes())
      value_error("k_prefix, v_prefix must be [P, Hkv, Sp, D] matching q and the caches");
    Sp = dim(x, 2, "k_prefix");
    kp = address(x, "k_prefix", at::kBFloat16, dev);
    vp = address(y, "v_prefix", at::kBFloat16, dev);
  }
  at::Tensor o = optional(a[10], "o"), lse = optional(a[11], "lse");
  if (!o.defined()) o = at::empty(q.sizes(), on(q, q.scalar_type()));
  if (!lse.defined()) lse = at::empty(q.sizes().slice(0, 3), on(q, at::kFloat));
  if (o.sizes() != q.sizes() || lse.sizes() != q.sizes().slice(0, 3)) value_error("o must be [B, Hq, Tq, D], lse [B, Hq, Tq]");
  at::Tensor ws = optional(a[12], "workspace");
  if (!ws.defined()) {
    const int64_t bytes = (int64_t)g_fn.prefix_ws(B, Hq, H, Tq, P, Sp, S, D);
    if (bytes > 0) ws = at::empty({bytes}, on(q, at::kByte));
  }
  void* wp = ws.defined() ? address(ws, "workspace", at::kByte, dev) : nullptr;
  const size_t wn = ws.defined() ? (size_t)ws.numel() : 0;
  const auto bf = at::kBFloat16;
  const void *qp = address(q, "q", bf, dev), *kc = address(k, kn, bf, dev), *vc = address(v, vn, bf, dev);
  const int *pn = lens_arg(pl, "prefix_lens", P, dev), *ln = lens_arg(lens, "cache_lens", B, dev);
  void* op = address(o, "o", bf, dev);
  float* lp = address_of<float>(lse, "lse", at::kFloat, dev);
  const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)float_arg(a[9]);
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  void* st = stream_of(dev);
  if (paged)
    check(g_fn.prefix_paged(qp, kc, vc, pt.p, pn, bt.p, ln, op, lp, wp, wn, B, Hq, H, Tq, P, per, N, pt.max_pages,
                            bt.max_pages, D, scale, st),
          "attn_decode_paged_prefix_fwd");
  else
    check(g_fn.prefix(qp, kp, vp, pn, kc, vc, ln, op, lp, wp, wn, B, Hq, H, Tq, P, Sp, S, D, scale, st),
          "attn_decode_prefix_fwd");
  return wrap2(std::move(o), std::move(lse));
}

// (addresses of the C functions by name, _check, current raw stream of a device)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 3);
  auto of = [&](const char* name) {
    PyObject* v = PyDict_GetItemString(a[0], name);
    if (!v) value_error(std::string("no address of ") + name);
    void* p = PyLong_AsVoidPtr(v);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
  };
#define BIND(field, name) g_fn.field = reinterpret_cast<decltype(g_fn.field)>(of(#name))
  BIND(plan, attn_cache_plan);
  BIND(rope_table, attn_rope_table);
  BIND(rope, attn_rope);
  BIND(rope_bwd, attn_rope_bwd);
  BIND(append, attn_cache_append);
  BIND(append_fp8, attn_cache_append_fp8);
  BIND(append_q4, attn_cache_append_q4);
  BIND(gather_q4, attn_cache_gather_q4);
  BIND(decode_ws, attn_decode_q4_workspace_size);
  BIND(decode, attn_decode_q4_fwd);
  BIND(decode_paged, attn_decode_paged_q4_fwd);
  BIND(weights, attn_cache_weights);
  BIND(weights_fp8, attn_cache_weights_fp8);
  BIND(weights_q4, attn_cache_weights_q4);
  BIND(evict, attn_cache_evict);
  BIND(prefix_ws, attn_decode_prefix_workspace_size);
  BIND(prefix, attn_decode_prefix_fwd);
  BIND(prefix_paged, attn_decode_paged_prefix_fwd);
#undef BIND
  PyObject** keep[2] = {&g_check, &g_stream};
  for (int i = 0; i < 2; ++i) {
    Py_INCREF(a[1 + i]);
    Py_XSETREF(*keep[i], a[1 + i]);
  }
  Py_RETURN_NONE;
}

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what());
  } catch (const std::exception&) {
    torch::translate_exception_to_python(std::current_exception());   // torch.OutOfMemoryError and the like
  }
  return nullptr;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(bind),   METHOD(plan),   METHOD(rope_table), METHOD(rope),
                           METHOD(append), METHOD(gather), METHOD(decode),     METHOD(weights),
                           METHOD(evict),  METHOD(prefix), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cache_ext", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_ext() { return PyModule_Create(&g_module); }
