// attn_bind.cpp -- the serving and packed-batch calls of attn.py in C++.
//
// A decoding step's kernels take a few microseconds; looking at its tensors,
// allocating its outputs and marshalling its arguments in Python took 20 us on
// the GPU's Grace host (every torch call among kernel launches costs 3-5 us
// there), so these calls do that here: check the tensors, allocate on the current
// stream, call the C ABI of libattn.so.  The computation is all in the library.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>
#include <vector>

#include "attn.h"

namespace {

PyObject* g_error = nullptr;  // attn.AttnError

struct Refused : std::exception {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& msg) {
  PyErr_SetString(PyExc_ValueError, msg.c_str());
  throw Refused();
}

void check(int rc) {
  if (rc == ATTN_OK) return;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", rc, attn_last_error_string()) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, attn_last_error_string());
  }
  throw Refused();
}

std::string say(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "] " + c10::toString(t.scalar_type()) + " on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The device that all tensors of a call are on, from its first one.
struct Call {
  c10::Device dev;
  explicit Call(const at::Tensor& t, const char* name) : dev(t.device()) {
    if (!dev.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor, got " + say(t));
  }
  // t: this type, these extents (-1: any), on the call's device.
  void want(const at::Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
            bool contiguous = true) const {
    bool ok = t.scalar_type() == type && t.device() == dev && t.dim() == (int64_t)shape.size() && t.layout() == at::kStrided;
    int64_t i = 0;
    for (int64_t n : shape) {
      if (!ok) break;
      ok = n < 0 || t.size(i) == n;
      ++i;
    }
    if (ok && contiguous) ok = t.is_contiguous();
    if (ok) return;
    std::string s = std::string(name) + " must be a " + (contiguous ? "contiguous " : "") + c10::toString(type) + " tensor [";
    const char* sep = "";
    for (int64_t n : shape) {
      s += sep + (n < 0 ? std::string("n") : std::to_string(n));
      sep = ", ";
    }
    refuse(s + "] on " + dev.str() + ", got " + say(t));
  }
  // t: [T, H, d], heads d apart; its token stride.
  int64_t packed(const at::Tensor& t, const char* name, at::ScalarType type, int64_t T, int64_t H, int64_t d) const {
    want(t, name, type, {T, H, d}, false);
    if (t.is_contiguous()) return H * d;
    if (t.stride(2) != 1 || (t.stride(1) != d && H > 1)) refuse(std::string(name) + ": the heads of a token must be contiguous");
    return T > 1 ? t.stride(0) : H * d;
  }
  // (the allocation behind torch.empty, without its dispatch: 0.55 against 0.77 us)
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
  }
  // Small int32 vectors in one allocation (0.2 us each instead of 0.6), 16 bytes aligned.
  std::vector<at::Tensor> vectors(std::initializer_list<int64_t> lens) const {
    int64_t n = 0;
    for (int64_t x : lens) n += (x + 3) / 4 * 4;
    const at::Tensor all = empty({n}, at::kInt);
    std::vector<at::Tensor> out;
    int64_t at = 0;
    for (int64_t x : lens) {
      at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
      t.unsafeGetTensorImpl()->set_storage_offset(at);
      t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(&x, 1));
      out.push_back(std::move(t));
      at += (x + 3) / 4 * 4;
    }
    return out;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

template <typename T>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

attn_dtype_t dtype16(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return ATTN_BF16;
  if (t.scalar_type() == at::kHalf) return ATTN_F16;
  refuse(std::string(name) + " must be fp16 or bf16, got " + say(t));
}

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int narrow(int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffff) refuse(std::string(name) + " = " + std::to_string(v) + " is out of range");
  return (int)v;
}

float scale_of(PyObject* o, int64_t d) {
  if (o == Py_None) return (float)(1.0 / std::sqrt((double)d));
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

int flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v;
}

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* t = PyTuple_New((Py_ssize_t)ts.size());
  if (!t) throw Refused();
  Py_ssize_t i = 0;
  for (const at::Tensor& x : ts) {
    PyObject* o = THPVariable_Wrap(x);
    if (!o) {
      Py_DECREF(t);
      throw Refused();
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// The caller's workspace, or one of `need` bytes for the call (freed after it: the
// allocator hands its memory on in stream order).
struct Workspace {
  c10::DataPtr own;
  void* p = nullptr;
  size_t n = 0;
  Workspace(const Call& c, PyObject* o, size_t need) {
    if (o != Py_None) {
      const at::Tensor& t = tensor(o, "ws");
      if (t.device() != c.dev || !t.is_contiguous()) refuse("ws must be contiguous on " + c.dev.str() + ", got " + say(t));
      p = t.data_ptr();
      n = t.nbytes();
    } else if (need) {
      own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
      p = own.get();
      n = need;
    }
  }
};

void count_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("wrong number of arguments");
}

// ------------------------------------------------------------------ pages
PyObject* pages_extend(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 9);
  const at::Tensor &lens = tensor(a[0], "lens"), &add = tensor(a[1], "add"), &table = tensor(a[2], "block_table"),
                   &free_pages = tensor(a[3], "free_pages"), &count = tensor(a[4], "free_count");
  const Call c(lens, "lens");
  c.want(lens, "lens", at::kInt, {-1});
  const int64_t B = lens.size(0), T = whole(a[6]);
  c.want(add, "add", at::kInt, {B});
  c.want(table, "block_table", at::kInt, {B, -1});
  c.want(free_pages, "free_pages", at::kInt, {-1});
  c.want(count, "free_count", at::kInt, {1});
  if (T < 0) refuse("max_new must not be negative");
  c10::cuda::CUDAGuard guard(c.dev);
  const std::vector<at::Tensor> v = c.vectors({B, B + 1, a[7] != Py_None ? 0 : B, a[8] != Py_None ? 0 : 1});
  const at::Tensor &granted = v[0], &cu = v[1];
  const at::Tensor &new_lens = a[7] != Py_None ? tensor(a[7], "new_lens") : v[2],
                   &left = a[8] != Py_None ? tensor(a[8], "free_left") : v[3];
  c.want(new_lens, "new_lens", at::kInt, {B});
  c.want(left, "free_left", at::kInt, {1});
  const at::Tensor slots = c.empty({T}, at::kLong);
  check(attn_pages_extend(ptr<int>(lens), ptr<int>(add), narrow(B, "B"), ptr<int>(table), narrow(table.size(1), "width"),
                          ptr<int>(free_pages), ptr<int>(count), narrow(free_pages.size(0), "free_pages"),
                          narrow(whole(a[5]), "page"), T, ptr<int>(new_lens), ptr<int>(granted), ptr<int>(cu),
                          ptr<int64_t>(slots), ptr<int>(left), c.stream()));
  return tuple({new_lens, granted, cu, slots, left});
}

PyObject* pages_release(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 8);
  const at::Tensor &lens = tensor(a[0], "lens"), &done = tensor(a[1], "finished"), &table = tensor(a[2], "block_table"),
                   &free_pages = tensor(a[3], "free_pages"), &count = tensor(a[4], "free_count");
  const Call c(lens, "lens");
  c.want(lens, "lens", at::kInt, {-1});
  const int64_t B = lens.size(0);
  c.want(done, "finished", at::kInt, {B});
  c.want(table, "block_table", at::kInt, {B, -1});
  c.want(free_pages, "free_pages", at::kInt, {-1});
  c.want(count, "free_count", at::kInt, {1});
  c10::cuda::CUDAGuard guard(c.dev);
  const std::vector<at::Tensor> o = c.vectors({a[6] != Py_None ? 0 : B, a[7] != Py_None ? 0 : 1});
  const at::Tensor &new_lens = a[6] != Py_None ? tensor(a[6], "new_lens") : o[0],
                   &left = a[7] != Py_None ? tensor(a[7], "free_left") : o[1];
  c.want(new_lens, "new_lens", at::kInt, {B});
  c.want(left, "free_left", at::kInt, {1});
  check(attn_pages_release(ptr<int>(lens), ptr<int>(done), narrow(B, "B"), ptr<int>(table), narrow(table.size(1), "width"),
                           ptr<int>(free_pages), ptr<int>(count), narrow(free_pages.size(0), "free_pages"),
                           narrow(whole(a[5]), "page"), ptr<int>(new_lens), ptr<int>(left), c.stream()));
  return tuple({new_lens, left});
}

// ------------------------------------------------------------------ 8-bit cache
struct Cache {
  int64_t P, H, page, d;
  Cache(const Call& c, const at::Tensor& k, const at::Tensor& v, const at::Tensor& ks, const at::Tensor& vs) {
    const at::ScalarType code = k.scalar_type();
    if (code != at::kFloat8_e4m3fn && code != at::kByte) refuse("the caches hold float8_e4m3fn or uint8 codes, got " + say(k));
    c.want(k, "k_cache", code, {-1, -1, -1, -1});
    P = k.size(0);
    H = k.size(1);
    page = k.size(2);
    d = k.size(3);
    c.want(v, "v_cache", code, {P, H, page, d});
    c.want(ks, "k_scale", at::kFloat, {P, H});
    c.want(vs, "v_scale", at::kFloat, {P, H});
  }
};

PyObject* kv8_append(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 7);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                   &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache"), &ks = tensor(a[5], "k_scale"),
                   &vs = tensor(a[6], "v_scale");
  const Call c(k, "k");
  const Cache m(c, kc, vc, ks, vs);
  const attn_dtype_t dt = dtype16(k, "k");
  const int64_t T = k.dim() ? k.size(0) : 0;
  const int64_t k_st = c.packed(k, "k", k.scalar_type(), T, m.H, m.d), v_st = c.packed(v, "v", k.scalar_type(), T, m.H, m.d);
  c.want(slots, "slots", at::kLong, {T});
  c10::cuda::CUDAGuard guard(c.dev);
  check(attn_kv8_append(ptr<void>(k), ptr<void>(v), k_st, v_st, ptr<int64_t>(slots), T, narrow(m.H, "H"),
                        narrow(m.d, "d"), ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<float>(ks), ptr<float>(vs),
                        narrow(m.P, "P"), narrow(m.page, "page"), dt, c.stream()));
  Py_RETURN_NONE;
}

PyObject* kv8_decode(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 10);
  const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                   &ks = tensor(a[3], "k_scale"), &vs = tensor(a[4], "v_scale"), &table = tensor(a[5], "block_table"),
                   &lens = tensor(a[6], "lens");
  const Call c(q, "q");
  const Cache m(c, kc, vc, ks, vs);
  const attn_dtype_t dt = dtype16(q, "q");
  c.want(q, "q", q.scalar_type(), {-1, -1, -1, m.d});
  const int64_t B = q.size(0), Nq = q.size(1), Hq = q.size(2);
  c.want(table, "block_table", at::kInt, {B, -1});
  c.want(lens, "lens", at::kInt, {B});
  const float scale = scale_of(a[7], m.d);
  const int causal = flag(a[8]), nq = narrow(Nq, "Nq"), hq = narrow(Hq, "Hq"), h = narrow(m.H, "H"), d = narrow(m.d, "d");
  c10::cuda::CUDAGuard guard(c.dev);
  const at::Tensor o = c.empty({B, Nq, Hq, m.d}, q.scalar_type()), lse = c.empty({B, Hq, Nq}, at::kFloat);
  const Workspace ws(c, a[9], attn_kv8_decode_workspace_size(nq, hq, h, d));
  check(attn_kv8_decode(ptr<void>(q), ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<float>(ks), ptr<float>(vs), ptr<int>(table),
                        ptr<int>(lens), ptr<void>(o), ptr<float>(lse), narrow(B, "B"), nq, hq, h, d, narrow(m.P, "P"),
                        narrow(m.page, "page"), narrow(table.size(1), "width"), scale, causal, dt, ws.p, ws.n, c.stream()));
  return tuple({o, lse});
}

// ------------------------------------------------------------------ 4-bit cache
struct Cache4 {
  int64_t P, H, page, d;
  Cache4(const Call& c, const at::Tensor& k, const at::Tensor& v, const at::Tensor& ks, const at::Tensor& vs) {
    c.want(k, "k_cache", at::kByte, {-1, -1, -1, -1});
    P = k.size(0);
    H = k.size(1);
    page = k.size(2);
    d = k.size(3) * 2;
    c.want(v, "v_cache", at::kByte, {P, H, page, d / 2});
    c.want(ks, "k_scale", at::kBFloat16, {P, H, page, d / 32});
    c.want(vs, "v_scale", at::kBFloat16, {P, H, page, d / 32});
  }
};

PyObject* kv4_append(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 7);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                   &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache"), &ks = tensor(a[5], "k_scale"),
                   &vs = tensor(a[6], "v_scale");
  const Call c(k, "k");
  const Cache4 m(c, kc, vc, ks, vs);
  const attn_dtype_t dt = dtype16(k, "k");
  const int64_t T = k.dim() ? k.size(0) : 0;
  const int64_t k_st = c.packed(k, "k", k.scalar_type(), T, m.H, m.d), v_st = c.packed(v, "v", k.scalar_type(), T, m.H, m.d);
  c.want(slots, "slots", at::kLong, {T});
  c10::cuda::CUDAGuard guard(c.dev);
  check(attn_kv4_append(ptr<void>(k), ptr<void>(v), k_st, v_st, ptr<int64_t>(slots), T, narrow(m.H, "H"),
                        narrow(m.d, "d"), ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<uint16_t>(ks), ptr<uint16_t>(vs),
                        narrow(m.P, "P"), narrow(m.page, "page"), dt, c.stream()));
  Py_RETURN_NONE;
}

PyObject* kv4_decode(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 10);
  const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                   &ks = tensor(a[3], "k_scale"), &vs = tensor(a[4], "v_scale"), &table = tensor(a[5], "block_table"),
                   &lens = tensor(a[6], "lens");
  const Call c(q, "q");
  const Cache4 m(c, kc, vc, ks, vs);
  const attn_dtype_t dt = dtype16(q, "q");
  c.want(q, "q", q.scalar_type(), {-1, -1, -1, m.d});
  const int64_t B = q.size(0), Nq = q.size(1), Hq = q.size(2);
  c.want(table, "block_table", at::kInt, {B, -1});
  c.want(lens, "lens", at::kInt, {B});
  const float scale = scale_of(a[7], m.d);
  const int causal = flag(a[8]), nq = narrow(Nq, "Nq"), hq = narrow(Hq, "Hq"), h = narrow(m.H, "H"), d = narrow(m.d, "d");
  c10::cuda::CUDAGuard guard(c.dev);
  const at::Tensor o = c.empty({B, Nq, Hq, m.d}, q.scalar_type()), lse = c.empty({B, Hq, Nq}, at::kFloat);
  const Workspace ws(c, a[9], attn_kv4_decode_workspace_size(nq, hq, h, d));
  check(attn_kv4_decode(ptr<void>(q), ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<uint16_t>(ks), ptr<uint16_t>(vs),
                        ptr<int>(table), ptr<int>(lens), ptr<void>(o), ptr<float>(lse), narrow(B, "B"), nq, hq, h, d,
                        narrow(m.P, "P"), narrow(m.page, "page"), narrow(table.size(1), "width"), scale, causal, dt, ws.p,
                        ws.n, c.stream()));
  return tuple({o, lse});
}

// ------------------------------------------------------------------ reading back
template <int BITS>
PyObject* kv_read(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 11);
  const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache"), &ks = tensor(a[2], "k_scale"),
                   &vs = tensor(a[3], "v_scale"), &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "lens"),
                   &cu = tensor(a[6], "cu");
  const Call c(kc, "k_cache");
  int64_t P, H, page, d;
  if constexpr (BITS == 8) {
    const Cache m(c, kc, vc, ks, vs);
    P = m.P, H = m.H, page = m.page, d = m.d;
  } else {
    const Cache4 m(c, kc, vc, ks, vs);
    P = m.P, H = m.H, page = m.page, d = m.d;
  }
  c.want(lens, "lens", at::kInt, {-1});
  const int64_t B = lens.size(0), T = whole(a[7]);
  c.want(table, "block_table", at::kInt, {B, -1});
  c.want(cu, "cu", at::kInt, {B + 1});
  if (T < 0) refuse("total must not be negative");
  const int64_t code = whole(a[8]);
  const at::ScalarType type = code == ATTN_BF16 ? at::kBFloat16 : at::kHalf;
  c10::cuda::CUDAGuard guard(c.dev);
  const at::Tensor k = a[9] != Py_None ? tensor(a[9], "k") : c.empty({T, H, d}, type);
  const at::Tensor v = a[10] != Py_None ? tensor(a[10], "v") : c.empty({T, H, d}, type);
  c.want(k, "k", type, {T, H, d});
  c.want(v, "v", type, {T, H, d});
  const int b = narrow(B, "B"), h = narrow(H, "H"), dd = narrow(d, "d"), pp = narrow(P, "P"), pg = narrow(page, "page"),
            width = narrow(table.size(1), "width");
  check(attn_kv_read(ptr<uint8_t>(kc), ptr<uint8_t>(vc), ks.data_ptr(), vs.data_ptr(), ptr<int>(table), ptr<int>(lens),
                     ptr<int>(cu), ptr<void>(k), ptr<void>(v), b, T, h, dd, pp, pg, width, BITS, (attn_dtype_t)code,
                     c.stream()));
  return tuple({k, v});
}

// ------------------------------------------------------------------ packed batches
struct Packed {
  int64_t B, Tq, Tk, Hq, Hkv, d, qs, ks, vs;
  Packed(const Call& c, const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& cu_q,
         const at::Tensor& cu_k) {
    const at::ScalarType type = q.scalar_type();
    c.want(q, "q", type, {-1, -1, -1}, false);
    c.want(k, "k", type, {-1, -1, q.size(2)}, false);
    Tq = q.size(0);
    Hq = q.size(1);
    d = q.size(2);
    Tk = k.size(0);
    Hkv = k.size(1);
    qs = c.packed(q, "q", type, Tq, Hq, d);
    ks = c.packed(k, "k", type, Tk, Hkv, d);
    vs = c.packed(v, "v", type, Tk, Hkv, d);
    c.want(cu_q, "cu_q", at::kInt, {-1});
    c.want(cu_k, "cu_k", at::kInt, {cu_q.size(0)});
    B = cu_q.size(0) - 1;
    narrow(B, "B");
    narrow(Hq, "Hq");
    narrow(Hkv, "Hkv");
    narrow(d, "d");
  }
};

PyObject* varlen_fwd(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 9);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &cu_q = tensor(a[3], "cu_q"),
                   &cu_k = tensor(a[4], "cu_k");
  const Call c(q, "q");
  const attn_dtype_t dt = dtype16(q, "q");
  const Packed s(c, q, k, v, cu_q, cu_k);
  const float scale = scale_of(a[5], s.d);
  const int causal = flag(a[6]);
  c10::cuda::CUDAGuard guard(c.dev);
  const at::Tensor o = a[8] != Py_None ? tensor(a[8], "o") : c.empty({s.Tq, s.Hq, s.d}, q.scalar_type());
  c.want(o, "o", q.scalar_type(), {s.Tq, s.Hq, s.d});
  const at::Tensor lse = c.empty({s.Hq, s.Tq}, at::kFloat);
  const Workspace ws(c, a[7], attn_varlen_fwd_workspace_size((int)s.B, s.Tq, s.Tk, (int)s.Hq, (int)s.Hkv, (int)s.d));
  check(attn_varlen_fwd(ptr<void>(q), ptr<void>(k), ptr<void>(v), ptr<void>(o), ptr<float>(lse), ptr<int>(cu_q),
                        ptr<int>(cu_k), (int)s.B, s.Tq, s.Tk, (int)s.Hq, (int)s.Hkv, (int)s.d, s.qs, s.ks, s.vs, scale,
                        causal, dt, ws.p, ws.n, c.stream()));
  return tuple({o, lse});
}

PyObject* varlen_bwd(PyObject* const* a, Py_ssize_t n) {
  count_args(n, 14);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &o = tensor(a[3], "o"),
                   &lse = tensor(a[4], "lse"), &g = tensor(a[5], "do"), &cu_q = tensor(a[6], "cu_q"),
                   &cu_k = tensor(a[7], "cu_k");
  const Call c(q, "q");
  const attn_dtype_t dt = dtype16(q, "q");
  const at::ScalarType type = q.scalar_type();
  const Packed s(c, q, k, v, cu_q, cu_k);
  c.want(o, "o", type, {s.Tq, s.Hq, s.d});
  c.want(g, "do", type, {s.Tq, s.Hq, s.d});
  c.want(lse, "lse", at::kFloat, {s.Hq, s.Tq});
  const float scale = scale_of(a[8], s.d);
  const int causal = flag(a[9]);
  c10::cuda::CUDAGuard guard(c.dev);
  const at::Tensor dq = a[11] != Py_None ? tensor(a[11], "dq") : c.empty({s.Tq, s.Hq, s.d}, type);
  const at::Tensor dk = a[12] != Py_None ? tensor(a[12], "dk") : c.empty({s.Tk, s.Hkv, s.d}, type);
  const at::Tensor dv = a[13] != Py_None ? tensor(a[13], "dv") : c.empty({s.Tk, s.Hkv, s.d}, type);
  c.want(dq, "dq", type, {s.Tq, s.Hq, s.d});
  c.want(dk, "dk", type, {s.Tk, s.Hkv, s.d});
  c.want(dv, "dv", type, {s.Tk, s.Hkv, s.d});
  const Workspace ws(c, a[10], attn_varlen_bwd_workspace_size((int)s.B, s.Tq, (int)s.Hq, (int)s.Hkv, (int)s.d));
  check(attn_varlen_bwd(ptr<void>(q), ptr<void>(k), ptr<void>(v), ptr<void>(o), ptr<float>(lse), ptr<void>(g),
                        ptr<void>(dq), ptr<void>(dk), ptr<void>(dv), ptr<int>(cu_q), ptr<int>(cu_k), (int)s.B, s.Tq, s.Tk,
                        (int)s.Hq, (int)s.Hkv, (int)s.d, s.qs, s.ks, s.vs, scale, causal, dt, ws.p, ws.n, c.stream()));
  return tuple({dq, dk, dv});
}

// Every C++ exception becomes a Python one.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XINCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<f>)), METH_FASTCALL
PyMethodDef methods[] = {{"pages_extend", FAST(pages_extend), nullptr}, {"pages_release", FAST(pages_release), nullptr},
                         {"kv8_append", FAST(kv8_append), nullptr},     {"kv8_decode", FAST(kv8_decode), nullptr},
                         {"kv4_append", FAST(kv4_append), nullptr},     {"kv4_decode", FAST(kv4_decode), nullptr},
                         {"kv4_read", FAST(kv_read<4>), nullptr},       {"kv8_read", FAST(kv_read<8>), nullptr},
                         {"varlen_fwd", FAST(varlen_fwd), nullptr},     {"varlen_bwd", FAST(varlen_bwd), nullptr},
                         {"set_error", set_error, METH_O, nullptr},     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "attn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_bind(void) { return PyModule_Create(&module); }
