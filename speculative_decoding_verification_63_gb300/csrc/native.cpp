// native.cpp -- argument marshalling of the calls that a model makes in every
// layer and step (sv_rotate, sv_kv_append, sv_token_logprobs), as a Python
// extension: tensors become the C ABI's structures (include/specverify.h), checked
// for type, shape, strides and device; results are allocated here unless they are
// given.  Written in Python the same took 14 to 19 us a call, most of what a small
// call takes.
//
// Every function takes the address of the library's entry point first.  With 0 it
// returns the packed structure instead (tests on the CPU).  It returns a tuple
// of the results, or the library's status where that is not SV_OK.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <sstream>
#include <string>

#include "specverify.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const std::string& why) {
  PyErr_SetString(PyExc_ValueError, why.c_str());
  throw Refused();
}

std::string text(IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << ")";
  return o.str();
}

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != nullptr && o != Py_None; }

// Everything lies on the workspace's device.
struct Place {
  c10::Device device{c10::kCPU};
  void check(const Tensor& t) const {
    if (t.device() != device)
      refuse("expected tensors of one device, got one on " + t.device().str() +
             " beside a workspace on " + device.str());
  }
};

// The address of a contiguous tensor of a type and shape; null for None.
const void* address(PyObject* o, ScalarType dtype, IntArrayRef shape, const char* what,
                    const Place& p) {
  if (!given(o)) return nullptr;
  const Tensor& t = tensor(o, what);
  if (t.scalar_type() != dtype || t.sizes() != shape || !t.is_contiguous())
    refuse(std::string(what) + ": expected contiguous " + c10::toString(dtype) + " " + text(shape) +
           ", got " + c10::toString(t.scalar_type()) + " " + text(t.sizes()));
  p.check(t);
  return t.data_ptr();
}

sv_dtype dtype_of(const Tensor& t, const char* what) {
  switch (t.scalar_type()) {
    case ScalarType::BFloat16: return SV_BF16;
    case ScalarType::Half: return SV_FP16;
    case ScalarType::Float: return SV_FP32;
    default: refuse(std::string(what) + ": expected bfloat16, float16 or float32, got " +
                    c10::toString(t.scalar_type()));
  }
}

// A [B][T][heads][D] tensor with contiguous D: its batch, token and head strides;
// that of a dimension of size 1, which says nothing, is 0.
void rows(const Tensor& t, IntArrayRef shape, const char* what, const Place& p, int64_t* stride) {
  if (t.sizes() != shape || t.stride(3) != 1)
    refuse(std::string(what) + ": expected " + text(shape) + " with contiguous rows, got " +
           text(t.sizes()));
  p.check(t);
  for (int i = 0; i < 3; ++i) stride[i] = shape[i] > 1 ? t.stride(i) : 0;
}

int whole(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + ": out of range");
  return static_cast<int>(v);
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();  // (an array's, say)
  return v != 0;
}

PyObject* field(PyObject* dict, const char* name, const char* what) {
  if (!PyDict_Check(dict)) refuse(std::string(what) + ": expected a dict");
  PyObject* v = PyDict_GetItemString(dict, name);
  if (v == nullptr) refuse(std::string(what) + ": " + name + " is missing");
  return v;
}

void rope(sv_rope& r, PyObject* o, const Place& p) {
  r.scale = 1.f;
  if (!given(o)) return;
  r.dim = whole(field(o, "dim", "rope"), "rope dim");
  r.interleaved = truth(field(o, "interleaved", "rope")) ? 1 : 0;
  r.scale = number(field(o, "scale", "rope"));
  r.freq = static_cast<const uint64_t*>(
      address(field(o, "freq", "rope"), ScalarType::Long, {r.dim / 2}, "rope freq", p));
}

void norm(sv_head_norm& n, PyObject* weight, PyObject* eps, int64_t D, const char* what,
          const Place& p) {
  if (!given(eps)) {
    if (given(weight)) refuse(std::string(what) + ": a norm's weight, but no eps");
    return;
  }
  n.eps = number(eps);
  if (!(n.eps > 0.f)) refuse("eps: expected a positive number");
  if (!given(weight)) return;
  const Tensor& w = tensor(weight, what);
  n.weight_dtype = dtype_of(w, what);
  n.weight = address(weight, w.scalar_type(), {D}, what, p);
}

int small(int64_t n, const char* what) {
  if (n > INT32_MAX) refuse(std::string(what) + ": out of range");
  return static_cast<int>(n);
}

Tensor empty(IntArrayRef shape, ScalarType dtype, const Place& p) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(p.device));
}

// New tensors belong to the current stream: a call on another one is given its
// results.
void own(PyObject* stream, const char* what) {
  if (given(stream)) refuse(std::string(what) + ": a call on a given stream needs its results");
}

// One kind of heads; `out` (kept in `keep`) is given, or allocated as `dtype`, or, for
// Ellipsis, x itself.
void heads(sv_heads& h, PyObject* x, PyObject* out, ScalarType dtype, PyObject* weight,
           PyObject* eps, PyObject* stream, const char* what, const Place& p, Tensor& keep) {
  const Tensor& t = tensor(x, what);
  const IntArrayRef shape = t.sizes();
  h.heads = small(shape[2], what);
  int64_t s[3];
  rows(t, shape, what, p, s);
  dtype_of(t, what);
  h.x = t.data_ptr();
  h.batch_stride = s[0];
  h.token_stride = s[1];
  h.head_stride = s[2];
  if (out == Py_Ellipsis) {
    keep = t;
  } else if (given(out)) {
    keep = tensor(out, what);
    rows(keep, shape, what, p, s);
  } else {
    own(stream, what);
    keep = empty(shape, dtype, p);
    for (int i = 0; i < 3; ++i) s[i] = shape[i] > 1 ? keep.stride(i) : 0;
  }
  h.out = keep.data_ptr();
  h.out_dtype = dtype_of(keep, what);
  h.out_batch_stride = s[0];
  h.out_token_stride = s[1];
  h.out_head_stride = s[2];
  norm(h.norm, weight, eps, shape[3], what, p);
}

void four(const Tensor& t, const char* what) {
  if (t.dim() != 4) refuse(std::string(what) + ": expected [B][T][heads][D], got " + text(t.sizes()));
}

// The packed structure for entry 0, else the call's results or status.
template <class A>
PyObject* call(PyObject* entry, const char* name, const A& a, const Tensor& workspace,
               PyObject* stream, std::initializer_list<const Tensor*> results) {
  void* const f = PyLong_AsVoidPtr(entry);
  if (f == nullptr) {
    if (PyErr_Occurred()) return nullptr;
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&a), sizeof(A));
  }
  if (!workspace.is_cuda()) refuse("libspecverify takes device tensors");
  // The library launches on the current device.
  const int dev = workspace.get_device();
  if (c10::cuda::current_device() != dev)
    refuse(std::string(name) + ": the tensors are on cuda:" + std::to_string(dev) +
           ", the current device is cuda:" + std::to_string(c10::cuda::current_device()));
  sv_stream_t st;
  if (given(stream)) {
    st = static_cast<sv_stream_t>(PyLong_AsVoidPtr(stream));
    if (PyErr_Occurred()) return nullptr;
  } else {
    st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }
  sv_status status;
  Py_BEGIN_ALLOW_THREADS
  status = reinterpret_cast<sv_status (*)(const A*, void*, size_t, sv_stream_t)>(f)(
      &a, workspace.data_ptr(), workspace.nbytes(), st);
  Py_END_ALLOW_THREADS
  if (status != SV_OK) return PyLong_FromLong(status);
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(results.size()));
  if (out == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : results) {
    PyObject* o = t->defined() ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (o == nullptr) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

bool arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// (entry, workspace, stream, q, q_out, k, k_out, start, num, offset, rope, q_weight,
// k_weight, eps) -> (q_out, k_out)
PyObject* rotate(PyObject*, PyObject* const* v, Py_ssize_t nv) {
  HANDLE_TH_ERRORS
  if (!arguments(nv, 14)) return nullptr;
  try {
    const Tensor& ws = tensor(v[1], "workspace");
    const Place p{ws.device()};
    const Tensor& q = tensor(v[3], "q");
    four(q, "q");
    sv_rotate_args a = {};
    const int64_t B = q.size(0), T = q.size(1), D = q.size(3);
    a.B = small(B, "q");
    a.T = small(T, "q");
    a.D = small(D, "q");
    a.dtype = dtype_of(q, "q");
    Tensor q_out, k_out;
    heads(a.q, v[3], v[4], q.scalar_type(), v[11], v[13], v[2], "q", p, q_out);
    if (given(v[5])) {
      const Tensor& k = tensor(v[5], "k");
      four(k, "k");
      if (k.size(0) != B || k.size(1) != T || k.size(3) != D || k.scalar_type() != q.scalar_type())
        refuse("k: expected [" + std::to_string(B) + "][" + std::to_string(T) + "][heads][" +
               std::to_string(D) + "] of q's dtype, got " + c10::toString(k.scalar_type()) + " " +
               text(k.sizes()));
      heads(a.k, v[5], v[6], k.scalar_type(), v[12], v[13], v[2], "k", p, k_out);
    } else if (given(v[12])) {
      refuse("k_weight: a norm's weight, but no k");
    }
    a.start = static_cast<const int32_t*>(address(v[7], ScalarType::Int, {B}, "start", p));
    a.num = static_cast<const int32_t*>(address(v[8], ScalarType::Int, {B}, "num", p));
    a.offset = static_cast<const int32_t*>(address(v[9], ScalarType::Int, {B, T}, "offset", p));
    rope(a.rope, v[10], p);
    return call(v[0], "sv_rotate", a, ws, v[2], {&q_out, &k_out});
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

void cache(sv_kv_cache& c, PyObject* o, PyObject* page_table, int64_t B, const Place& p) {
  const Tensor& k = tensor(field(o, "k", "cache"), "cache k");
  const Tensor& v = tensor(field(o, "v", "cache"), "cache v");
  if (k.scalar_type() != ScalarType::Float8_e4m3fn || k.dim() != 4)
    refuse("cache k: expected float8_e4m3fn [pages][heads][page][D], got " +
           std::string(c10::toString(k.scalar_type())) + " " + text(k.sizes()));
  const IntArrayRef s = k.sizes();
  bool same = v.scalar_type() == k.scalar_type() && v.sizes() == s;
  // (the stride of a dimension of size 1 says nothing)
  for (int i = 0; same && i < 4; ++i) same = s[i] <= 1 || v.stride(i) == k.stride(i);
  if (!same) refuse("cache v: expected k's dtype, shape and strides");
  if (k.stride(3) != 1 || k.stride(2) != s[3])
    refuse("cache: the tokens of a page and head must be contiguous");
  p.check(k);
  p.check(v);
  c.num_pages = small(s[0], "cache");
  c.Hkv = small(s[1], "cache");
  c.page_size = small(s[2], "cache");
  c.D = small(s[3], "cache");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.page_stride = s[0] > 1 ? k.stride(0) : 0;
  c.head_stride = s[1] > 1 ? k.stride(1) : s[2] * s[3];
  const IntArrayRef scales = s.slice(0, 2);
  c.k_scale = const_cast<float*>(static_cast<const float*>(
      address(field(o, "k_scale", "cache"), ScalarType::Float, scales, "k_scale", p)));
  c.v_scale = const_cast<float*>(static_cast<const float*>(
      address(field(o, "v_scale", "cache"), ScalarType::Float, scales, "v_scale", p)));
  const Tensor& table = tensor(page_table, "page_table");
  if (table.dim() != 2) refuse("page_table: expected contiguous int32 [B][slots]");
  c.slots = small(table.size(1), "page_table");
  c.page_table = static_cast<const int32_t*>(
      address(page_table, ScalarType::Int, {B, table.size(1)}, "page_table", p));
}

// (entry, workspace, stream, cache, page_table, kv_len, q, q_out, q_dtype, k_new, v_new,
// num_new, offset, rope, q_weight, k_weight, eps) -> (q_out,)
PyObject* kv_append(PyObject*, PyObject* const* v, Py_ssize_t nv) {
  HANDLE_TH_ERRORS
  if (!arguments(nv, 17)) return nullptr;
  try {
    const Tensor& ws = tensor(v[1], "workspace");
    const Place p{ws.device()};
    const Tensor& k = tensor(v[9], "k_new");
    const Tensor& vn = tensor(v[10], "v_new");
    four(k, "k_new");
    sv_kv_append_args a = {};
    const int64_t B = k.size(0), T = k.size(1);
    cache(a.cache, v[3], v[4], B, p);
    const int64_t D = a.cache.D, shape[4] = {B, T, a.cache.Hkv, D};
    a.B = small(B, "k_new");
    a.T = small(T, "k_new");
    a.dtype = dtype_of(k, "k_new");
    int64_t s[3];
    rows(k, shape, "k_new", p, s);
    a.k_new = k.data_ptr();
    a.k_batch_stride = s[0];
    a.k_token_stride = s[1];
    a.k_head_stride = s[2];
    if (vn.scalar_type() != k.scalar_type()) refuse("v_new: expected k_new's dtype");
    rows(vn, shape, "v_new", p, s);
    a.v_new = vn.data_ptr();
    a.v_batch_stride = s[0];
    a.v_token_stride = s[1];
    a.v_head_stride = s[2];
    Tensor q_out;
    if (given(v[6])) {
      const Tensor& q = tensor(v[6], "q");
      four(q, "q");
      if (q.size(0) != B || q.size(1) != T || q.size(3) != D || q.scalar_type() != k.scalar_type())
        refuse("q: expected [" + std::to_string(B) + "][" + std::to_string(T) + "][heads][" +
               std::to_string(D) + "] of k_new's dtype, got " + c10::toString(q.scalar_type()) + " " +
               text(q.sizes()));
      ScalarType dtype = q.scalar_type();
      if (given(v[8])) {
        if (!THPDtype_Check(v[8])) refuse("q_dtype: expected a dtype");
        dtype = reinterpret_cast<THPDtype*>(v[8])->scalar_type;
      }
      heads(a.q, v[6], v[7], dtype, v[14], v[16], v[2], "q", p, q_out);
    } else if (given(v[14])) {
      refuse("q_weight: a norm's weight, but no q");
    }
    norm(a.k_norm, v[15], v[16], D, "k_weight", p);
    a.kv_len = static_cast<const int32_t*>(address(v[5], ScalarType::Int, {B}, "kv_len", p));
    a.num_new = static_cast<const int32_t*>(address(v[11], ScalarType::Int, {B}, "num_new", p));
    a.offset = static_cast<const int32_t*>(address(v[12], ScalarType::Int, {B, T}, "offset", p));
    rope(a.rope, v[13], p);
    return call(v[0], "sv_kv_append", a, ws, v[2], {&q_out});
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (entry, workspace, stream, logits, R, tokens, num_rows, rows, temperature, top, allocate,
// logprobs, entropy, top_tokens, top_logprobs) -> (logprobs, entropy, top_tokens,
// top_logprobs); R None: that of tokens or rows, or all rows; allocate: all that is asked
// for, into new tensors
PyObject* token_logprobs(PyObject*, PyObject* const* v, Py_ssize_t nv) {
  HANDLE_TH_ERRORS
  if (!arguments(nv, 15)) return nullptr;
  try {
    const Tensor& ws = tensor(v[1], "workspace");
    const Place p{ws.device()};
    const Tensor& x = tensor(v[3], "logits");
    if (x.dim() != 3 || (x.size(2) > 1 && x.stride(2) != 1))
      refuse("logits: expected [B][N][V] with contiguous rows, got " + text(x.sizes()));
    if (x.scalar_type() != ScalarType::BFloat16 && x.scalar_type() != ScalarType::Float)
      refuse(std::string("logits must be bfloat16 or float32, got ") + c10::toString(x.scalar_type()));
    p.check(x);
    sv_token_logprobs_args a = {};
    const int64_t B = x.size(0);
    a.B = small(B, "logits");
    a.N = small(x.size(1), "logits");
    a.V = small(x.size(2), "logits");
    a.dtype = dtype_of(x, "logits");
    a.logits = x.data_ptr();
    a.batch_stride = B > 1 ? x.stride(0) : 0;
    a.row_stride = a.N > 1 ? x.stride(1) : 0;
    int64_t R = a.N, M = 0;
    bool each = false;  // tokens [B][R][M]
    if (given(v[5])) {
      const Tensor& t = tensor(v[5], "tokens");
      if (t.dim() != 2 && t.dim() != 3) refuse("tokens: expected [B][R] or [B][R][M]");
      R = t.size(1);
      each = t.dim() == 3;
      M = each ? t.size(2) : 1;
    } else if (given(v[7])) {
      const Tensor& t = tensor(v[7], "rows");
      if (t.dim() != 2) refuse("rows: expected [B][R]");
      R = t.size(1);
    }
    if (given(v[4])) R = whole(v[4], "R");
    a.R = small(R, "R");
    a.M = small(M, "tokens");
    a.top = whole(v[9], "top");
    if (a.top < 0 || a.top > SV_MAX_TOPK) refuse("top: expected 0 .. " + std::to_string(SV_MAX_TOPK));
    const int64_t wanted[3] = {B, R, M}, best[3] = {B, R, a.top};
    const IntArrayRef asked(wanted, each ? 3 : 2), one(wanted, 2), top(best, 3);
    a.tokens = static_cast<const int32_t*>(address(v[5], ScalarType::Int, asked, "tokens", p));
    a.num_rows = static_cast<const int32_t*>(address(v[6], ScalarType::Int, {B}, "num_rows", p));
    a.rows = static_cast<const int32_t*>(address(v[7], ScalarType::Int, one, "rows", p));
    a.temperature =
        static_cast<const float*>(address(v[8], ScalarType::Float, {B}, "temperature", p));
    Tensor out[4];
    if (truth(v[10])) {
      own(v[2], "logits");
      if (R < 0) refuse("R: out of range");
      if (given(v[5])) out[0] = empty(asked, ScalarType::Float, p);
      out[1] = empty(one, ScalarType::Float, p);
      if (a.top > 0) {
        out[2] = empty(top, ScalarType::Int, p);
        out[3] = empty(top, ScalarType::Float, p);
      }
    } else {
      if (given(v[11]) && !given(v[5])) refuse("logprobs: given, but no tokens");
      address(v[11], ScalarType::Float, asked, "logprobs", p);
      address(v[12], ScalarType::Float, one, "entropy", p);
      address(v[13], ScalarType::Int, top, "top_tokens", p);
      address(v[14], ScalarType::Float, top, "top_logprobs", p);
      for (int i = 0; i < 4; ++i)
        if (given(v[11 + i])) out[i] = THPVariable_Unpack(v[11 + i]);
    }
    auto at = [&](int i) { return out[i].defined() ? out[i].data_ptr() : nullptr; };
    a.logprob = static_cast<float*>(at(0));
    a.entropy = static_cast<float*>(at(1));
    a.top_token = static_cast<int32_t*>(at(2));
    a.top_logprob = static_cast<float*>(at(3));
    return call(v[0], "sv_token_logprobs", a, ws, v[2], {&out[0], &out[1], &out[2], &out[3]});
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}

PyMethodDef methods[] = {{"rotate", fast<rotate>(), METH_FASTCALL, nullptr},
                         {"kv_append", fast<kv_append>(), METH_FASTCALL, nullptr},
                         {"token_logprobs", fast<token_logprobs>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
