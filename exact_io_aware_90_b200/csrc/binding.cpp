// binding.cpp — the hot half of the Python wrappers in paged.py: argument checks on torch tensors, allocation of outputs
// and workspaces, the current stream, and the call of the C ABI (fa.h).  A decoding step's kernels take 3 to 10
// microseconds; checked and allocated from Python with ctypes, the calls took 9 to 28.
//
// Each function takes all its arguments by position, None for those that are not given, and raises ValueError or
// TypeError for arguments the wrappers refuse and FAError for a status of the library.  No C++ exception leaves it.
#include <Python.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <string>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fa.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct ValueProblem { std::string text; };
struct TypeProblem { std::string text; };
struct Status { int code; const char* where; };
struct PythonError {};  // already set

PyObject* g_error_class = nullptr;   // FAError
PyObject* g_memory_class = nullptr;  // torch.OutOfMemoryError

[[noreturn]] void refuse(const std::string& text) { throw ValueProblem{text}; }

std::string list(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

std::string describe(const Tensor& t) {
  return std::string(c10::toString(t.scalar_type())) + " " + list(t.sizes()) + " with strides " + list(t.strides()) + " on " + t.device().str();
}

// ---------------------------------------------------------------- arguments
struct Args {
  PyObject* const* v;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) throw TypeProblem{"too few arguments"};
    return v[i++];
  }
  bool none() const { return i < n && v[i] == Py_None; }
  const Tensor& tensor(const char* name) {
    PyObject* o = next();
    if (!THPVariable_Check(o)) throw TypeProblem{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
  }
  const Tensor* maybe(const char* name) {
    if (none()) {
      ++i;
      return nullptr;
    }
    return &tensor(name);
  }
  double real(const char* name) {
    const double x = PyFloat_AsDouble(next());
    if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
    (void)name;
    return x;
  }
  long long whole(const char* name) {
    PyObject* o = next();
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw PythonError{};
    (void)name;
    return x;
  }
  bool truth() {
    const int x = PyObject_IsTrue(next());
    if (x < 0) throw PythonError{};
    return x != 0;
  }
};

int as_int(int64_t x, const char* name) {
  if (x < INT32_MIN || x > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(x);
}

int code_of(ScalarType t, const char* name) {
  if (t == at::kBFloat16) return FA_BF16;
  if (t == at::kHalf) return FA_FP16;
  throw TypeProblem{std::string("unsupported dtype: ") + name + " must be bfloat16 or float16"};
}

void need_cuda(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor: got " + describe(t));
}

// [T, H, d] whose heads and features are packed: its heads and token stride.
struct Rows { int heads; int64_t stride; };
Rows rows_of(const Tensor& t, const char* name, ScalarType dtype, at::Device dev, int64_t T, int64_t d, int64_t heads = -1) {
  if (t.dim() != 3 || t.scalar_type() != dtype || t.device() != dev || t.size(0) != T || t.size(2) != d ||
      (heads >= 0 && t.size(1) != heads) || (d != 1 && t.stride(2) != 1) || (t.size(1) != 1 && t.stride(1) != d)) {
    std::ostringstream s;
    s << name << " must be " << c10::toString(dtype) << " [" << T << ", " << (heads >= 0 ? std::to_string(heads) : std::string("heads")) << ", " << d
      << "] on " << dev.str() << ", packed in heads and features (any token stride): got " << describe(t);
    refuse(s.str());
  }
  return {as_int(t.size(1), name), T != 1 ? t.stride(0) : t.size(1) * d};
}

void* flat(const Tensor& t, const char* name, ScalarType dtype, at::IntArrayRef shape, at::Device dev) {
  if (t.scalar_type() != dtype || t.sizes() != shape || t.device() != dev || !t.is_contiguous()) {
    std::ostringstream s;
    s << name << " must be contiguous " << c10::toString(dtype) << " " << list(shape) << " on " << dev.str() << ": got " << describe(t);
    refuse(s.str());
  }
  return t.data_ptr();
}

// A caller's workspace: as many bytes as its elements have, from its address on.  Of a slice with gaps or an expanded tensor
// that would be memory beside its own.
void check_workspace(const Tensor* t, at::Device dev) {
  if (t != nullptr && (t->device() != dev || !t->is_contiguous())) refuse("workspace must be contiguous and on " + dev.str() + ": got " + describe(*t));
}

// The device made current, and the stream of the call: the given one, else the device's current one.  Memory is
// allocated on that stream, so that the allocator reuses it in that stream's order.
struct Place {
  std::optional<c10::cuda::CUDAGuard> device;
  std::optional<c10::cuda::CUDAStreamGuard> own;
  cudaStream_t stream;
  at::Device dev;
  Place(Args& a, at::Device d) : dev(d) {
    if (d.index() != c10::cuda::current_device()) device.emplace(d);
    if (a.none()) {
      a.next();
      stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
    } else {
      PyObject* o = a.next();
      void* p = PyLong_AsVoidPtr(o);
      if (p == nullptr && PyErr_Occurred()) throw PythonError{};
      if (p == cudaStreamLegacy) p = nullptr;  // the default stream, which torch knows as 0
      stream = static_cast<cudaStream_t>(p);
      own.emplace(c10::cuda::getStreamFromExternal(stream, d.index()));
    }
  }
  Tensor empty(at::IntArrayRef shape, ScalarType dtype) const {
    return at::detail::empty_cuda(shape, dtype, dev, std::nullopt);
  }
};

void check(int status, const char* where) {
  if (status != FA_OK) throw Status{status, where};
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

template <typename... T>
PyObject* wrap_tuple(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (r == nullptr) throw PythonError{};
  Py_ssize_t i = 0;
  auto put = [&](const Tensor* x) {
    PyObject* o = x == nullptr ? Py_NewRef(Py_None) : wrap(*x);
    if (o == nullptr) {
      Py_DECREF(r);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  };
  (put(t), ...);
  return r;
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const ValueProblem& e) {
    PyErr_SetString(PyExc_ValueError, e.text.c_str());
  } catch (const TypeProblem& e) {
    PyErr_SetString(PyExc_TypeError, e.text.c_str());
  } catch (const Status& e) {
    PyObject* x = PyObject_CallFunction(g_error_class, "is", e.code, e.where);
    if (x != nullptr) {
      PyErr_SetObject(g_error_class, x);
      Py_DECREF(x);
    }
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory_class, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ---------------------------------------------------------------- shared groups of arguments
// cos, sin, positions, sections (a tuple or None); cos None with `optional`: no rotation.
struct Rope {
  const float *cos = nullptr, *sin = nullptr;
  const int32_t* positions = nullptr;
  int rot = 0, rows = 0, axes = 1;
  int sections[16] = {};
  bool has_sections = false;
  const int* section_ptr() const { return has_sections ? sections : nullptr; }
};

Rope rope_of(Args& a, int64_t T, at::Device dev, bool optional, bool need_positions) {
  Rope r;
  const Tensor *cos = a.maybe("cos"), *sin = a.maybe("sin"), *pos = a.maybe("positions");
  PyObject* sec = a.next();
  if ((cos == nullptr) != (sin == nullptr)) refuse("cos and sin come in pairs");
  if (cos == nullptr) {
    if (!optional) refuse("cos and sin are required");
    if (pos != nullptr || sec != Py_None) refuse("positions and sections need cos and sin");
    return r;
  }
  if (need_positions && pos == nullptr) refuse("positions are required");
  if (cos->dim() != 2) refuse("cos and sin must be [rows, rot_dim / 2] tables: got " + describe(*cos));
  const auto shape = cos->sizes();
  r.cos = static_cast<const float*>(flat(*cos, "cos", at::kFloat, shape, dev));
  r.sin = static_cast<const float*>(flat(*sin, "sin", at::kFloat, shape, dev));
  r.rows = as_int(shape[0], "the table's rows");
  r.rot = as_int(2 * shape[1], "rot_dim");
  if (sec != Py_None) {
    PyObject* seq = PySequence_Fast(sec, "sections must be a sequence of whole numbers");
    if (seq == nullptr) throw PythonError{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    long long sum = 0;
    bool good = n >= 1 && n <= 16;
    for (Py_ssize_t i = 0; good && i < n; ++i) {
      const long long x = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
      if (x == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw PythonError{};
      }
      good = x >= -(1 << 20) && x <= (1 << 20);
      r.sections[i] = static_cast<int>(x);
      sum += x;
    }
    Py_DECREF(seq);
    if (!good || sum != shape[1]) refuse("sections must add up to rot_dim / 2");
    r.axes = static_cast<int>(n);
    r.has_sections = true;
  }
  if (pos != nullptr) {
    if (pos->scalar_type() != at::kInt || pos->device() != dev || !pos->is_contiguous() || pos->dim() < 1 || pos->size(-1) != T ||
        pos->numel() != r.axes * T) {
      std::ostringstream s;
      s << "positions must be contiguous int32 [" << r.axes << ", " << T << "] on " << dev.str() << ": got " << describe(*pos);
      refuse(s.str());
    }
    r.positions = pos->const_data_ptr<int32_t>();
  }
  return r;
}

struct Weights { const void *q = nullptr, *k = nullptr; };
Weights weights_of(const Tensor* wq, const Tensor* wk, int64_t d, ScalarType dtype, at::Device dev) {
  Weights w;
  if (wq != nullptr) w.q = flat(*wq, "wq", dtype, {d}, dev);
  if (wk != nullptr) w.k = flat(*wk, "wk", dtype, {d}, dev);
  return w;
}

// k_cache, v_cache, page_table
struct Cache {
  const void *k, *v;
  const int32_t* table;
  int d, heads, page_size, pages, B, most, format;
  ScalarType dtype;
};
Cache cache_of(const Tensor& k, const Tensor& v, const Tensor& table, at::Device dev) {
  if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || k.device() != dev || v.device() != dev ||
      !k.is_contiguous() || !v.is_contiguous()) {
    std::ostringstream s;
    s << "k_cache and v_cache must be alike, contiguous, [num_pages, Hk, page_size, row] on " << dev.str() << ": got " << describe(k) << " and " << describe(v);
    refuse(s.str());
  }
  if (table.dim() != 2 || table.scalar_type() != at::kInt || table.device() != dev || !table.is_contiguous()) {
    std::ostringstream s;
    s << "page_table must be contiguous int32 [B, max_pages] on " << dev.str() << ": got " << describe(table);
    refuse(s.str());
  }
  Cache c;
  c.dtype = k.scalar_type();
  int64_t d = k.size(3);
  c.format = FA_CACHE_16BIT;
  if (c.dtype == at::kByte) {
    if (d % 5 != 0) refuse("a 4-bit cache has rows of 5·d/8 bytes: got " + describe(k));
    d = d / 5 * 8;
    c.format = FA_CACHE_INT4;
  } else {
    code_of(c.dtype, "a 16-bit cache");
  }
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.table = table.const_data_ptr<int32_t>();
  c.d = as_int(d, "d");
  c.pages = as_int(k.size(0), "num_pages");
  c.heads = as_int(k.size(1), "Hk");
  c.page_size = as_int(k.size(2), "page_size");
  c.B = as_int(table.size(0), "B");
  c.most = as_int(table.size(1), "max_pages");
  return c;
}

// ---------------------------------------------------------------- entry points
// q, k, cos, sin, positions, sections, wq, wk, eps, interleaved, q_out, k_out, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{args, n};
    const Tensor& q = a.tensor("q");
    const Tensor& k = a.tensor("k");
    need_cuda(q, "q");
    if (q.dim() != 3) refuse("q must be [T, heads, d]: got " + describe(q));
    const auto dev = q.device();
    const auto dtype = q.scalar_type();
    const int64_t T = q.size(0), d = q.size(2);
    const Rows rq = rows_of(q, "q", dtype, dev, T, d), rk = rows_of(k, "k", dtype, dev, T, d);
    const int code = code_of(dtype, "q");
    const Rope r = rope_of(a, T, dev, false, true);
    const Tensor *wq = a.maybe("wq"), *wk = a.maybe("wk");
    if ((wq == nullptr) != (wk == nullptr)) refuse("norm weights come in pairs");
    const Weights w = weights_of(wq, wk, d, dtype, dev);
    const double eps = a.real("eps");
    const bool inter = a.truth();
    const Tensor *qo = a.maybe("q_out"), *ko = a.maybe("k_out");
    const Rows ro = qo != nullptr ? rows_of(*qo, "q_out", dtype, dev, T, d, rq.heads) : Rows{rq.heads, rq.heads * d};
    const Rows rp = ko != nullptr ? rows_of(*ko, "k_out", dtype, dev, T, d, rk.heads) : Rows{rk.heads, rk.heads * d};
    const Place at_(a, dev);
    const Tensor q_out = qo != nullptr ? *qo : at_.empty({T, rq.heads, d}, dtype);
    const Tensor k_out = ko != nullptr ? *ko : at_.empty({T, rk.heads, d}, dtype);
    check(fa_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), w.q, w.k, r.cos, r.sin, r.positions,
                          as_int(T, "T"), rq.heads, rk.heads, as_int(d, "d"), rq.stride, rk.stride, ro.stride, rp.stride, r.rot, r.rows,
                          r.axes, r.section_ptr(), inter, static_cast<float>(eps), code, at_.stream),
          "fa_qk_norm_rope");
    return wrap_tuple(&q_out, &k_out);
  });
}

// dq_out, dk_out, cos, sin, positions, sections, q, k, wq, wk, eps, interleaved, dq, dk, dwq, dwk, workspace, stream
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{args, n};
    const Tensor& gq = a.tensor("dq_out");
    const Tensor& gk = a.tensor("dk_out");
    need_cuda(gq, "dq_out");
    if (gq.dim() != 3) refuse("dq_out must be [T, heads, d]: got " + describe(gq));
    const auto dev = gq.device();
    const auto dtype = gq.scalar_type();
    const int64_t T = gq.size(0), d = gq.size(2);
    const Rows rgq = rows_of(gq, "dq_out", dtype, dev, T, d), rgk = rows_of(gk, "dk_out", dtype, dev, T, d);
    const int code = code_of(dtype, "dq_out");
    const Rope r = rope_of(a, T, dev, false, true);
    const Tensor *q = a.maybe("q"), *k = a.maybe("k"), *wq = a.maybe("wq"), *wk = a.maybe("wk");
    if ((wq == nullptr) != (wk == nullptr)) refuse("norm weights come in pairs");
    const bool norm = wq != nullptr;
    const Weights w = weights_of(wq, wk, d, dtype, dev);
    Rows rq{0, 0}, rk{0, 0};
    if (norm) {
      if (q == nullptr || k == nullptr) refuse("q and k are needed for the norm's gradient");
      rq = rows_of(*q, "q", dtype, dev, T, d, rgq.heads);
      rk = rows_of(*k, "k", dtype, dev, T, d, rgk.heads);
    }
    const double eps = a.real("eps");
    const bool inter = a.truth();
    const Tensor *oq = a.maybe("dq"), *ok = a.maybe("dk"), *owq = a.maybe("dwq"), *owk = a.maybe("dwk"), *ows = a.maybe("workspace");
    const Rows rdq = oq != nullptr ? rows_of(*oq, "dq", dtype, dev, T, d, rgq.heads) : Rows{rgq.heads, rgq.heads * d};
    const Rows rdk = ok != nullptr ? rows_of(*ok, "dk", dtype, dev, T, d, rgk.heads) : Rows{rgk.heads, rgk.heads * d};
    if (norm && owq != nullptr) flat(*owq, "dwq", at::kFloat, {d}, dev);
    if (norm && owk != nullptr) flat(*owk, "dwk", at::kFloat, {d}, dev);
    check_workspace(ows, dev);
    const Place at_(a, dev);
    const Tensor dq = oq != nullptr ? *oq : at_.empty({T, rgq.heads, d}, dtype), dk = ok != nullptr ? *ok : at_.empty({T, rgk.heads, d}, dtype);
    Tensor dwq, dwk, ws;
    if (norm) {
      dwq = owq != nullptr ? *owq : at_.empty({d}, at::kFloat);
      dwk = owk != nullptr ? *owk : at_.empty({d}, at::kFloat);
      ws = ows != nullptr ? *ows : at_.empty({static_cast<int64_t>(fa_qk_norm_rope_bwd_workspace_bytes(static_cast<int>(d)) + 256)}, at::kByte);
    }
    check(fa_qk_norm_rope_bwd(gq.data_ptr(), gk.data_ptr(), norm ? q->data_ptr() : nullptr, norm ? k->data_ptr() : nullptr, w.q, w.k, r.cos,
                              r.sin, r.positions, dq.data_ptr(), dk.data_ptr(), norm ? dwq.data_ptr<float>() : nullptr,
                              norm ? dwk.data_ptr<float>() : nullptr, as_int(T, "T"), rgq.heads, rgk.heads, as_int(d, "d"), rgq.stride,
                              rgk.stride, rq.stride, rk.stride, rdq.stride, rdk.stride, r.rot, r.rows, r.axes, r.section_ptr(), inter,
                              static_cast<float>(eps), code, norm ? ws.data_ptr() : nullptr, norm ? ws.nbytes() : 0, at_.stream),
          "fa_qk_norm_rope_bwd");
    const Tensor* none = nullptr;
    return norm ? wrap_tuple(&dq, &dk, &dwq, &dwk) : wrap_tuple(&dq, &dk, none, none);
  });
}

// k, v, k_cache, v_cache, page_table, seqlens_k, cos, sin, positions, sections, q, wq, wk, eps, interleaved, cu_seqlens, q_out, stream
PyObject* cache_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{args, n};
    const Tensor& k = a.tensor("k");
    const Tensor& v = a.tensor("v");
    need_cuda(k, "k");
    if (k.dim() != 3) refuse("k must be [T, heads, d]: got " + describe(k));
    const auto dev = k.device();
    const auto dtype = k.scalar_type();
    const int64_t T = k.size(0), d = k.size(2);
    const Rows rk = rows_of(k, "k", dtype, dev, T, d), rv = rows_of(v, "v", dtype, dev, T, d, rk.heads);
    const int code = code_of(dtype, "k");
    const Tensor& kc = a.tensor("k_cache");
    const Tensor& vc = a.tensor("v_cache");
    const Cache c = cache_of(kc, vc, a.tensor("page_table"), dev);
    if (c.d != d || c.heads != rk.heads || (c.format == FA_CACHE_16BIT && c.dtype != dtype))
      refuse("the cache's heads, d and dtype must be those of k and v");
    const auto* lens = static_cast<const int32_t*>(flat(a.tensor("seqlens_k"), "seqlens_k", at::kInt, {c.B}, dev));
    const Rope r = rope_of(a, T, dev, true, false);
    const Tensor *q = a.maybe("q"), *wq = a.maybe("wq"), *wk = a.maybe("wk");
    if (q == nullptr && wq != nullptr) refuse("wq without q");
    if (q != nullptr && (wq == nullptr) != (wk == nullptr)) refuse("norm weights come in pairs");
    const Weights w = weights_of(wq, wk, d, dtype, dev);
    const double eps = a.real("eps");
    const bool inter = a.truth();
    const Tensor *cu = a.maybe("cu_seqlens"), *qo = a.maybe("q_out");
    const auto* cup = cu == nullptr ? nullptr : static_cast<const int32_t*>(flat(*cu, "cu_seqlens", at::kInt, {c.B + 1}, dev));
    Rows rq{0, 0}, ro{0, 0};
    if (q != nullptr) {
      rq = rows_of(*q, "q", dtype, dev, T, d);
      ro = qo != nullptr ? rows_of(*qo, "q_out", dtype, dev, T, d, rq.heads) : Rows{rq.heads, rq.heads * d};
    } else if (qo != nullptr) {
      refuse("q_out without q");
    }
    const Place at_(a, dev);
    Tensor q_out;
    if (q != nullptr) q_out = qo != nullptr ? *qo : at_.empty({T, rq.heads, d}, dtype);
    check(fa_cache_append(q != nullptr ? q->data_ptr() : nullptr, k.data_ptr(), v.data_ptr(), q != nullptr ? q_out.data_ptr() : nullptr,
                          const_cast<void*>(c.k), const_cast<void*>(c.v), w.q, w.k, r.cos, r.sin, r.positions, c.table, lens, cup, c.B,
                          as_int(T, "T"), rq.heads, rk.heads, as_int(d, "d"), rq.stride, rk.stride, rv.stride, ro.stride, c.page_size, c.pages,
                          c.most, r.rot, r.rows, r.axes, r.section_ptr(), inter, static_cast<float>(eps), code, c.format, at_.stream),
          "fa_cache_append");
    if (q == nullptr) Py_RETURN_NONE;
    return wrap(q_out);
  });
}

// k_cache, v_cache, page_table, cu_seqlens_k, total_keys, starts, dtype code (-1: k's, or bf16), k, v, stream
PyObject* cache_gather(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{args, n};
    const Tensor& kc = a.tensor("k_cache");
    const Tensor& vc = a.tensor("v_cache");
    need_cuda(kc, "k_cache");
    const auto dev = kc.device();
    const Cache c = cache_of(kc, vc, a.tensor("page_table"), dev);
    const Tensor* cu = a.maybe("cu_seqlens_k");
    const long long total = a.whole("total_keys");
    const Tensor* starts = a.maybe("starts");
    long long asked = a.whole("dtype");
    const Tensor *ko = a.maybe("k"), *vo = a.maybe("v");
    if (c.format == FA_CACHE_16BIT) {
      const int own = code_of(c.dtype, "a 16-bit cache");
      if (asked >= 0 && asked != own) refuse("a 16-bit cache is read in its own dtype");
      asked = own;
    } else if (asked < 0) {
      asked = ko != nullptr ? code_of(ko->scalar_type(), "k") : FA_BF16;
    }
    const ScalarType dtype = asked == FA_BF16 ? at::kBFloat16 : at::kHalf;
    if (total < 1) throw Status{FA_ERR_INVALID_ARG, "fa_cache_gather"};
    const auto* cup = cu == nullptr ? nullptr : static_cast<const int32_t*>(flat(*cu, "cu_seqlens_k", at::kInt, {c.B + 1}, dev));
    const auto* sp = starts == nullptr ? nullptr : static_cast<const int32_t*>(flat(*starts, "starts", at::kInt, {c.B}, dev));
    if (ko != nullptr) flat(*ko, "k", dtype, {total, c.heads, c.d}, dev);
    if (vo != nullptr) flat(*vo, "v", dtype, {total, c.heads, c.d}, dev);
    const Place at_(a, dev);
    const Tensor k = ko != nullptr ? *ko : at_.empty({total, c.heads, c.d}, dtype), v = vo != nullptr ? *vo : at_.empty({total, c.heads, c.d}, dtype);
    check(fa_cache_gather(c.k, c.v, k.data_ptr(), v.data_ptr(), c.table, cup, sp, c.B, as_int(total, "total_keys"), c.heads, c.d, c.page_size,
                          c.pages, c.most, static_cast<int>(asked), c.format, at_.stream),
          "fa_cache_gather");
    return wrap_tuple(&k, &v);
  });
}

// q, k_cache, v_cache, page_table, seqlens_k, max_seqlen_k (None: the table's capacity), scale (None: 1/√d), out, lse, workspace, stream
PyObject* decode_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a{args, n};
    const Tensor& q = a.tensor("q");
    need_cuda(q, "q");
    const auto dev = q.device();
    const auto dtype = q.scalar_type();
    const Tensor& kc = a.tensor("k_cache");
    const Tensor& vc = a.tensor("v_cache");
    const Cache c = cache_of(kc, vc, a.tensor("page_table"), dev);
    const int64_t dim = q.dim();
    if ((dim != 3 && dim != 4) || q.size(0) != c.B || q.size(dim - 1) != c.d || (c.format == FA_CACHE_16BIT && c.dtype != dtype) ||
        !q.is_contiguous())
      refuse("q must be contiguous, [B, H, d] or [B, Nq, H, d] with the page table's B and the cache's d and dtype: got " + describe(q));
    const int code = code_of(dtype, "q");
    const int Nq = dim == 4 ? as_int(q.size(1), "Nq") : 1, H = as_int(q.size(dim - 2), "H");
    const auto* lens = static_cast<const int32_t*>(flat(a.tensor("seqlens_k"), "seqlens_k", at::kInt, {c.B}, dev));
    int64_t Nk = static_cast<int64_t>(c.most) * c.page_size;
    if (a.none()) a.next();
    else Nk = a.whole("max_seqlen_k");
    double scale = 1.0 / std::sqrt(static_cast<double>(c.d));
    if (a.none()) a.next();
    else scale = a.real("scale");
    const Tensor *oo = a.maybe("out"), *ol = a.maybe("lse"), *ow = a.maybe("workspace");
    const auto rows = q.sizes().slice(0, dim - 1);
    if (oo != nullptr) flat(*oo, "out", dtype, q.sizes(), dev);
    if (ol != nullptr) flat(*ol, "lse", at::kFloat, rows, dev);
    check_workspace(ow, dev);
    const int bound = as_int(Nk, "max_seqlen_k");
    const Place at_(a, dev);
    const Tensor out = oo != nullptr ? *oo : at_.empty(q.sizes(), dtype), lse = ol != nullptr ? *ol : at_.empty(rows, at::kFloat);
    const size_t need = ow != nullptr ? 0 : fa_decode_paged_workspace_bytes(c.B, Nq, H, c.heads, bound, c.d);
    Tensor ws;  // small calls need none
    if (ow != nullptr) ws = *ow;
    else if (need > 0) ws = at_.empty({static_cast<int64_t>(need)}, at::kByte);
    check(fa_decode_paged(q.data_ptr(), c.k, c.v, out.data_ptr(), lse.data_ptr<float>(), c.table, lens, c.B, Nq, H, c.heads, bound, c.d,
                          static_cast<float>(scale), c.page_size, c.pages, c.most, code, c.format, ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0,
                          at_.stream),
          "fa_decode_paged");
    return wrap_tuple(&out, &lse);
  });
}

// Called once by paged.py before anything else.
PyObject* set_error_classes(PyObject*, PyObject* classes) {
  PyObject *error, *memory;
  if (!PyArg_ParseTuple(classes, "OO", &error, &memory)) return nullptr;
  g_error_class = Py_NewRef(error);
  g_memory_class = Py_NewRef(memory);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(qk_norm_rope), FAST(qk_norm_rope_backward), FAST(cache_append), FAST(cache_gather), FAST(decode_paged),
                         {"set_error_classes", set_error_classes, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
