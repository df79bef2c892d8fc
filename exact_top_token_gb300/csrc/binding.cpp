// binding.cpp -- the Python entry points of the operators around the selection
// (rope, cache_write, cache_read, attend, attend_backward) and of the cache in pages
// (page_write, attend_pages, page_fork, page_free, page_grow, page_compact, page_copy):
// checks of tensors, the results' allocation and the call of the C ABI. They also serve single tokens, where
// a call's time is the host's: written in Python around a foreign call of twenty
// arguments, attend took the host 20.5 us a call, rope 14.4, cache_read 14.0 and
// cache_write 9.1; here 6.8, 3.6, 4.1 and 5.5, of which the launch is the most.
//
// The C entry points come as addresses (init), so that this module links to nothing
// of the library; it is built against the torch that imports it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/record_stream.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>

#include "hytopk.h"

namespace {

decltype(&hytopk_rope) p_rope;
decltype(&hytopk_cache_write) p_cache_write;
decltype(&hytopk_cache_read) p_cache_read;
decltype(&hytopk_attend) p_attend;
decltype(&hytopk_attend_backward) p_attend_backward;
decltype(&hytopk_attend_pages_workspace_size) p_attend_pages_workspace_size;
decltype(&hytopk_attend_pages) p_attend_pages;
decltype(&hytopk_page_write) p_page_write;
decltype(&hytopk_page_workspace_size) p_page_workspace_size;
decltype(&hytopk_page_fork) p_page_fork;
decltype(&hytopk_page_free) p_page_free;
decltype(&hytopk_page_grow) p_page_grow;
decltype(&hytopk_page_compact) p_page_compact;
decltype(&hytopk_page_copy) p_page_copy;
PyObject* status_error;  // the package's exception class
PyObject* memory_error;  // torch's

struct Raised {};  // a Python exception is set

template <class... A>
[[noreturn]] void raise(PyObject* type, const A&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  PyErr_SetString(type, s.str().c_str());
  throw Raised{};
}

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, name, " must be a tensor");
  return THPVariable_Unpack(o);
}

enum { BF16 = 1 << HYTOPK_ELEM_BF16, E4M3 = 1 << HYTOPK_ELEM_E4M3, F32 = 1 << HYTOPK_ELEM_F32 };

hytopk_elem elem(const char* name, at::ScalarType t, int allowed) {
  int code = -1;
  if (t == at::kBFloat16) code = HYTOPK_ELEM_BF16;
  if (t == at::kFloat) code = HYTOPK_ELEM_F32;
  if (t == at::kFloat8_e4m3fn || t == at::kByte) code = HYTOPK_ELEM_E4M3;
  if (code < 0 || !(allowed >> code & 1)) {
    const char* sep = "";
    std::string list;
    for (auto [bit, text] : {std::pair{BF16, "bfloat16"}, {F32, "float32"}, {E4M3, "float8_e4m3fn"}})
      if (allowed & bit) {
        list += sep;
        list += text;
        sep = " or ";
      }
    raise(PyExc_TypeError, name, " must be ", list, ", got ", t);
  }
  return static_cast<hytopk_elem>(code);
}

at::ScalarType dtype_or(PyObject* o, at::ScalarType otherwise) {
  if (!given(o)) return otherwise;
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, "dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// A contiguous tensor of this type and shape on this device; its pointer.
void* need(const char* name, const at::Tensor& t, at::Device device, at::ScalarType type,
           at::IntArrayRef shape) {
  if (t.device() != device)
    raise(PyExc_ValueError, name, " is on ", t.device(), ", expected ", device);
  if (!t.is_contiguous()) raise(PyExc_ValueError, name, " must be contiguous");
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, name, " must be ", type, ", got ", t.scalar_type());
  if (t.sizes() != shape)
    raise(PyExc_ValueError, name, " has shape ", t.sizes(), ", expected ", shape);
  return t.data_ptr();
}
void* need(const char* name, PyObject* o, at::Device device, at::ScalarType type,
           at::IntArrayRef shape) {
  return need(name, tensor(name, o), device, type, shape);
}

// [rows, heads, d] or [rows, d], strides in elements. A stride of an axis of length
// 1 is never used and is replaced by a packed one.
struct Rows {
  int64_t n, H, d, row, head;
};
Rows rows(const char* name, const at::Tensor& t) {
  const auto shape = t.sizes();
  const auto st = t.strides();
  if (shape.size() != 2 && shape.size() != 3)
    raise(PyExc_ValueError, name, " must be [rows, heads, d] or [rows, d]");
  if (!t.is_cuda()) raise(PyExc_ValueError, "inputs must be CUDA tensors");
  const bool three = shape.size() == 3;
  Rows r{shape[0], three ? shape[1] : 1, shape.back(), st[0], three ? st[1] : 0};
  if (st.back() != 1 && r.d > 1)
    raise(PyExc_ValueError, name, ": the last axis must be contiguous");
  if (r.H == 1) r.head = r.d;
  if (r.n <= 1) r.row = r.H * r.head;
  for (int64_t x : {r.n, r.H, r.d})
    if (x > INT32_MAX) raise(PyExc_ValueError, name, " has an axis of 2^31 or more");
  return r;
}
Rows packed_rows(const char* name, const at::Tensor& t) {
  const Rows r = rows(name, t);
  if (r.head != r.d) raise(PyExc_ValueError, name, ": heads must be contiguous within a row");
  return r;
}

uint32_t* status_ptr(PyObject* o, at::Device device) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor("status", o);
  if (t.element_size() != 4 || t.numel() < 1 || t.device() != device)
    raise(PyExc_ValueError, "status must be a 32-bit integer tensor on the inputs' device");
  return static_cast<uint32_t*>(t.data_ptr());
}

// Where a call runs: the tensors' device, which is current while this lives (the C entry
// points launch on the current one), and the device's current stream, or the one given. A
// stream given is current too, so that results are taken from its memory: the caller's
// stream's may still be read there by work that was launched before it was freed.
class Place {
 public:
  Place(PyObject* o, at::Device device) : caller_(c10::cuda::getCurrentCUDAStream(device.index())) {
    // (set and restored only where it differs; the question takes 0.1 us of a call)
    if (c10::cuda::current_device() != device.index()) device_.set_device(device);
    stream_ = caller_.stream();
    if (!given(o)) return;
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Raised{};
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised{};
    stream_ = static_cast<cudaStream_t>(p);
    if (stream_ != caller_.stream())
      other_.reset_stream(c10::cuda::getStreamFromExternal(stream_, device.index()));
  }
  cudaStream_t stream() const { return stream_; }
  // A result of a call on a stream given. Made here it is read on the caller's stream, so it
  // is recorded there: once dropped, the given stream does not take it anew before that is
  // done. One that the caller gave (`own`) is recorded with the stream that writes it.
  void result(const at::Tensor& t, bool own = false) const {
    if (stream_ == caller_.stream()) return;
    t.record_stream(own ? other_.current_stream()->unwrap() : caller_.unwrap());
  }

 private:
  c10::cuda::OptionalCUDAGuard device_;
  c10::cuda::CUDAStream caller_;
  cudaStream_t stream_;
  c10::cuda::OptionalCUDAStreamGuard other_;
};

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}
int integer(PyObject* o) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x < INT32_MIN || x > INT32_MAX ? -1 : static_cast<int>(x);  // (-1 is refused)
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised{};
  return x != 0;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

// Other Python threads run while this lives; taken back on every way out of its scope:
// a pointer asked of a tensor that holds no memory (inside a vmap) throws.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

template <class F>
void call(const char* what, F&& f) {
  const hytopk_status st = [&] {
    Unlocked u;
    return f();
  }();
  if (st == HYTOPK_OK) return;
  PyObject* args = Py_BuildValue("(is)", static_cast<int>(st), what);
  if (args) PyErr_SetObject(status_error, args);
  Py_XDECREF(args);
  throw Raised{};
}

PyObject* ref(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// The result of f, or NULL with a Python exception: nothing is thrown through Python.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(memory_error, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

hytopk_rope_params rope_params(PyObject* positions, PyObject* inv_freq, int64_t n,
                               at::Device device, PyObject* first, PyObject* interleaved,
                               bool inverse, PyObject* mscale) {
  const at::Tensor& f = tensor("inv_freq", inv_freq);
  if (f.dim() != 1) raise(PyExc_ValueError, "inv_freq must be [rot / 2]");
  hytopk_rope_params p{};
  p.positions = static_cast<int32_t*>(need("positions", positions, device, at::kInt, {n}));
  p.inv_freq = static_cast<float*>(need("inv_freq", f, device, at::kFloat, f.sizes()));
  p.rot = static_cast<int>(2 * f.size(0));
  p.first = integer(first);
  p.interleaved = truth(interleaved);
  p.inverse = inverse;
  p.mscale = static_cast<float>(number(mscale));
  return p;
}

// rope(x, positions, inv_freq, first, interleaved, mscale, inverse, out, status, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 10, [&]() -> PyObject* {
    const at::Tensor& x = tensor("x", a[0]);
    const Rows r = rows("x", x);
    const at::Device dev = x.device();
    const hytopk_elem type = elem("x", x.scalar_type(), BF16 | F32);
    const auto params = rope_params(a[1], a[2], r.n, dev, a[3], a[4], truth(a[6]), a[5]);
    const Place place(a[9], dev);
    at::Tensor made;
    Rows o{r.n, r.H, r.d, r.H * r.d, r.d};
    const bool own = given(a[7]);
    if (own) {
      const at::Tensor& out = tensor("out", a[7]);
      if (out.sizes() != x.sizes() || out.scalar_type() != x.scalar_type() || out.device() != dev)
        raise(PyExc_ValueError, "out must match x in shape, type and device");
      o = rows("out", out);
    } else {
      made = empty(x.sizes(), x.scalar_type(), dev);
    }
    void* out = own ? THPVariable_Unpack(a[7]).data_ptr() : made.data_ptr();
    uint32_t* status = status_ptr(a[8], dev);
    place.result(own ? THPVariable_Unpack(a[7]) : made, own);
    call("hytopk_rope", [&] {
      return p_rope(x.data_ptr(), r.row, r.head, type, r.n, r.H, r.d, &params, out, o.row, o.head,
                    status, place.stream());
    });
    return own ? ref(a[7]) : THPVariable_Wrap(std::move(made));
  });
}

struct Cache {
  Rows r;
  hytopk_elem type;
  float* scale;
};
Cache cache_of(const at::Tensor& c, PyObject* scale) {
  Cache k{rows("cache", c), HYTOPK_ELEM_BF16, nullptr};
  if (!c.is_contiguous()) raise(PyExc_ValueError, "cache must be contiguous");
  k.type = elem("cache", c.scalar_type(), E4M3 | BF16);
  if ((k.type == HYTOPK_ELEM_E4M3) != given(scale))
    raise(PyExc_ValueError, "an e4m3 cache needs cache_scale, a bf16 cache takes none");
  if (given(scale))
    k.scale = static_cast<float*>(need("cache_scale", scale, c.device(), at::kFloat,
                                       c.sizes().slice(0, c.dim() - 1)));
  return k;
}

// cache_write(x, cache, cache_scale, slots, positions, inv_freq, first, interleaved, mscale,
//             status, stream)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 11, [&]() -> PyObject* {
    const at::Tensor& x = tensor("x", a[0]);
    const Rows r = rows("x", x);
    const at::Device dev = x.device();
    const hytopk_elem type = elem("x", x.scalar_type(), BF16 | F32);
    const at::Tensor& cache = tensor("cache", a[1]);
    const Cache c = cache_of(cache, a[2]);
    if (cache.device() != dev || c.r.H != r.H || c.r.d != r.d)
      raise(PyExc_ValueError, "cache rows are ", c.r.H, " x ", c.r.d, " on ", cache.device(),
            ", expected ", r.H, " x ", r.d, " on ", dev);
    if (given(a[4]) != given(a[5]))
      raise(PyExc_ValueError, "positions and inv_freq go together");
    hytopk_rope_params params{};
    if (given(a[4])) params = rope_params(a[4], a[5], r.n, dev, a[6], a[7], false, a[8]);
    const int32_t* slots =
        given(a[3]) ? static_cast<int32_t*>(need("slots", a[3], dev, at::kInt, {r.n})) : nullptr;
    uint32_t* status = status_ptr(a[9], dev);
    const Place place(a[10], dev);
    call("hytopk_cache_write", [&] {
      return p_cache_write(x.data_ptr(), r.row, r.head, type, r.n, r.H, r.d,
                           given(a[4]) ? &params : nullptr, slots, cache.data_ptr(), c.type,
                           c.scale, c.r.n, status, place.stream());
    });
    return ref(a[1]);
  });
}

// cache_read(cache, cache_scale, slots, dtype, out, status, stream)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 7, [&]() -> PyObject* {
    const at::Tensor& cache = tensor("cache", a[0]);
    const Cache c = cache_of(cache, a[1]);
    const at::Device dev = cache.device();
    int64_t n = c.r.n;
    const int32_t* slots = nullptr;
    if (given(a[2])) {
      const at::Tensor& s = tensor("slots", a[2]);
      if (s.dim() != 1) raise(PyExc_ValueError, "slots must be [m]");
      n = s.size(0);
      if (n > INT32_MAX) raise(PyExc_ValueError, "slots has 2^31 entries or more");
      slots = static_cast<int32_t*>(need("slots", s, dev, at::kInt, {n}));
    }
    at::DimVector shape(cache.sizes().begin(), cache.sizes().end());
    shape[0] = n;
    at::Tensor out;
    if (given(a[4])) {
      out = tensor("out", a[4]);
      need("out", out, dev, dtype_or(a[3], out.scalar_type()), shape);
    }
    const hytopk_elem type = elem(
        "dtype", given(a[4]) ? out.scalar_type() : dtype_or(a[3], at::kBFloat16), BF16 | F32);
    uint32_t* status = status_ptr(a[5], dev);
    const Place place(a[6], dev);
    if (!given(a[4])) out = empty(shape, dtype_or(a[3], at::kBFloat16), dev);
    place.result(out, given(a[4]));
    call("hytopk_cache_read", [&] {
      return p_cache_read(cache.data_ptr(), c.type, c.scale, c.r.n, slots, n, c.r.H, c.r.d,
                          out.data_ptr(), type, status, place.stream());
    });
    return given(a[4]) ? ref(a[4]) : THPVariable_Wrap(std::move(out));
  });
}

// What attend and attend_backward share.
struct Attention {
  const at::Tensor &q, &k, &v;
  at::Device dev;
  Rows rq, rk, rv;
  hytopk_elem type;
  int k_top;
  const int32_t* idx;
  float scale;
};
Attention attention(PyObject* const* a, int allowed, PyObject* scale) {
  const at::Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]);
  const at::Tensor& idx = tensor("idx", a[3]);
  const hytopk_elem type = elem("k", k.scalar_type(), allowed);
  elem("q", q.scalar_type(), BF16);
  if (k.scalar_type() != v.scalar_type() || k.sizes() != v.sizes())
    raise(PyExc_ValueError, "k and v must have one shape and type");
  const at::Device dev = q.device();
  Attention t{q, k, v, dev, packed_rows("q", q), packed_rows("k", k), packed_rows("v", v), type,
              0, nullptr, 0.0f};
  if (t.rk.d != t.rq.d || k.device() != dev || v.device() != dev)
    raise(PyExc_ValueError, "k and v rows must be [", t.rq.d, "] per head on ", dev);
  if (idx.dim() != 2) raise(PyExc_ValueError, "idx must be [n, k]");
  if (idx.size(1) > INT32_MAX) raise(PyExc_ValueError, "idx has an axis of 2^31 or more");
  t.k_top = static_cast<int>(idx.size(1));
  t.idx = static_cast<int32_t*>(need("idx", idx, dev, at::kInt, {t.rq.n, t.k_top}));
  t.scale = static_cast<float>(given(scale) ? number(scale) : std::pow((double)t.rq.d, -0.5));
  return t;
}

// attend(q, k, v, idx, k_scale, v_scale, scale, out_dtype, out, status, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 11, [&]() -> PyObject* {
    const Attention t = attention(a, E4M3 | BF16, a[6]);
    if ((t.type == HYTOPK_ELEM_E4M3) != given(a[4]) || given(a[4]) != given(a[5]))
      raise(PyExc_ValueError,
            "an e4m3 cache needs k_scale and v_scale, a bf16 cache takes none");
    const float *ks = nullptr, *vs = nullptr;
    if (given(a[4])) {
      const auto shape = t.k.sizes().slice(0, t.k.dim() - 1);
      ks = static_cast<float*>(need("k_scale", a[4], t.dev, at::kFloat, shape));
      vs = static_cast<float*>(need("v_scale", a[5], t.dev, at::kFloat, shape));
    }
    const int64_t shape[3] = {t.rq.n, t.rq.H, t.rq.d};
    at::Tensor out;
    if (given(a[8])) {
      out = tensor("out", a[8]);
      need("out", out, t.dev, dtype_or(a[7], out.scalar_type()), shape);
    }
    const at::ScalarType type = given(a[8]) ? out.scalar_type() : dtype_or(a[7], at::kBFloat16);
    const hytopk_elem otype = elem("out_dtype", type, BF16 | F32);
    uint32_t* status = status_ptr(a[9], t.dev);
    const Place place(a[10], t.dev);
    if (!given(a[8])) out = empty(shape, type, t.dev);
    at::Tensor lse = empty({t.rq.n, t.rq.H}, at::kFloat, t.dev);
    place.result(out, given(a[8]));
    place.result(lse);
    call("hytopk_attend", [&] {
      return p_attend(t.q.data_ptr(), t.rq.row, t.k.data_ptr(), t.rk.row, ks, t.v.data_ptr(),
                      t.rv.row, vs, t.idx, t.rq.n, t.rk.n, t.rq.H, t.rk.H, t.rq.d, t.k_top, t.type,
                      t.scale, out.data_ptr(), otype, static_cast<float*>(lse.data_ptr()), status,
                      place.stream());
    });
    PyObject* o = given(a[8]) ? ref(a[8]) : THPVariable_Wrap(std::move(out));
    return Py_BuildValue("(NN)", o, THPVariable_Wrap(std::move(lse)));
  });
}

// attend_backward(q, k, v, idx, out, lse, grad, scale, dk, dv, status, stream)
PyObject* attend_backward(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 12, [&]() -> PyObject* {
    const Attention t = attention(a, BF16, a[7]);
    const int64_t shape[3] = {t.rq.n, t.rq.H, t.rq.d};
    const at::Tensor& out = tensor("out", a[4]);
    const void* grad = need("grad", a[6], t.dev, at::kBFloat16, shape);
    need("out", out, t.dev, out.scalar_type(), shape);
    const void* lse = need("lse", a[5], t.dev, at::kFloat, {t.rq.n, t.rq.H});
    const hytopk_elem otype = elem("out", out.scalar_type(), BF16 | F32);
    const bool add = given(a[8]);
    if (add != given(a[9])) raise(PyExc_ValueError, "dk and dv go together");
    uint32_t* status = status_ptr(a[10], t.dev);
    const Place place(a[11], t.dev);
    at::Tensor dk, dv;
    if (add) {
      need("dk", dk = tensor("dk", a[8]), t.dev, at::kFloat, t.k.sizes());
      need("dv", dv = tensor("dv", a[9]), t.dev, at::kFloat, t.v.sizes());
    } else {
      dk = empty(t.k.sizes(), at::kFloat, t.dev);
      dv = empty(t.v.sizes(), at::kFloat, t.dev);
    }
    place.result(dk, add);
    place.result(dv, add);
    at::Tensor dq = empty(shape, at::kFloat, t.dev);
    place.result(dq);
    call("hytopk_attend_backward", [&] {
      return p_attend_backward(
          t.q.data_ptr(), t.rq.row, t.k.data_ptr(), t.rk.row, t.v.data_ptr(), t.rv.row, t.idx,
          out.data_ptr(), otype, static_cast<const float*>(lse), grad, t.rq.n, t.rk.n, t.rq.H,
          t.rk.H, t.rq.d, t.k_top, t.scale, static_cast<float*>(dq.data_ptr()),
          static_cast<float*>(dk.data_ptr()), static_cast<float*>(dv.data_ptr()), add, status,
          place.stream());
    });
    PyObject* pk = add ? ref(a[8]) : THPVariable_Wrap(std::move(dk));
    PyObject* pv = add ? ref(a[9]) : THPVariable_Wrap(std::move(dv));
    return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(dq)), pk, pv);
  });
}

// ---- the cache in pages ---------------------------------------------------------------

// [N, P, H, d] e4m3 pages with scales [N, H].
struct Pages {
  int N, P, H, d;
  void* codes;
  float* scale;
};
Pages pages_of(const char* name, const at::Tensor& t, const char* scale_name, PyObject* scale) {
  if (t.dim() != 4) raise(PyExc_ValueError, name, " must be [pages, rows, heads, d]");
  if (!t.is_cuda()) raise(PyExc_ValueError, "inputs must be CUDA tensors");
  elem(name, t.scalar_type(), E4M3);
  if (!t.is_contiguous()) raise(PyExc_ValueError, name, " must be contiguous");
  for (const int64_t x : t.sizes())
    if (x > INT32_MAX) raise(PyExc_ValueError, name, " has an axis of 2^31 or more");
  Pages p{(int)t.size(0), (int)t.size(1), (int)t.size(2), (int)t.size(3), t.data_ptr(), nullptr};
  p.scale = static_cast<float*>(need(scale_name, scale, t.device(), at::kFloat, {p.N, p.H}));
  return p;
}

// table [B, columns] of a call
const at::Tensor& table_of(PyObject* o) {
  const at::Tensor& t = tensor("table", o);
  if (t.dim() != 2) raise(PyExc_ValueError, "table must be [sequences, columns]");
  if (!t.is_cuda()) raise(PyExc_ValueError, "inputs must be CUDA tensors");
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
    raise(PyExc_ValueError, "table has an axis of 2^31 or more");
  return t;
}

hytopk_paged paged(PyObject* table, PyObject* lengths, PyObject* cu_q, const Pages& p,
                   at::Device dev) {
  const at::Tensor& t = table_of(table);
  const int64_t B = t.size(0);
  hytopk_paged s{};
  s.table = static_cast<int32_t*>(need("table", t, dev, at::kInt, t.sizes()));
  s.lengths = static_cast<int32_t*>(need("lengths", lengths, dev, at::kInt, {B}));
  if (given(cu_q)) s.cu_q = static_cast<int32_t*>(need("cu_q", cu_q, dev, at::kInt, {B + 1}));
  s.B = static_cast<int>(B);
  s.columns = static_cast<int>(t.size(1));
  s.N = p.N;
  s.P = p.P;
  return s;
}

// page_write(x, pages, page_scale, table, lengths, cu_q, positions, inv_freq, first, interleaved,
//            mscale, status, stream)
PyObject* page_write(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 13, [&]() -> PyObject* {
    const at::Tensor& x = tensor("x", a[0]);
    const Rows r = rows("x", x);
    const at::Device dev = x.device();
    const hytopk_elem type = elem("x", x.scalar_type(), BF16 | F32);
    const at::Tensor& pages = tensor("pages", a[1]);
    const Pages p = pages_of("pages", pages, "page_scale", a[2]);
    if (pages.device() != dev || p.H != r.H || p.d != r.d)
      raise(PyExc_ValueError, "page rows are ", p.H, " x ", p.d, " on ", pages.device(),
            ", expected ", r.H, " x ", r.d, " on ", dev);
    const hytopk_paged s = paged(a[3], a[4], a[5], p, dev);
    hytopk_rope_params params{};
    if (given(a[6]) && !given(a[7])) raise(PyExc_ValueError, "positions need inv_freq");
    if (given(a[7])) {
      const at::Tensor& f = tensor("inv_freq", a[7]);
      if (f.dim() != 1) raise(PyExc_ValueError, "inv_freq must be [rot / 2]");
      if (given(a[6]))
        params.positions = static_cast<int32_t*>(need("positions", a[6], dev, at::kInt, {r.n}));
      params.inv_freq = static_cast<float*>(need("inv_freq", f, dev, at::kFloat, f.sizes()));
      params.rot = static_cast<int>(2 * f.size(0));
      params.first = integer(a[8]);
      params.interleaved = truth(a[9]);
      params.mscale = static_cast<float>(number(a[10]));
    }
    uint32_t* status = status_ptr(a[11], dev);
    const Place place(a[12], dev);
    call("hytopk_page_write", [&] {
      return p_page_write(x.data_ptr(), r.row, r.head, type, (int)r.n, (int)r.H, (int)r.d,
                          given(a[7]) ? &params : nullptr, p.codes, p.scale, &s, status,
                          place.stream());
    });
    return ref(a[1]);
  });
}

// attend_pages(q, k_pages, v_pages, k_scale, v_scale, table, lengths, cu_q, scale, out, lse,
//              status, stream)
PyObject* attend_pages(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 13, [&]() -> PyObject* {
    const at::Tensor& q = tensor("q", a[0]);
    const Rows r = packed_rows("q", q);
    const at::Device dev = q.device();
    elem("q", q.scalar_type(), BF16);
    const at::Tensor &kt = tensor("k_pages", a[1]), &vt = tensor("v_pages", a[2]);
    const Pages k = pages_of("k_pages", kt, "k_scale", a[3]);
    const Pages v = pages_of("v_pages", vt, "v_scale", a[4]);
    if (kt.sizes() != vt.sizes()) raise(PyExc_ValueError, "k_pages and v_pages must have one shape");
    if (k.d != r.d || kt.device() != dev || vt.device() != dev)
      raise(PyExc_ValueError, "k_pages and v_pages rows must be [", r.d, "] per head on ", dev);
    const hytopk_paged s = paged(a[5], a[6], a[7], k, dev);
    const float scale = static_cast<float>(given(a[8]) ? number(a[8]) : std::pow((double)r.d, -0.5));
    const int64_t shape[3] = {r.n, r.H, r.d};
    at::Tensor out, lse;
    if (given(a[9])) need("out", out = tensor("out", a[9]), dev, at::kBFloat16, shape);
    if (given(a[10])) need("lse", lse = tensor("lse", a[10]), dev, at::kFloat, {r.n, r.H});
    uint32_t* status = status_ptr(a[11], dev);
    const Place place(a[12], dev);
    if (!given(a[9])) out = empty(shape, at::kBFloat16, dev);
    if (!given(a[10])) lse = empty({r.n, r.H}, at::kFloat, dev);
    place.result(out, given(a[9]));
    place.result(lse, given(a[10]));
    const size_t bytes = p_attend_pages_workspace_size((int)r.n, (int)r.H, k.H, (int)r.d);
    const at::Tensor workspace = empty({(int64_t)bytes}, at::kByte, dev);
    call("hytopk_attend_pages", [&] {
      return p_attend_pages(q.data_ptr(), r.row, k.codes, k.scale, v.codes, v.scale, &s, (int)r.n,
                            (int)r.H, k.H, (int)r.d, scale, out.data_ptr(),
                            static_cast<float*>(lse.data_ptr()), workspace.data_ptr(), bytes,
                            status, place.stream());
    });
    PyObject* o = given(a[9]) ? ref(a[9]) : THPVariable_Wrap(std::move(out));
    PyObject* l = given(a[10]) ? ref(a[10]) : THPVariable_Wrap(std::move(lse));
    return Py_BuildValue("(NN)", o, l);
  });
}

// The pool's state: table [B, columns], lengths [B], refs [N].
struct Pool {
  at::Device dev;
  int32_t *table, *lengths, *refs;
  int B, columns, N, P;
};
Pool pool_of(PyObject* table, PyObject* lengths, PyObject* refs, PyObject* page) {
  const at::Tensor& t = table_of(table);
  const at::Tensor& r = tensor("refs", refs);
  Pool p{t.device(), nullptr, nullptr, nullptr, (int)t.size(0), (int)t.size(1), 0, integer(page)};
  p.table = static_cast<int32_t*>(need("table", t, p.dev, at::kInt, t.sizes()));
  p.lengths = static_cast<int32_t*>(need("lengths", lengths, p.dev, at::kInt, {p.B}));
  if (r.dim() != 1 || r.size(0) > INT32_MAX)
    raise(PyExc_ValueError, "refs must be [pages], fewer than 2^31");
  p.refs = static_cast<int32_t*>(need("refs", r, p.dev, at::kInt, r.sizes()));
  p.N = (int)r.size(0);
  return p;
}
int32_t* list_of(const char* name, PyObject* o, at::Device dev, int& count) {
  const at::Tensor& t = tensor(name, o);
  if (t.dim() != 1 || t.size(0) > INT32_MAX)
    raise(PyExc_ValueError, name, " must be [count], fewer than 2^31");
  count = (int)t.size(0);
  return static_cast<int32_t*>(need(name, t, dev, at::kInt, t.sizes()));
}

// page_fork(table, lengths, refs, src, dst, page, status, stream)
PyObject* page_fork(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 8, [&]() -> PyObject* {
    const Pool p = pool_of(a[0], a[1], a[2], a[5]);
    int count = 0, other = 0;
    const int32_t* src = list_of("src", a[3], p.dev, count);
    const int32_t* dst = list_of("dst", a[4], p.dev, other);
    if (count != other) raise(PyExc_ValueError, "src and dst must have one length");
    uint32_t* status = status_ptr(a[6], p.dev);
    const Place place(a[7], p.dev);
    call("hytopk_page_fork", [&] {
      return p_page_fork(p.table, p.lengths, p.refs, p.B, p.columns, p.N, p.P, src, dst, count,
                         status, place.stream());
    });
    return ref(a[0]);
  });
}

// page_free(table, lengths, refs, rows, page, status, stream)
PyObject* page_free(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 7, [&]() -> PyObject* {
    const Pool p = pool_of(a[0], a[1], a[2], a[4]);
    int count = 0;
    const int32_t* rows = list_of("sequences", a[3], p.dev, count);
    uint32_t* status = status_ptr(a[5], p.dev);
    const Place place(a[6], p.dev);
    call("hytopk_page_free", [&] {
      return p_page_free(p.table, p.lengths, p.refs, p.B, p.columns, p.N, p.P, rows, count, status,
                         place.stream());
    });
    return ref(a[0]);
  });
}

// The lists of copies that page_grow and page_compact make. (Two tensors: views of one take
// 2 us of a call more each.)
struct Lists {
  at::Tensor src, dst;
  Lists(int64_t count, at::Device dev, const Place& place)
      : src(empty({count}, at::kInt, dev)), dst(empty({count}, at::kInt, dev)) {
    place.result(src);
    place.result(dst);
  }
  static int32_t* at(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
  PyObject* give() {
    PyObject* s = THPVariable_Wrap(std::move(src));
    PyObject* d = THPVariable_Wrap(std::move(dst));
    return Py_BuildValue("(NN)", s, d);
  }
};

// page_grow(table, lengths, refs, add, page, status, stream)
PyObject* page_grow(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 7, [&]() -> PyObject* {
    const Pool p = pool_of(a[0], a[1], a[2], a[4]);
    const void* add = need("add", a[3], p.dev, at::kInt, {p.B});
    uint32_t* status = status_ptr(a[5], p.dev);
    const Place place(a[6], p.dev);
    Lists lists(p.B, p.dev, place);
    const size_t bytes = p_page_workspace_size(p.N);
    const at::Tensor workspace = empty({(int64_t)bytes}, at::kByte, p.dev);
    call("hytopk_page_grow", [&] {
      return p_page_grow(p.table, p.lengths, p.refs, p.B, p.columns, p.N, p.P,
                         static_cast<const int32_t*>(add), Lists::at(lists.src), Lists::at(lists.dst),
                         workspace.data_ptr(), bytes, status, place.stream());
    });
    return lists.give();
  });
}

// page_compact(table, lengths, refs, page, status, stream)
PyObject* page_compact(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 6, [&]() -> PyObject* {
    const Pool p = pool_of(a[0], a[1], a[2], a[3]);
    uint32_t* status = status_ptr(a[4], p.dev);
    const Place place(a[5], p.dev);
    Lists lists(p.N > 3 ? p.N / 2 : 1, p.dev, place);
    const size_t bytes = p_page_workspace_size(p.N);
    const at::Tensor workspace = empty({(int64_t)bytes}, at::kByte, p.dev);
    call("hytopk_page_compact", [&] {
      return p_page_compact(p.table, p.lengths, p.refs, p.B, p.columns, p.N, p.P,
                            Lists::at(lists.src), Lists::at(lists.dst), workspace.data_ptr(), bytes,
                            status, place.stream());
    });
    return lists.give();
  });
}

// page_copy(k_pages, v_pages, k_scale, v_scale, src, dst, status, stream)
PyObject* page_copy(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 8, [&]() -> PyObject* {
    const at::Tensor& kt = tensor("k_pages", a[0]);
    const Pages k = pages_of("k_pages", kt, "k_scale", a[2]);
    const at::Device dev = kt.device();
    Pages v{};
    if (given(a[1]) != given(a[3])) raise(PyExc_ValueError, "v_pages and v_scale go together");
    if (given(a[1])) {
      const at::Tensor& vt = tensor("v_pages", a[1]);
      v = pages_of("v_pages", vt, "v_scale", a[3]);
      if (vt.sizes() != kt.sizes() || vt.device() != dev)
        raise(PyExc_ValueError, "k_pages and v_pages must have one shape and device");
    }
    int count = 0, other = 0;
    const int32_t* src = list_of("src", a[4], dev, count);
    const int32_t* dst = list_of("dst", a[5], dev, other);
    if (count != other) raise(PyExc_ValueError, "src and dst must have one length");
    uint32_t* status = status_ptr(a[6], dev);
    const Place place(a[7], dev);
    call("hytopk_page_copy", [&] {
      return p_page_copy(k.codes, k.scale, v.codes, v.scale, k.N, (int64_t)k.P * k.H * k.d, k.H,
                         src, dst, count, status, place.stream());
    });
    return ref(Py_None);
  });
}

// init_pages(addresses of the C entry points of the cache in pages)
PyObject* init_pages(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 9, [&]() -> PyObject* {
    void* p[9];
    for (int i = 0; i < 9; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (PyErr_Occurred()) throw Raised{};
    }
    p_attend_pages_workspace_size = reinterpret_cast<decltype(p_attend_pages_workspace_size)>(p[0]);
    p_attend_pages = reinterpret_cast<decltype(p_attend_pages)>(p[1]);
    p_page_write = reinterpret_cast<decltype(p_page_write)>(p[2]);
    p_page_workspace_size = reinterpret_cast<decltype(p_page_workspace_size)>(p[3]);
    p_page_fork = reinterpret_cast<decltype(p_page_fork)>(p[4]);
    p_page_free = reinterpret_cast<decltype(p_page_free)>(p[5]);
    p_page_grow = reinterpret_cast<decltype(p_page_grow)>(p[6]);
    p_page_compact = reinterpret_cast<decltype(p_page_compact)>(p[7]);
    p_page_copy = reinterpret_cast<decltype(p_page_copy)>(p[8]);
    return ref(Py_None);
  });
}

// init(error class, torch's out-of-memory class, addresses of the five C entry points)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded(na, 7, [&]() -> PyObject* {
    void* p[5];
    for (int i = 0; i < 5; ++i) {
      p[i] = PyLong_AsVoidPtr(a[2 + i]);
      if (PyErr_Occurred()) throw Raised{};
    }
    p_rope = reinterpret_cast<decltype(p_rope)>(p[0]);
    p_cache_write = reinterpret_cast<decltype(p_cache_write)>(p[1]);
    p_cache_read = reinterpret_cast<decltype(p_cache_read)>(p[2]);
    p_attend = reinterpret_cast<decltype(p_attend)>(p[3]);
    p_attend_backward = reinterpret_cast<decltype(p_attend_backward)>(p[4]);
    Py_XDECREF(status_error);
    Py_XDECREF(memory_error);
    status_error = ref(a[0]);
    memory_error = ref(a[1]);
    return ref(Py_None);
  });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(init),   METHOD(rope),   METHOD(cache_write),
                         METHOD(cache_read), METHOD(attend), METHOD(attend_backward),
                         METHOD(init_pages), METHOD(page_write), METHOD(attend_pages),
                         METHOD(page_fork), METHOD(page_free), METHOD(page_grow),
                         METHOD(page_compact), METHOD(page_copy),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operators", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators() { return PyModule_Create(&module); }
