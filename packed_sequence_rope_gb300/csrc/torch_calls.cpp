// The per-step calls of the serving operators for Python: argument checks,
// output allocation and the C call, in one native step.
//
// A decoding step's kernels take 3 to 7 us. Marshalled in Python, a call cost 15 to
// 21 us of host time (three for each small allocation, the rest attribute
// tests and ctypes), so that the host set the pace; here it costs about half.
// Nothing is computed: the operators are libanchorattn.so's, whose C ABI these
// functions call. A status other than 0 comes back as an int, which the Python
// side turns into AAError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <optional>
#include <string>
#include <utility>

#include "../../include/anchorattn.h"

namespace {

using at::Tensor;

// How messages name a shape; -1: any size.
std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + (s[i] < 0 ? std::string("any") : std::to_string(s[i]));
  return t + ")";
}

const Tensor* given(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return &THPVariable_Unpack(o);
}

const Tensor& need(PyObject* o, const char* name) {
  const Tensor* t = given(o, name);
  TORCH_CHECK_VALUE(t, name, " must be a tensor");
  return *t;
}

void check_kind(const Tensor& t, const char* name, at::ScalarType type, at::Device dev) {
  TORCH_CHECK_VALUE(t.layout() == at::kStrided && t.scalar_type() == type && t.device() == dev, name, " must be a ",
                    c10::toString(type), " tensor on ", dev);
}

// [T, H, D] bf16 (T, H -1: any)
void check_rows(const Tensor& t, const char* name, int64_t T, int64_t H, int64_t D, at::Device dev) {
  check_kind(t, name, at::kBFloat16, dev);
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(2) == D && (T < 0 || t.size(0) == T) && (H < 0 || t.size(1) == H), name,
                    " must have shape ", shape_text({T, H, D}), ", got ", shape_text(t.sizes()));
}

void check_exact(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  check_kind(t, name, type, dev);
  TORCH_CHECK_VALUE(t.sizes() == shape && t.is_contiguous(), name, " must be contiguous with shape ", shape_text(shape),
                    ", got ", shape_text(t.sizes()));
}

// A [T, H, D] input as the kernels read it: a token's heads contiguous, rows
// 16-byte aligned; copied if it is not.
struct Rows {
  Tensor copy;
  const void* ptr;
  int64_t stride;
  explicit Rows(const Tensor& x) {
    const int64_t T = x.size(0), H = x.size(1), D = x.size(2), token = H * D;
    auto aligned = [](const Tensor& t) { return (reinterpret_cast<uintptr_t>(t.const_data_ptr()) & 15u) == 0; };
    ptr = x.const_data_ptr();
    stride = token;
    if (x.stride(2) == 1 && (x.stride(1) == D || H == 1) && aligned(x)) {
      if (T <= 1) return;
      if (x.stride(0) >= token && x.stride(0) % 8 == 0) {
        stride = x.stride(0);
        return;
      }
    }
    copy = x.contiguous();
    if (!aligned(copy)) copy = copy.clone();
    ptr = copy.const_data_ptr();
  }
};

Tensor make(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// A given result tensor is checked here; written() tells autograd of it once it is.
Tensor out_or_new(const Tensor* out, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  if (!out) return make(shape, type, dev);
  check_exact(*out, name, shape, type, dev);
  TORCH_CHECK_VALUE(!(out->requires_grad() && at::GradMode::is_enabled()), name,
                    " requires grad: the result written into it would carry none");
  return *out;
}
void written(const Tensor* out) {
  if (out && !out->is_inference()) out->unsafeGetTensorImpl()->bump_version();
}

int64_t as_int(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t as_i32(PyObject* o, const char* name) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw python_error();
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i, &overflow);
  Py_DECREF(i);
  TORCH_CHECK_VALUE(!overflow && v >= INT32_MIN && v <= INT32_MAX, name, " must be a 32-bit integer");
  return (int32_t)v;
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
template <class T>
T as_handle(PyObject* o) {
  return reinterpret_cast<T>(static_cast<uintptr_t>(as_int(o)));
}

// The stream of a call (None: the current one of the device); new tensors are
// allocated on it.
struct OnStream {
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  aa_stream_t s;
  OnStream(PyObject* o, at::Device dev) {
    if (o == Py_None) {
      s = reinterpret_cast<aa_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
      return;
    }
    PyObject* p = PyObject_GetAttrString(o, "cuda_stream");
    if (!p) throw python_error();
    const auto raw = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(p));
    Py_DECREF(p);
    if (PyErr_Occurred()) throw python_error();
    s = reinterpret_cast<aa_stream_t>(raw);
    guard.emplace(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(raw), dev.index()));
  }
};

const int32_t* positions(const Tensor& pos, int64_t axes, int64_t T, at::Device dev, Tensor* keep) {
  check_kind(pos, "pos", at::kInt, dev);
  const bool fits = (pos.dim() == 2 && pos.size(0) == axes && pos.size(1) == T) || (axes == 1 && pos.dim() == 1 && pos.size(0) == T);
  TORCH_CHECK_VALUE(fits, "pos must have shape ", shape_text({axes, T}), ", got ", shape_text(pos.sizes()));
  *keep = pos.contiguous();
  return keep->const_data_ptr<int32_t>();
}

aa_cache_batch batch_of(PyObject* table, PyObject* cu, PyObject* kv, int64_t T, int32_t layer, at::Device dev) {
  const Tensor &t = need(table, "page_table"), &c = need(cu, "cu_q"), &k = need(kv, "kv_len");
  for (auto [x, name] : {std::pair(&t, "page_table"), std::pair(&c, "cu_q"), std::pair(&k, "kv_len")}) {
    check_kind(*x, name, at::kInt, dev);
    TORCH_CHECK_VALUE(x->is_contiguous(), name, " must be contiguous");
  }
  TORCH_CHECK_VALUE(t.dim() == 2 && c.dim() == 1 && k.dim() == 1 && c.size(0) == t.size(0) + 1 && k.size(0) == t.size(0),
                    "page_table [B, W], cu_q [B + 1] and kv_len [B] do not fit together: ", shape_text(t.sizes()), ", ",
                    shape_text(c.sizes()), ", ", shape_text(k.sizes()));
  TORCH_CHECK_VALUE(t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX && T <= INT32_MAX, "the batch is too large");
  aa_cache_batch b;
  b.page_table = t.const_data_ptr<int32_t>();
  b.cu_q = c.const_data_ptr<int32_t>();
  b.kv_len = k.const_data_ptr<int32_t>();
  b.num_seqs = (int32_t)t.size(0);
  b.table_width = (int32_t)t.size(1);
  b.total_tokens = (int32_t)T;
  b.layer = layer;
  return b;
}

template <class Fn>
int without_gil(Fn fn) {
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = fn();
  Py_END_ALLOW_THREADS;
  return status;
}

void check_count(const char* name, Py_ssize_t got, Py_ssize_t want) {
  TORCH_CHECK_TYPE(got == want, name, " takes ", want, " arguments, got ", got);
}

// ---------------------------------------------------------------- rotation
struct Rotated {
  int status;
  Tensor q, k;
};

Rotated rotate(const aa_rope_axes* rope, const Tensor& pos, const Tensor& q, const Tensor* k, bool inverse,
               const Tensor* out_q, const Tensor* out_k, PyObject* stream) {
  TORCH_CHECK_VALUE(q.is_cuda(), "q must be a CUDA tensor");
  const at::Device dev = q.device();
  check_rows(q, "q", -1, -1, rope->head_dim, dev);
  TORCH_CHECK_VALUE(dev.index() == c10::cuda::current_device(), "q is on ", dev, ", which is not the current device");
  const int64_t T = q.size(0);
  TORCH_CHECK_VALUE(k || !out_k, "out_k goes with k");
  if (k) check_rows(*k, "k", T, -1, rope->head_dim, dev);
  TORCH_CHECK_VALUE(T <= INT32_MAX && q.size(1) <= INT32_MAX && (!k || k->size(1) <= INT32_MAX), "q or k is too large");
  const OnStream on(stream, dev);
  Tensor keep;
  Rotated r;
  const int32_t* p = positions(pos, rope->num_axes, T, dev, &keep);
  r.q = out_or_new(out_q, "out_q", q.sizes(), at::kBFloat16, dev);
  const Rows rq(q);
  std::optional<Rows> rk;
  if (k) {
    r.k = out_or_new(out_k, "out_k", k->sizes(), at::kBFloat16, dev);
    rk.emplace(*k);
  }
  r.status = aa_rope_axes_apply(rope, p, (int32_t)T, rq.ptr, rq.stride, r.q.mutable_data_ptr(), (int32_t)q.size(1),
                                k ? rk->ptr : nullptr, k ? rk->stride : 0, k ? r.k.mutable_data_ptr() : nullptr,
                                k ? (int32_t)k->size(1) : 0, inverse, on.s);
  return r;
}

PyObject* wrap(Tensor q, Tensor k) {
  PyObject* pq = THPVariable_Wrap(std::move(q));
  if (!k.defined()) return pq;
  PyObject* pk = THPVariable_Wrap(std::move(k));
  PyObject* r = PyTuple_Pack(2, pq, pk);
  Py_XDECREF(pq);
  Py_XDECREF(pk);
  return r;
}

// rope_apply(rope, pos, q, k, inverse, out_q, out_k, stream)
PyObject* rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count("rope_apply", n, 8);
  Rotated r = rotate(as_handle<const aa_rope_axes*>(a[0]), need(a[1], "pos"), need(a[2], "q"), given(a[3], "k"), as_bool(a[4]),
                     given(a[5], "out_q"), given(a[6], "out_k"), a[7]);
  if (r.status) return PyLong_FromLong(r.status);
  written(given(a[5], "out_q"));
  written(given(a[6], "out_k"));
  return wrap(std::move(r.q), std::move(r.k));
  END_HANDLE_TH_ERRORS
}

// The rotation is orthogonal: its gradient is the rotation back, and so on.
struct RopeHold : torch::CustomClassHolder {
  aa_rope_axes rope;
  explicit RopeHold(const aa_rope_axes& r) : rope(r) {}
};
using RopePtr = c10::intrusive_ptr<RopeHold>;

struct RopeFn : torch::autograd::Function<RopeFn> {
  using List = torch::autograd::variable_list;
  static List turn(const RopePtr& rope, bool inverse, const Tensor& pos, const Tensor& q, const std::optional<Tensor>& k) {
    Rotated r = rotate(&rope->rope, pos, q, k ? &*k : nullptr, inverse, nullptr, nullptr, Py_None);
    TORCH_CHECK(r.status == 0, aa_status_string((aa_status)r.status), ": ", aa_last_error());
    return r.k.defined() ? List{r.q, r.k} : List{r.q};
  }
  static List forward(torch::autograd::AutogradContext* ctx, RopePtr rope, bool inverse, Tensor pos, Tensor q,
                      std::optional<Tensor> k) {
    ctx->save_for_backward({pos});
    ctx->saved_data["rope"] = c10::IValue::make_capsule(rope);
    ctx->saved_data["inverse"] = inverse;
    return turn(rope, inverse, pos, q, k);
  }
  static List backward(torch::autograd::AutogradContext* ctx, List g) {
    const Tensor pos = ctx->get_saved_variables()[0];
    const RopePtr rope = c10::static_intrusive_pointer_cast<RopeHold>(ctx->saved_data["rope"].toCapsule());
    const bool inverse = !ctx->saved_data["inverse"].toBool();
    // edges: pos, q, k
    const bool need_q = ctx->needs_input_grad(1), need_k = g.size() > 1 && ctx->needs_input_grad(2);
    auto both = [&](const Tensor& q, const std::optional<Tensor>& k) {
      return at::GradMode::is_enabled() ? apply(rope, inverse, pos, q, k) : turn(rope, inverse, pos, q, k);
    };
    Tensor gq, gk;
    if (need_q) {
      List r = both(g[0], need_k ? std::optional<Tensor>(g[1]) : std::nullopt);
      gq = r[0];
      if (need_k) gk = r[1];
    } else if (need_k) {
      gk = both(g[1], std::nullopt)[0];
    }
    return {Tensor(), Tensor(), Tensor(), gq, gk};
  }
};

// rope_autograd(rope, pos, q, k)
PyObject* rope_autograd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count("rope_autograd", n, 4);
  const Tensor& q = need(a[2], "q");
  const Tensor* k = given(a[3], "k");
  const auto rope = c10::make_intrusive<RopeHold>(*as_handle<const aa_rope_axes*>(a[0]));
  RopeFn::List r = RopeFn::apply(rope, false, need(a[1], "pos"), q, k ? std::optional<Tensor>(*k) : std::nullopt);
  return wrap(r[0], r.size() > 1 ? r[1] : Tensor());
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- cache
// cache_append(cache, device, Hkv, head_dim, k, v, table, cu_q, kv_len, layer, rope, axes, pos, q, out_q, stream)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count("cache_append", n, 16);
  const auto cache = as_handle<aa_cache_t>(a[0]);
  const at::Device dev(at::kCUDA, (c10::DeviceIndex)as_int(a[1]));
  const int64_t H = as_int(a[2]), D = as_int(a[3]);
  const Tensor &k = need(a[4], "k"), &v = need(a[5], "v");
  check_rows(k, "k", -1, H, D, dev);
  const int64_t T = k.size(0);
  check_rows(v, "v", T, H, D, dev);
  const aa_cache_batch batch = batch_of(a[6], a[7], a[8], T, as_i32(a[9], "layer"), dev);
  const auto* rope = a[10] == Py_None ? nullptr : as_handle<const aa_rope_axes*>(a[10]);
  const Tensor *pos = given(a[12], "pos"), *q = given(a[13], "q"), *out_q = given(a[14], "out_q");
  TORCH_CHECK_VALUE((rope != nullptr) == (pos != nullptr), "give both rope and pos or neither");
  TORCH_CHECK_VALUE(q || !out_q, "out_q goes with q");
  if (q) {
    check_rows(*q, "q", T, -1, D, dev);
    TORCH_CHECK_VALUE(rope, "q is rotated: it needs rope and pos");
    TORCH_CHECK_VALUE(q->size(1) <= INT32_MAX, "q is too large");
  }
  const OnStream on(a[15], dev);
  Tensor keep, yq;
  const int32_t* pp = pos ? positions(*pos, as_int(a[11]), T, dev, &keep) : nullptr;
  const Rows rk(k), rv(v);
  std::optional<Rows> rq;
  if (q) {
    yq = out_or_new(out_q, "out_q", q->sizes(), at::kBFloat16, dev);
    rq.emplace(*q);
  }
  const int status = without_gil([&] {
    return aa_cache_append(cache, &batch, rk.ptr, rk.stride, rv.ptr, rv.stride, rope, pp, q ? rq->ptr : nullptr,
                           q ? rq->stride : 0, q ? yq.mutable_data_ptr() : nullptr, q ? (int32_t)q->size(1) : 0, on.s);
  });
  if (status) return PyLong_FromLong(status);
  written(out_q);
  if (q) return THPVariable_Wrap(std::move(yq));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// cache_attend(cache, device, head_dim, q, table, cu_q, kv_len, max_q, layer, key_lo, anchor, scale, out, lse,
//              workspace, return_lse, stream)
PyObject* cache_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count("cache_attend", n, 17);
  const auto cache = as_handle<aa_cache_t>(a[0]);
  const at::Device dev(at::kCUDA, (c10::DeviceIndex)as_int(a[1]));
  const int64_t D = as_int(a[2]);
  const Tensor& q = need(a[3], "q");
  check_rows(q, "q", -1, -1, D, dev);
  const int64_t T = q.size(0), H = q.size(1);
  TORCH_CHECK_VALUE(H <= INT32_MAX, "q is too large");
  const int32_t max_q = as_i32(a[7], "max_q");
  const aa_cache_batch batch = batch_of(a[4], a[5], a[6], T, as_i32(a[8], "layer"), dev);
  const Tensor *key_lo = given(a[9], "key_lo"), *out = given(a[12], "out"), *lse_in = given(a[13], "lse"),
               *work_in = given(a[14], "workspace");
  const double scale = PyFloat_AsDouble(a[11]);
  if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  const bool anchor = as_bool(a[10]), return_lse = as_bool(a[15]);
  if (key_lo) {
    check_kind(*key_lo, "key_lo", at::kInt, dev);
    TORCH_CHECK_VALUE(key_lo->dim() == 1 && key_lo->size(0) == T, "key_lo must have shape ", shape_text({T}));
  }
  const OnStream on(a[16], dev);
  Tensor lo, lse, work;
  if (key_lo) lo = key_lo->contiguous();
  Tensor o = out_or_new(out, "out", q.sizes(), at::kBFloat16, dev);
  if (lse_in || return_lse) lse = out_or_new(lse_in, "lse", {H, T}, at::kFloat, dev);
  if (work_in) {
    check_kind(*work_in, "workspace", at::kByte, dev);
    TORCH_CHECK_VALUE(work_in->is_contiguous(), "workspace must be contiguous");
    work = *work_in;
  } else {
    const size_t bytes = aa_cache_attend_workspace_bytes(cache, batch.num_seqs, (int32_t)T, max_q, batch.table_width, (int32_t)H);
    work = make({(int64_t)std::max<size_t>(bytes, 256)}, at::kByte, dev);
  }
  const Rows rq(q);
  const int status = without_gil([&] {
    return aa_cache_attend(cache, &batch, rq.ptr, rq.stride, (int32_t)H, max_q, key_lo ? lo.const_data_ptr<int32_t>() : nullptr,
                           anchor, (float)scale, o.mutable_data_ptr(),
                           lse.defined() ? static_cast<float*>(lse.mutable_data_ptr()) : nullptr, work.mutable_data_ptr(),
                           (size_t)work.numel(), on.s);
  });
  if (status) return PyLong_FromLong(status);
  written(out);
  written(lse_in);
  return wrap(std::move(o), return_lse ? std::move(lse) : Tensor());
  END_HANDLE_TH_ERRORS
}

// Page numbers: a buffer of contiguous 32-bit integers (an int32 array).
struct HostInts {
  Py_buffer b;
  HostInts(PyObject* o, const char* name) {
    if (PyObject_GetBuffer(o, &b, PyBUF_FORMAT | PyBUF_C_CONTIGUOUS)) throw python_error();
    const bool fits = b.ndim == 1 && b.itemsize == 4 && b.format && (b.format[0] == 'i' || b.format[0] == 'l') && !b.format[1];
    if (!fits) PyBuffer_Release(&b);
    TORCH_CHECK_VALUE(fits, name, " must be an int32 array");
  }
  ~HostInts() { PyBuffer_Release(&b); }
  HostInts(const HostInts&) = delete;
  const int32_t* data() const { return static_cast<const int32_t*>(b.buf); }
  Py_ssize_t size() const { return b.len / 4; }
};

// cache_copy_pages(cache, device, src, dst, stream)
PyObject* cache_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count("cache_copy_pages", n, 5);
  const auto cache = as_handle<aa_cache_t>(a[0]);
  const int64_t dev = as_int(a[1]);  // -1: no device, which the library refuses
  const HostInts src(a[2], "src"), dst(a[3], "dst");
  TORCH_CHECK_VALUE(src.size() == dst.size(), "src and dst must have the same number of entries");
  TORCH_CHECK_VALUE(src.size() <= INT32_MAX, "src and dst are too long");
  std::optional<OnStream> on;
  if (dev >= 0) on.emplace(a[4], at::Device(at::kCUDA, (c10::DeviceIndex)dev));
  const aa_stream_t s = on ? on->s : nullptr;
  return PyLong_FromLong(without_gil([&] { return aa_cache_copy_pages(cache, src.data(), dst.data(), (int32_t)src.size(), s); }));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rope_apply", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_apply)), METH_FASTCALL, nullptr},
    {"rope_autograd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_autograd)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_append)), METH_FASTCALL, nullptr},
    {"cache_attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_attend)), METH_FASTCALL, nullptr},
    {"cache_copy_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_copy_pages)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
