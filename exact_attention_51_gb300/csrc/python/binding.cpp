// Torch binding of the calls that a decoding step makes once a layer: rotary
// positions, the paged append and paged attention.
//
// Such a step's kernels run for a few microseconds, less than a binding written
// in Python takes to look its tensors over (measured on the GB300's host, per call:
// attn_fwd_fp8_paged 37 us through ctypes, 8 here).  The checks, the
// defaults and the errors are those of the Python wrappers that call this module;
// everything else is behind the C ABI of include/.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/CUDAContextLight.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <string>

#include "attn_paged.h"
#include "attn_rope.h"

namespace {

PyObject* g_attn_error = nullptr;  // the package's AttnError

// A Python error to raise.
struct Refused {
  PyObject* type;
  std::string what;
};

[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }

void check(bool ok, const char* what) {
  if (!ok) value_error(what);
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

const at::Tensor& must_be_tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o);
  if (!t) value_error(std::string(name) + " must be a tensor");
  return *t;
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

int integer32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// The stream of a call: the given one, or torch's current one on the device.
//
// What the call allocates is of the call's stream: torch's allocator hands out a freed block again
// in the order of the stream that it is of, so that on any other one the kernels before could still
// be using it.
struct Stream {
  void* handle;
  c10::cuda::CUDAStream current;  // the caller's
  std::optional<c10::cuda::CUDAStream> given;

  Stream(PyObject* o, c10::DeviceIndex device) : current(c10::cuda::getCurrentCUDAStream(device)) {
    if (o == Py_None) {
      handle = current.stream();
      return;
    }
    unsigned long long bits;
    if (PyLong_Check(o)) {
      bits = PyLong_AsUnsignedLongLong(o);
    } else {
      PyObject* attr = PyObject_GetAttrString(o, "cuda_stream");
      if (!attr) throw python_error();
      bits = PyLong_AsUnsignedLongLong(attr);
      Py_DECREF(attr);
    }
    if (bits == static_cast<unsigned long long>(-1) && PyErr_Occurred()) throw python_error();
    handle = reinterpret_cast<void*>(bits);
    given = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), device);
  }

  // make() with the call's stream as torch's current one.
  template <typename F>
  at::Tensor alloc(F&& make) const {
    if (!given) return make();
    const c10::cuda::CUDAStreamGuard on(*given);
    return make();
  }

  // Tells torch's allocator that the caller, who gets `t`, uses it on a stream of its own.
  void returns(const at::Tensor& t) const {
    if (given && *given != current) t.record_stream(current.unwrap());
  }
};

void int32_of(const char* name, const at::Tensor& t, at::IntArrayRef shape, const at::Device& device) {
  if (t.scalar_type() != at::kInt || !t.is_contiguous() || t.device() != device || t.sizes() != shape) {
    std::string s = std::string(name) + " must be a contiguous int32 tensor [";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    value_error(s + "] on the inputs' device");
  }
}

const uint64_t* phases_of(const at::Tensor& t, int64_t d, const at::Device& device) {
  check(t.scalar_type() == at::kLong && t.dim() == 1 && t.is_contiguous() && t.device() == device,
        "phases must be a contiguous int64 tensor [rot_dim / 2] on the inputs' device");
  check(t.numel() >= 1 && t.numel() <= d / 2, "phases must have rot_dim / 2 entries, 1 to d / 2");
  return static_cast<const uint64_t*>(t.data_ptr());
}

// New tensors by torch's CUDA allocator, past the dispatcher (a third of a call's host time goes into them).
at::Tensor new_tensor(at::IntArrayRef sizes, at::ScalarType type, const at::Device& device) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, device, std::nullopt));
}
// As empty_like: x's strides where its elements fill their extent, else contiguous.
at::Tensor new_like(const at::Tensor& x) {
  if (x.is_non_overlapping_and_dense())
    return at::Tensor(at::detail::empty_strided_cuda(x.sizes(), x.strides(), x.scalar_type(), x.device()));
  return new_tensor(x.sizes(), x.scalar_type(), x.device());
}

// Counts a write into a tensor of the caller's, as torch's in-place operations do: autograd then
// refuses a value that it saved and that has changed since.  (Inference tensors have no count, and
// autograd saves none.)
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

int dim32(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(n);
}

PyObject* status_error(int rc, const char* what) {
  if (!g_attn_error) {
    PyErr_Format(PyExc_RuntimeError, "%s: status %d", what, rc);
    return nullptr;
  }
  PyObject* e = PyObject_CallFunction(g_attn_error, "is", rc, what);
  if (e) {
    PyErr_SetObject(g_attn_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// Runs a call's body, turning C++ exceptions into Python errors.
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return body();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (python_error& e) {
    e.restore();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());  // torch's own error types
  }
  return nullptr;
}

// rope(backward, x, phases, positions, position0, interleaved, attention_factor, out, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) type_error("rope takes 9 arguments");
    const bool backward = truth(a[0]);
    const at::Tensor* xp = tensor(a[1]);
    if (!xp || !xp->is_cuda()) type_error("x must be a CUDA bfloat16, float16 or float32 tensor");
    const at::Tensor& x = *xp;
    const at::ScalarType type = x.scalar_type();
    int dtype = 0;
    if (type == at::kBFloat16) dtype = ATTN_ROPE_BF16;
    else if (type == at::kHalf) dtype = ATTN_ROPE_F16;
    else if (type == at::kFloat) dtype = ATTN_ROPE_F32;
    else type_error("x must be a CUDA bfloat16, float16 or float32 tensor");
    check(x.dim() == 4 && (x.stride(3) == 1 || x.size(3) == 1), "x must be [B, H, N, d] with the elements of a head adjacent");
    const at::Device device = x.device();
    const int B = dim32(x.size(0), "B"), H = dim32(x.size(1), "H"), N = dim32(x.size(2), "N"), d = dim32(x.size(3), "d");
    const at::Tensor& phases = must_be_tensor(a[2], "phases");
    const uint64_t* u = phases_of(phases, d, device);
    const int32_t* pos = nullptr;
    int64_t stride_b = 0;
    if (a[3] != Py_None) {
      const at::Tensor& t = must_be_tensor(a[3], "positions");
      if (t.dim() == 2) {
        int32_of("positions", t, {B, N}, device);
        stride_b = N;
      } else {
        int32_of("positions", t, {N}, device);
      }
      pos = static_cast<const int32_t*>(t.data_ptr());
    }
    const int position0 = integer32(a[4], "position0");
    const bool interleaved = truth(a[5]);
    const float factor = static_cast<float>(number(a[6]));
    const c10::cuda::OptionalCUDAGuard guard(device);
    const Stream stream(a[8], device.index());
    at::Tensor y;
    const bool made = a[7] == Py_None;
    if (made) {
      y = stream.alloc([&] { return new_like(x); });
    } else {
      y = must_be_tensor(a[7], "out");
      check(y.sizes() == x.sizes() && y.scalar_type() == type && y.device() == device && (y.stride(3) == 1 || d == 1),
            "out must be shaped and typed like x on its device, with the elements of a head adjacent");
    }
    if (x.numel() > 0) {
      const auto xs = x.strides(), ys = y.strides();
      const int rc = (backward ? attn_rope_bwd : attn_rope)(
          x.data_ptr(), y.data_ptr(), dtype, B, H, N, d, xs[0], xs[1], xs[2], ys[0], ys[1], ys[2], pos, stride_b, position0, u,
          2 * static_cast<int>(phases.numel()), interleaved, factor, stream.handle);
      if (rc != ATTN_OK) return status_error(rc, backward ? "attn_rope_bwd" : "attn_rope");
      if (made) stream.returns(y);
      else written(y);
    }
    return THPVariable_Wrap(std::move(y));
  });
}

bool is_codes(const at::Tensor& t) {
  return t.is_cuda() && (t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte);
}

struct Cache {
  const at::Tensor *k, *v, *ks, *vs;
  int pages, heads, page_size, d;

  explicit Cache(PyObject* const* a) {
    k = tensor(a[0]), v = tensor(a[1]);
    if (!k || !is_codes(*k)) type_error("k_cache must be a CUDA float8_e4m3fn (or uint8) tensor");
    if (!v || !is_codes(*v)) type_error("v_cache must be a CUDA float8_e4m3fn (or uint8) tensor");
    check(k->dim() == 4 && k->is_contiguous(), "k_cache must be contiguous [num_pages, Hkv, page_size, d]");
    check(v->dim() == 4 && v->is_contiguous(), "v_cache must be contiguous [num_pages, Hkv, page_size, d]");
    check(k->sizes() == v->sizes() && k->device() == v->device(), "k_cache and v_cache must have one shape and device");
    ks = &must_be_tensor(a[2], "k_scale"), vs = &must_be_tensor(a[3], "v_scale");
    for (const at::Tensor* s : {ks, vs})
      check(s->scalar_type() == at::kFloat && s->dim() == 2 && s->size(0) == k->size(0) && s->size(1) == k->size(1) &&
                s->is_contiguous() && s->device() == k->device(),
            "k_scale and v_scale must be contiguous fp32 [num_pages, Hkv] tensors on the cache's device");
    pages = dim32(k->size(0), "num_pages"), heads = dim32(k->size(1), "Hkv");
    page_size = dim32(k->size(2), "page_size"), d = dim32(k->size(3), "d");
  }
};

const at::Tensor& bf16_rows(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda() || t->scalar_type() != at::kBFloat16) type_error(std::string(name) + " must be a CUDA bfloat16 tensor");
  if (t->dim() != 3 || (t->stride(2) != 1 && t->size(2) != 1))
    value_error(std::string(name) + " must be [T, heads, d] with the elements of a head adjacent");
  return *t;
}

// append(k, v, slots, k_cache, v_cache, k_scale, v_scale, phases, positions, interleaved,
// attention_factor, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) type_error("append takes 12 arguments");
    const at::Tensor &k = bf16_rows(a[0], "k"), &v = bf16_rows(a[1], "v");
    const Cache c(a + 3);
    const at::Device device = k.device();
    check(v.sizes() == k.sizes() && k.size(1) == c.heads && k.size(2) == c.d, "k, v must be [T, Hkv, d] with the cache's Hkv and d");
    check(v.device() == device && c.k->device() == device, "k, v and the cache must be on one device");
    const int T = dim32(k.size(0), "T");
    const at::Tensor& slots = must_be_tensor(a[2], "slots");
    int32_of("slots", slots, {T}, device);
    const uint64_t* u = nullptr;
    const int32_t* pos = nullptr;
    int rot = 0;
    if (a[7] != Py_None) {
      const at::Tensor& phases = must_be_tensor(a[7], "phases");
      u = phases_of(phases, c.d, device);
      rot = 2 * static_cast<int>(phases.numel());
      check(a[8] != Py_None, "positions must be given with phases");
      const at::Tensor& t = must_be_tensor(a[8], "positions");
      int32_of("positions", t, {T}, device);
      pos = static_cast<const int32_t*>(t.data_ptr());
    }
    const bool interleaved = truth(a[9]);
    const float factor = static_cast<float>(number(a[10]));
    if (T == 0) Py_RETURN_NONE;
    const c10::cuda::OptionalCUDAGuard guard(device);
    const Stream stream(a[11], device.index());
    const int rc = attn_paged_append_fp8(k.data_ptr(), v.data_ptr(), T, c.heads, c.d, k.stride(0), k.stride(1), v.stride(0),
                                         v.stride(1), static_cast<const int32_t*>(slots.data_ptr()), pos, u, rot, interleaved,
                                         factor, c.k->data_ptr(), c.v->data_ptr(), static_cast<float*>(c.ks->data_ptr()),
                                         static_cast<float*>(c.vs->data_ptr()), c.pages, c.page_size, stream.handle);
    if (rc != ATTN_OK) return status_error(rc, "attn_paged_append_fp8");
    for (const at::Tensor* t : {c.k, c.v, c.ks, c.vs}) written(*t);
    Py_RETURN_NONE;
  });
}

// paged(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, q_start, max_q, max_kv, causal,
// scale, num_splits,
//       out, lse, workspace, stream)
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 17) type_error("paged takes 17 arguments");
    const at::Tensor& q = bf16_rows(a[0], "q");
    const Cache c(a + 1);
    const at::Device device = q.device();
    const int T = dim32(q.size(0), "T"), Hq = dim32(q.size(1), "Hq"), d = c.d;
    check(q.size(2) == d && c.heads > 0 && Hq % c.heads == 0, "q must have the cache's d and a multiple of its heads");
    check(c.k->device() == device, "q and the cache must be on one device");
    const at::Tensor &table = must_be_tensor(a[5], "block_table"), &lens = must_be_tensor(a[6], "kv_len");
    check(table.dim() == 2, "block_table must be [B, pages]");
    const int B = dim32(table.size(0), "B"), width = dim32(table.size(1), "pages");
    int32_of("block_table", table, {B, width}, device);
    int32_of("kv_len", lens, {B}, device);
    const int32_t* start = nullptr;
    if (a[7] != Py_None) {
      const at::Tensor& t = must_be_tensor(a[7], "q_start");
      int32_of("q_start", t, {B + 1LL}, device);
      start = static_cast<const int32_t*>(t.data_ptr());
    } else {
      check(B > 0 && T % B == 0, "without q_start, T must be a multiple of the batch");
    }
    const c10::cuda::OptionalCUDAGuard guard(device);
    const Stream stream(a[16], device.index());
    at::Tensor o, lse, ws;
    const bool made_o = a[13] == Py_None, made_l = a[14] == Py_None;
    if (made_o) {
      o = stream.alloc([&] { return new_tensor({T, Hq, d}, at::kBFloat16, device); });
    } else {
      o = must_be_tensor(a[13], "out");
      check(o.sizes() == q.sizes() && o.scalar_type() == at::kBFloat16 && o.is_contiguous() && o.device() == device,
            "out must be a contiguous bf16 tensor shaped like q on q's device");
    }
    if (made_l) {
      lse = stream.alloc([&] { return new_tensor({T, Hq}, at::kFloat, device); });
    } else {
      lse = must_be_tensor(a[14], "lse");
      check(lse.dim() == 2 && lse.size(0) == T && lse.size(1) == Hq && lse.scalar_type() == at::kFloat && lse.is_contiguous() &&
                lse.device() == device,
            "lse must be a contiguous fp32 [T, Hq] tensor on q's device");
    }
    if (T > 0 && B > 0) {
      const float scale = a[11] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : static_cast<float>(number(a[11]));
      const int max_q = a[8] == Py_None ? (start ? T : T / B) : integer32(a[8], "max_q");
      const int64_t held = std::max<int64_t>(static_cast<int64_t>(width) * c.page_size, 1);
      const int max_kv = a[9] == Py_None ? static_cast<int>(std::min<int64_t>(held, INT32_MAX)) : integer32(a[9], "max_kv");
      const bool causal = truth(a[10]);
      const int splits = a[12] == Py_None
                             ? attn_fwd_fp8_paged_num_splits(B, Hq, c.heads, d, c.page_size, max_q, max_kv, at::cuda::getCurrentDeviceProperties()->multiProcessorCount)
                             : integer32(a[12], "num_splits");
      void* ws_ptr = nullptr;
      size_t ws_bytes = 0;
      if (a[15] != Py_None) {
        ws = must_be_tensor(a[15], "workspace");
        check(ws.device() == device && ws.is_contiguous(), "workspace must be a contiguous tensor on q's device");
        ws_bytes = ws.nbytes();
      } else if ((ws_bytes = attn_fwd_fp8_paged_workspace_size(T, Hq, c.heads, d, max_q, splits)) > 0) {
        ws = stream.alloc([&] { return new_tensor({static_cast<int64_t>(ws_bytes)}, at::kByte, device); });
      }
      if (ws.defined()) ws_ptr = ws.data_ptr();
      const int rc = attn_fwd_fp8_paged(
          q.data_ptr(), q.stride(0), q.stride(1), c.k->data_ptr(), c.v->data_ptr(), static_cast<const float*>(c.ks->data_ptr()),
          static_cast<const float*>(c.vs->data_ptr()), static_cast<const int32_t*>(table.data_ptr()), width, start,
          static_cast<const int32_t*>(lens.data_ptr()), o.data_ptr(), static_cast<float*>(lse.data_ptr()), B, T, Hq, c.heads, d,
          c.pages, c.page_size, max_q, max_kv, scale, causal, splits, ws_ptr, ws_bytes, stream.handle);
      if (rc != ATTN_OK) return status_error(rc, "attn_fwd_fp8_paged");
      if (made_o) stream.returns(o);
      else written(o);
      if (made_l) stream.returns(lse);
      else written(lse);
    }
    PyObject* po = THPVariable_Wrap(std::move(o));
    PyObject* pl = THPVariable_Wrap(std::move(lse));
    if (!po || !pl) throw python_error();
    PyObject* both = PyTuple_Pack(2, po, pl);
    Py_DECREF(po);
    Py_DECREF(pl);
    return both;
  });
}

// set_error(AttnError)
PyObject* set_error(PyObject*, PyObject* type) {
  Py_XDECREF(g_attn_error);
  Py_INCREF(type);
  g_attn_error = type;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
