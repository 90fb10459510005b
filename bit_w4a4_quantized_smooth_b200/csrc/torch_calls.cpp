// The 8-bit layer's calls on torch tensors: argument checks, outputs from
// torch's caching allocator, the current stream, then the C ABI
// (include/svdq.h).  At a few tokens a call's kernel takes a few microseconds,
// and a ctypes call with its checks in Python took 13 to 17 (measured, with
// outputs allocated): that is why these checks are native.
//
// Every function takes its arguments by position (binding.py holds the
// documented signatures), returns its outputs, raises ValueError for tensors
// that the C ABI could not see to be wrong, and the package's SvdqError for a
// status of the ABI.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <sstream>
#include <string>

#include "../../include/svdq.h"

namespace {

PyObject* g_error = nullptr;  // the package's SvdqError

struct Refusal {
  std::string message;
};

struct StatusError {
  int status;
  const char* what;
};

template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refusal{s.str()};
}

using Opt = std::optional<at::Tensor>;

at::Tensor tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, ": expected a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

Opt maybe(PyObject* o, const char* name) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, name);
}

void* ptr(const Opt& t) { return t ? t->data_ptr() : nullptr; }

bool truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw python_error();
  return t != 0;
}

constexpr auto kCodes = at::kFloat8_e4m3fn;
constexpr auto kScales = at::kFloat8_e8m0fnu;

// One tensor's type, shape, device and density.  `alt` is a second type allowed.
void need(const at::Tensor& t, const char* name, at::ScalarType type, at::ScalarType alt, at::IntArrayRef shape,
          at::Device dev) {
  const auto st = t.scalar_type();
  if (st != type && st != alt) refuse(name, ": dtype ", st, ", expected ", type, type == alt ? "" : " (or its alternative)");
  if (t.sizes() != shape) refuse(name, ": shape ", t.sizes(), ", expected ", shape);
  if (t.device() != dev) refuse(name, ": on ", t.device(), ", expected ", dev);
  if (!t.is_contiguous()) refuse(name, ": not contiguous");
}

int64_t scales_len(int64_t rows, int64_t K) { return ((rows + 127) / 128) * ((K + 511) / 512) * 512; }

// (M, K, row stride) of a 2-D bf16 CUDA tensor with unit column stride and rows that do not overlap.
struct Rows {
  int64_t M, K, ld;
};

Rows rows_of(const at::Tensor& X, const char* name) {
  if (X.scalar_type() != at::kBFloat16 || X.dim() != 2)
    refuse(name, ": expected a 2-D bfloat16 tensor, got ", X.dim(), "-D ", X.scalar_type());
  if (!X.is_cuda()) refuse(name, ": on ", X.device(), ", expected a CUDA device");
  const int64_t M = X.size(0), K = X.size(1), s0 = X.stride(0), s1 = X.stride(1);
  if ((s1 != 1 && K > 1) || (M > 1 && s0 < K))
    refuse(name, ": strides (", s0, ", ", s1, "), expected unit columns and rows that do not overlap");
  return {M, K, M > 1 ? s0 : K};
}

// The stream argument's handle: None = the device's current stream.
struct StreamArg {
  bool given = false;
  cudaStream_t handle = nullptr;
};

StreamArg stream_arg(PyObject* o, at::Device dev) {
  StreamArg s;
  if (o == Py_None) return s;
  const pybind11::handle h(o);
  if (h.attr("device_index").cast<int>() != dev.index())
    refuse("the stream is on device ", h.attr("device_index").cast<int>(), ", the tensors on ", dev);
  s.given = true;
  s.handle = reinterpret_cast<cudaStream_t>(h.attr("cuda_stream").cast<uintptr_t>());
  return s;
}

// Runs `f(stream)` with the tensors' device current and without the GIL (f
// also allocates outputs, which belong to the stream that writes them), and
// turns its status into an exception.
template <typename F>
void run(const char* what, at::Device dev, const StreamArg& s, F&& f) {
  int status = 0;
  {
    pybind11::gil_scoped_release nogil;
    if (s.given) {
      const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(s.handle, dev.index()));
      status = f(static_cast<void*>(s.handle));
    } else {
      const c10::cuda::CUDAGuard guard(dev);
      status = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    }
  }
  if (status != SVDQ_OK) throw StatusError{status, what};
}

// Outputs that were not given, up to two dimensions each, in ONE allocation:
// an allocation with its release costs 0.6 us of a 4 us call, a tensor 0.3.
// Straight from the allocator, past the dispatcher; the device and the stream
// that writes them are current (run()).
struct Wanted {
  Opt* out;
  int64_t rows, cols;  // cols 0: one dimension
  at::ScalarType type;
  int64_t bytes() const { return (rows * (cols ? cols : 1) * static_cast<int64_t>(at::elementSize(type)) + 255) / 256 * 256; }
};

void make_outputs(at::ArrayRef<Wanted> all) {
  int64_t bytes = 0;
  for (const Wanted& w : all) bytes += w.bytes();
  c10::Allocator* from = c10::cuda::CUDACachingAllocator::get();
  const c10::Storage storage(c10::Storage::use_byte_size_t(), static_cast<size_t>(bytes),
                             from->allocate(static_cast<size_t>(bytes)), from, /*resizable=*/true);
  int64_t at_byte = 0;
  for (const Wanted& w : all) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(storage),
                                                            c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                            c10::scalarTypeToTypeMeta(w.type));
    const int64_t shape[2] = {w.rows, w.cols};
    t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(shape, w.cols ? 2 : 1));
    t.unsafeGetTensorImpl()->set_storage_offset(at_byte / static_cast<int64_t>(at::elementSize(w.type)));
    at_byte += w.bytes();
    *w.out = std::move(t);
  }
}

// Outputs that a caller may keep for different times share an allocation only
// up to this size, the allocator's small blocks: a kept one keeps the others'
// memory.  (Codes and scales, which are used together, always share.)
constexpr int64_t kShareBytes = 1 << 20;

// Codes and scales of [rows][K]: given ones are checked here, missing ones are made by fill().
struct Fp8Out {
  int64_t rows, K;
  at::Device dev;
  Opt codes, scales;
  Fp8Out(int64_t rows, int64_t K, at::Device dev, PyObject* c, PyObject* s, const char* cn, const char* sn)
      : rows(rows), K(K), dev(dev), codes(maybe(c, cn)), scales(maybe(s, sn)) {
    if (codes) need(*codes, cn, kCodes, at::kByte, {rows, K}, dev);
    if (scales) need(*scales, sn, kScales, at::kByte, {scales_len(rows, K)}, dev);
  }
  template <typename List>
  void want(List& list) {
    if (!codes) list.push_back({&codes, rows, K, kCodes});
    if (!scales) list.push_back({&scales, scales_len(rows, K), 0, kScales});
  }
  void fill() {
    c10::SmallVector<Wanted, 2> list;
    want(list);
    if (!list.empty()) make_outputs(list);
  }
  uint8_t* c() const { return static_cast<uint8_t*>(ptr(codes)); }
  uint8_t* s() const { return static_cast<uint8_t*>(ptr(scales)); }
};

// Outputs that the caller gave have been written to: autograd's version counter
// of each goes up, as after any in-place operation, so that a backward pass
// that saved one of them notices.  (Inference tensors have none.)
void written(std::initializer_list<const Opt*> outs) {
  for (const Opt* t : outs)
    if (*t && !(*t)->is_inference()) (*t)->unsafeGetTensorImpl()->bump_version();
}

PyObject* wrap(const Opt& t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}

PyObject* tuple(std::initializer_list<const Opt*> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const Opt* t : ts) PyTuple_SET_ITEM(out, i++, wrap(*t));
  return out;
}

template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) return PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
  try {
    return F(a);
  } catch (const Refusal& e) {
    PyErr_SetString(PyExc_ValueError, e.message.c_str());
    return nullptr;
  } catch (const StatusError& e) {
    PyObject* inst = PyObject_CallFunction(g_error, "is", e.status, e.what);
    if (inst) {
      PyErr_SetObject(g_error, inst);
      Py_DECREF(inst);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (W, w_codes, w_scales, stream)
PyObject* pack_weight(PyObject* const* a) {
  const at::Tensor W = tensor(a[0], "W");
  if (W.dim() != 2 || !W.is_cuda()) refuse("W: expected a 2-D CUDA tensor, got ", W.dim(), "-D on ", W.device());
  const int64_t K = W.size(0), N = W.size(1);
  need(W, "W", at::kBFloat16, at::kFloat, {K, N}, W.device());
  Fp8Out out(N, K, W.device(), a[1], a[2], "w_codes", "w_scales");
  run("svdq_pack_weight_fp8", W.device(), stream_arg(a[3], W.device()), [&](void* st) {
    out.fill();
    return svdq_pack_weight_fp8(W.data_ptr(), W.scalar_type() == at::kFloat ? SVDQ_F32 : SVDQ_BF16, K, N, out.c(),
                                out.s(), st);
  });
  written({&out.codes, &out.scales});
  return tuple({&out.codes, &out.scales});
}

// (X, x_codes, x_scales, stream, gelu)
PyObject* quantize(PyObject* const* a) {
  const at::Tensor X = tensor(a[0], "X");
  const Rows r = rows_of(X, "X");
  Fp8Out out(r.M, r.K, X.device(), a[1], a[2], "x_codes", "x_scales");
  const int gelu = truth(a[4]);
  run("svdq_quantize_fp8", X.device(), stream_arg(a[3], X.device()), [&](void* st) {
    out.fill();
    return svdq_quantize_fp8(X.data_ptr(), r.ld, r.M, r.K, gelu, out.c(), out.s(), st);
  });
  written({&out.codes, &out.scales});
  return tuple({&out.codes, &out.scales});
}

// (X, gamma, residual, eps, residual_out, Y, x_codes, x_scales, fp8_out, bf16_out, stream)
PyObject* rmsnorm(PyObject* const* a) {
  const at::Tensor X = tensor(a[0], "X");
  const Rows r = rows_of(X, "X");
  const at::Device dev = X.device();
  const Opt gamma = maybe(a[1], "gamma"), residual = maybe(a[2], "residual");
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  Opt residual_out = maybe(a[4], "residual_out"), Y = maybe(a[5], "Y");
  const bool fp8_out = truth(a[8]), bf16_out = truth(a[9]);
  if (gamma) need(*gamma, "gamma", at::kBFloat16, at::kBFloat16, {r.K}, dev);
  if (residual) {
    need(*residual, "residual", at::kBFloat16, at::kFloat, {r.M, r.K}, dev);
    if (residual_out)
      need(*residual_out, "residual_out", residual->scalar_type(), residual->scalar_type(), {r.M, r.K}, dev);
  } else if (residual_out) {
    refuse("residual_out without a residual");
  }
  if (!fp8_out && (a[6] != Py_None || a[7] != Py_None)) refuse("x_codes or x_scales with fp8_out=False");
  Fp8Out out(r.M, r.K, dev, a[6], a[7], "x_codes", "x_scales");
  if (Y) need(*Y, "Y", at::kBFloat16, at::kBFloat16, {r.M, r.K}, dev);
  run("svdq_rmsnorm", dev, stream_arg(a[10], dev), [&](void* st) {
    c10::SmallVector<Wanted, 4> list;
    if (fp8_out) out.want(list);
    const size_t fp8 = list.size();
    if (residual && !residual_out) list.push_back({&residual_out, r.M, r.K, residual->scalar_type()});
    if (!Y && bf16_out) list.push_back({&Y, r.M, r.K, at::kBFloat16});
    int64_t bytes = 0;
    for (const Wanted& w : list) bytes += w.bytes();
    if (bytes > kShareBytes) {
      if (fp8) make_outputs(at::ArrayRef<Wanted>(list.data(), fp8));
      for (size_t i = fp8; i < list.size(); ++i) make_outputs(at::ArrayRef<Wanted>(list.data() + i, 1));
    } else if (!list.empty()) {
      make_outputs(list);
    }
    return svdq_rmsnorm(X.data_ptr(), r.ld, ptr(residual),
                        residual && residual->scalar_type() == at::kFloat ? SVDQ_F32 : SVDQ_BF16, ptr(gamma),
                        static_cast<float>(eps), r.M, r.K, ptr(residual_out), ptr(Y), out.c(), out.s(), st);
  });
  written({&out.codes, &out.scales, &residual_out, &Y});
  return tuple({&out.codes, &out.scales, &residual_out, &Y});
}

struct LinearArgs {
  at::Tensor xc, xs, wc, ws;
  Opt bias;
  int64_t M, K, N;
  at::Device dev;
  explicit LinearArgs(PyObject* const* a)
      : xc(tensor(a[0], "x_codes")), xs(tensor(a[1], "x_scales")), wc(tensor(a[2], "w_codes")),
        ws(tensor(a[3], "w_scales")), bias(maybe(a[4], "bias")), M(0), K(0), N(0), dev(xc.device()) {
    if (xc.dim() != 2 || wc.dim() != 2 || !xc.is_cuda())
      refuse("x_codes, w_codes: expected 2-D CUDA tensors, got ", xc.dim(), "-D on ", dev, " and ", wc.dim(), "-D");
    M = xc.size(0);
    K = xc.size(1);
    N = wc.size(0);
    need(xc, "x_codes", kCodes, at::kByte, {M, K}, dev);
    need(xs, "x_scales", kScales, at::kByte, {scales_len(M, K)}, dev);
    need(wc, "w_codes", kCodes, at::kByte, {N, K}, dev);
    need(ws, "w_scales", kScales, at::kByte, {scales_len(N, K)}, dev);
    if (bias) need(*bias, "bias", at::kBFloat16, at::kBFloat16, {N}, dev);
  }
  static const uint8_t* u8(const at::Tensor& t) { return static_cast<const uint8_t*>(t.data_ptr()); }
};

// (x_codes, x_scales, w_codes, w_scales, bias, Y, stream)
PyObject* linear(PyObject* const* a) {
  const LinearArgs l(a);
  Opt Y = maybe(a[5], "Y");
  if (Y) need(*Y, "Y", at::kBFloat16, at::kBFloat16, {l.M, l.N}, l.dev);
  run("svdq_linear_fp8", l.dev, stream_arg(a[6], l.dev), [&](void* st) {
    if (!Y) make_outputs(Wanted{&Y, l.M, l.N, at::kBFloat16});
    return svdq_linear_fp8(l.u8(l.xc), l.u8(l.xs), l.u8(l.wc), l.u8(l.ws), ptr(l.bias), l.M, l.K, l.N, ptr(Y), st);
  });
  written({&Y});
  return wrap(Y);
}

// (x_codes, x_scales, w_codes, w_scales, bias, y_codes, y_scales, stream)
PyObject* linear_gelu(PyObject* const* a) {
  const LinearArgs l(a);
  Fp8Out out(l.M, l.N, l.dev, a[5], a[6], "y_codes", "y_scales");
  run("svdq_linear_fp8_gelu", l.dev, stream_arg(a[7], l.dev), [&](void* st) {
    out.fill();
    return svdq_linear_fp8_gelu(l.u8(l.xc), l.u8(l.xs), l.u8(l.wc), l.u8(l.ws), ptr(l.bias), l.M, l.K, l.N, out.c(),
                                out.s(), st);
  });
  written({&out.codes, &out.scales});
  return tuple({&out.codes, &out.scales});
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  Py_INCREF(cls);
  g_error = cls;
  Py_RETURN_NONE;
}

#define SVDQ_ENTRY(f, n) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"pack_weight_fp8", SVDQ_ENTRY(pack_weight, 4)},
                         {"quantize_fp8", SVDQ_ENTRY(quantize, 5)},
                         {"rmsnorm", SVDQ_ENTRY(rmsnorm, 11)},
                         {"linear_fp8", SVDQ_ENTRY(linear, 7)},
                         {"linear_fp8_gelu", SVDQ_ENTRY(linear_gelu, 8)},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_svdq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__svdq_torch() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", SVDQ_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
