// binding.cpp -- native argument marshalling of the verify step's calls.
//
// A single token's kernels take two to ten microseconds, less than a Python function
// needs to check a call's tensors, allocate its outputs and fill the C structs.  This
// module does that against PyTorch's C++ tensors and calls the C ABI of nvfp4draft.h
// through the addresses that the Python package has loaded (bind()), so that there is
// one library whichever way it is reached.  It computes nothing.
//
// Refusals raise ValueError before the library is called; a status other than
// NVFP4_OK raises the package's error class.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "nvfp4draft.h"

namespace {

using at::Tensor;

constexpr int64_t kBlock = 128;

struct Library {
  decltype(&::fp8b_quantize) quantize = nullptr;
  decltype(&::fp8b_rmsnorm) rmsnorm = nullptr;
  decltype(&::fp8b_gemm) gemm = nullptr;
  decltype(&::spec_verify) verify = nullptr;
  PyObject* error = nullptr;
} lib;

PyObject *s_codes, *s_scales, *s_m, *s_n, *s_k;

struct Refusal : std::runtime_error {
  using std::runtime_error::runtime_error;
};

int64_t blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }

std::string shape_text(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << ")";
  return o.str();
}

const char* dtype_text(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn (or torch.uint8)";
    default: return "another type";
  }
}

[[noreturn]] void refuse(const char* name, const Tensor* t, at::ScalarType want, at::IntArrayRef shape,
                         const char* more) {
  std::ostringstream o;
  o << name << " must be " << dtype_text(want) << " " << shape_text(shape) << more << " on the call's device, got ";
  if (t == nullptr)
    o << "no tensor";
  else
    o << c10::toString(t->scalar_type()) << " " << shape_text(t->sizes()) << " strides " << shape_text(t->strides())
      << " on " << t->device();
  throw Refusal(o.str());
}

const Tensor* tensor_of(PyObject* o) {  // nullptr for what is not a tensor
  return o != nullptr && THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// The device of the call: its first tensor's.
at::Device device_of(PyObject* o, const char* name) {
  const Tensor* t = tensor_of(o);
  if (t == nullptr || !t->is_cuda()) throw Refusal(std::string(name) + " must be a CUDA tensor");
  return t->device();
}

bool is(const Tensor* t, at::ScalarType type, at::Device dev, at::IntArrayRef shape) {
  return t != nullptr && t->scalar_type() == type && t->device() == dev && t->sizes() == shape;
}
// 2-D with unit column stride and rows that do not overlap
bool rows_ok(const Tensor& t) {
  return (t.stride(1) == 1 || t.size(1) <= 1) && (t.stride(0) >= t.size(1) || t.size(0) <= 1);
}
constexpr const char* kRowsText = " with unit column stride and rows that do not overlap";

const Tensor& need_rows(PyObject* o, const char* name, at::ScalarType type, at::Device dev, at::IntArrayRef shape) {
  const Tensor* t = tensor_of(o);
  if (!is(t, type, dev, shape) || !rows_ok(*t)) refuse(name, t, type, shape, kRowsText);
  return *t;
}
// E4M3 codes: torch's own type, or the same bytes as uint8
const Tensor& need_codes(PyObject* o, const char* name, at::Device dev, at::IntArrayRef shape) {
  const Tensor* t = tensor_of(o);
  if (!(is(t, at::kFloat8_e4m3fn, dev, shape) || is(t, at::kByte, dev, shape)) || !rows_ok(*t))
    refuse(name, t, at::kFloat8_e4m3fn, shape, kRowsText);
  return *t;
}
const Tensor& need_vector(PyObject* o, const char* name, at::ScalarType type, at::Device dev, int64_t n) {
  const Tensor* t = tensor_of(o);
  if (!is(t, type, dev, {n}) || (t->stride(0) != 1 && n != 1)) refuse(name, t, type, {n}, " contiguous");
  return *t;
}
// Row stride for the library: a single row's is its length rounded up to a multiple
// of 16 (torch leaves the stride of an extent of 1 arbitrary).
int64_t ld(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : (t.size(1) + 15) / 16 * 16; }

Tensor make(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

int64_t integer(PyObject* o, PyObject* name) {
  PyObject* v = PyObject_GetAttr(o, name);
  if (v == nullptr) throw python_error();
  const int64_t x = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}
// An attribute, held until the call ends.
struct Attribute {
  PyObject* o;
  Attribute(PyObject* of, PyObject* name) : o(PyObject_GetAttr(of, name)) {
    if (o == nullptr) throw python_error();
  }
  Attribute(const Attribute&) = delete;
  ~Attribute() { Py_DECREF(o); }
};

// Stream, status word and current device of one call.  While it lives, the call's stream
// is the current one, so that outputs are allocated on it: memory that work queued on
// another stream may still use is not handed to this call, nor this call's to others.
// (So it is made before any output.)
struct Call {
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard stream_guard;
  nvfp4_exec ex;
  Call(at::Device dev, PyObject* stream, PyObject* status) {
    if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
    ex = nvfp4_exec{};
    const cudaStream_t current = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    if (stream == Py_None) {
      ex.stream = current;
    } else {
      ex.stream = PyLong_AsVoidPtr(stream);
      if (ex.stream == nullptr && PyErr_Occurred()) throw python_error();
      // (the legacy default stream's handle is another name of PyTorch's default stream)
      const cudaStream_t given =
          ex.stream == cudaStreamLegacy ? nullptr : static_cast<cudaStream_t>(ex.stream);
      if (given != current) stream_guard.reset_stream(c10::cuda::getStreamFromExternal(given, dev.index()));
    }
    if (status != Py_None) {
      const Tensor* t = tensor_of(status);
      if (t == nullptr || t->scalar_type() != at::kInt || t->device() != dev || t->numel() < 1)
        refuse("dev_status", t, at::kInt, {1}, "");
      ex.dev_status = t->data_ptr<int32_t>();
    }
  }
};

PyObject* fail(const char* call, int rc) {
  PyObject* e = PyObject_CallFunction(lib.error, "si", call, rc);
  if (e != nullptr) {
    PyErr_SetObject(lib.error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

#define CALL_BEGIN(n)                                                        \
  HANDLE_TH_ERRORS                                                           \
  if (nargs != (n) || lib.error == nullptr) {                                \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or bind() was not called"); \
    return nullptr;                                                          \
  }                                                                          \
  try {
#define CALL_END                                        \
  }                                                     \
  catch (const Refusal& r) {                            \
    PyErr_SetString(PyExc_ValueError, r.what());        \
    return nullptr;                                     \
  }                                                     \
  END_HANDLE_TH_ERRORS

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

struct Acts {
  Attribute codes, scales;
  at::Device dev;
  fp8b_act a{};
  explicit Acts(PyObject* o) : codes(o, s_codes), scales(o, s_scales), dev(device_of(codes.o, "acts.codes")) {
    a.m = integer(o, s_m);
    a.k = integer(o, s_k);
    const Tensor& c = need_codes(codes.o, "acts.codes", dev, {a.m, a.k});
    const Tensor& s = need_rows(scales.o, "acts.scales", at::kFloat, dev, {blocks(a.k), a.m});
    a.codes = static_cast<uint8_t*>(c.data_ptr());
    a.ld = ld(c);
    a.scales = s.data_ptr<float>();
    a.ld_scales = s.size(0) > 1 ? s.stride(0) : a.m;
  }
};

// quantize(w, codes | None, scales | None, stream, dev_status) -> (codes, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(5)
  const at::Device dev = device_of(a[0], "w");
  const Tensor& w = *tensor_of(a[0]);
  if (w.dim() != 2 || w.scalar_type() != at::kBFloat16 || !rows_ok(w))
    refuse("w", &w, at::kBFloat16, {-1, -1}, kRowsText);
  const Call call(dev, a[3], a[4]);
  const int64_t n = w.size(0), k = w.size(1);
  Tensor codes, scales;
  if (a[1] != Py_None) {
    codes = need_codes(a[1], "out.codes", dev, {n, k});
    scales = need_rows(a[2], "out.scales", at::kFloat, dev, {blocks(n), blocks(k)});
    if (!codes.is_contiguous() || !scales.is_contiguous()) throw Refusal("out must be contiguous");
  } else {
    codes = make({n, k}, at::kFloat8_e4m3fn, dev);
    scales = make({blocks(n), blocks(k)}, at::kFloat, dev);
  }
  const int rc = lib.quantize(w.data_ptr(), n, k, ld(w), static_cast<uint8_t*>(codes.data_ptr()), scales.data_ptr<float>(), &call.ex);
  if (rc != NVFP4_OK) return fail("fp8b_quantize", rc);
  return Py_BuildValue("(NN)", wrap(codes), wrap(scales));
  CALL_END
}

// rmsnorm(x, gamma | None, eps, residual | None, residual_out | None, out | None, stream,
//         dev_status) -> (codes, scales, h | None)
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(8)
  const at::Device dev = device_of(a[0], "x");
  const Tensor& x = *tensor_of(a[0]);
  if (x.dim() != 2 || x.scalar_type() != at::kBFloat16 || !rows_ok(x))
    refuse("x", &x, at::kBFloat16, {-1, -1}, kRowsText);
  const Call call(dev, a[6], a[7]);
  const int64_t m = x.size(0), k = x.size(1);
  fp8b_norm_input in{};
  in.x = x.data_ptr();
  in.ld_x = ld(x);
  if (a[1] != Py_None) in.gamma = need_vector(a[1], "gamma", at::kBFloat16, dev, k).data_ptr();
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  in.eps = (float)eps;
  Tensor h;
  if (a[3] != Py_None) {
    const Tensor& r = need_rows(a[3], "residual", at::kBFloat16, dev, {m, k});
    in.residual = r.data_ptr();
    in.ld_residual = ld(r);
    if (a[4] == Py_None) h = make({m, k}, at::kBFloat16, dev);
  }
  if (a[4] != Py_None) h = need_rows(a[4], "residual_out", at::kBFloat16, dev, {m, k});
  if (h.defined()) {
    in.residual_out = h.data_ptr();
    in.ld_residual_out = ld(h);
  }
  fp8b_act out{};
  Tensor codes, scales;
  if (a[5] != Py_None) {
    const Acts given(a[5]);
    if (given.dev != dev || given.a.m != m || given.a.k != k)
      throw Refusal("out must be activations of the shape and device of x");
    out = given.a;
  } else {
    codes = make({m, k}, at::kFloat8_e4m3fn, dev);
    scales = make({blocks(k), m}, at::kFloat, dev);
    out = fp8b_act{static_cast<uint8_t*>(codes.data_ptr()), ld(codes), scales.data_ptr<float>(), m, m, k};
  }
  const int rc = lib.rmsnorm(&in, &out, &call.ex);
  if (rc != NVFP4_OK) return fail("fp8b_rmsnorm", rc);
  PyObject* ho = a[4] != Py_None ? Py_NewRef(a[4]) : h.defined() ? wrap(h) : Py_NewRef(Py_None);
  if (a[5] != Py_None) return Py_BuildValue("(OON)", Py_None, Py_None, ho);
  return Py_BuildValue("(NNN)", wrap(codes), wrap(scales), ho);
  CALL_END
}

// gemm(acts, weight, dtype, out | None, stream, dev_status) -> out
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(6)
  const Acts acts(a[0]);
  const Attribute wc(a[1], s_codes), ws(a[1], s_scales);
  fp8b_weight w{};
  w.n = integer(a[1], s_n);
  w.k = integer(a[1], s_k);
  const at::Device dev = device_of(wc.o, "weight.codes");
  const Tensor& codes = need_codes(wc.o, "weight.codes", dev, {w.n, w.k});
  const Tensor& scales = need_rows(ws.o, "weight.scales", at::kFloat, dev, {blocks(w.n), blocks(w.k)});
  if (!codes.is_contiguous() || !scales.is_contiguous())
    throw Refusal("weight.codes and weight.scales must be contiguous");
  w.codes = static_cast<uint8_t*>(codes.data_ptr());
  w.scales = scales.data_ptr<float>();
  if (acts.dev != dev) throw Refusal("acts must be on the weight's device");
  if (acts.a.k != w.k) throw Refusal("acts must have k = " + std::to_string(w.k) + " columns, got " + std::to_string(acts.a.k));
  const Tensor* given = a[3] != Py_None ? tensor_of(a[3]) : nullptr;
  if (given == nullptr && (a[3] != Py_None || !THPDtype_Check(a[2]))) throw Refusal("out must be a tensor and out_dtype a torch.dtype");
  const at::ScalarType type = given != nullptr ? given->scalar_type() : reinterpret_cast<THPDtype*>(a[2])->scalar_type;
  if (type != at::kFloat && type != at::kBFloat16) throw Refusal("out must be float32 or bfloat16");
  const Call call(dev, a[4], a[5]);
  Tensor out = given != nullptr ? need_rows(a[3], "out", type, dev, {acts.a.m, w.n}) : make({acts.a.m, w.n}, type, dev);
  const int rc = lib.gemm(&acts.a, &w, out.data_ptr(), type == at::kFloat ? NVFP4_DTYPE_F32 : NVFP4_DTYPE_BF16,
                          out.size(0) > 1 ? out.stride(0) : out.size(1), &call.ex);
  if (rc != NVFP4_OK) return fail("fp8b_gemm", rc);
  return given != nullptr ? Py_NewRef(a[3]) : wrap(out);
  CALL_END
}

// verify(target, tokens, accept_u, sample_u, draft | None, num_draft | None,
//        out_tokens | None, out_accepted | None, stream, dev_status) -> (tokens, accepted)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(10)
  const at::Device dev = device_of(a[0], "target_probs");
  const Tensor& p = *tensor_of(a[0]);
  const at::ScalarType type = p.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) throw Refusal("target_probs must be float32 or bfloat16");
  if (p.dim() != 3 || p.size(1) < 1 || (p.stride(2) != 1 && p.size(2) != 1))
    refuse("target_probs", &p, type, {-1, -1, -1}, " [batch, g + 1, vocab] with unit stride along the vocabulary");
  spec_verify_input in{};
  in.batch = p.size(0);
  in.g = p.size(1) - 1;
  in.vocab = p.size(2);
  in.target = p.data_ptr();
  in.ld_target_seq = p.stride(0);
  in.ld_target_pos = p.stride(1);
  in.dtype = type == at::kFloat ? NVFP4_DTYPE_F32 : NVFP4_DTYPE_BF16;
  const bool one = in.batch == 1;  // torch leaves the stride of an extent of 1 arbitrary
  const Tensor& tokens = need_rows(a[1], "draft_tokens", at::kInt, dev, {in.batch, in.g});
  const Tensor& u = need_rows(a[2], "accept_u", at::kFloat, dev, {in.batch, in.g});
  in.sample_u = need_vector(a[3], "sample_u", at::kFloat, dev, in.batch).data_ptr<float>();
  if (in.g > 0) {
    in.tokens = tokens.data_ptr<int32_t>();
    in.ld_tokens = one ? in.g : tokens.stride(0);
    in.accept_u = u.data_ptr<float>();
    in.ld_accept_u = one ? in.g : u.stride(0);
  }
  if (a[4] != Py_None) {
    const Tensor* q = tensor_of(a[4]);
    const int64_t dv = q != nullptr && q->dim() == 3 ? q->size(2) : 0;
    if (!is(q, type, dev, {in.batch, in.g, dv}) || dv < 1 || dv > in.vocab || (q->stride(2) != 1 && dv != 1))
      refuse("draft_probs", q, type, {in.batch, in.g, in.vocab},
             " (or fewer of the first tokens) with unit stride along the vocabulary");
    if (in.g > 0) {
      in.draft = q->data_ptr();
      in.ld_draft_seq = q->stride(0);
      in.ld_draft_pos = q->stride(1);
      in.draft_vocab = dv;
    }
  }
  if (a[5] != Py_None) in.num_draft = need_vector(a[5], "num_draft", at::kInt, dev, in.batch).data_ptr<int32_t>();
  const Call call(dev, a[8], a[9]);
  Tensor out, accepted;
  if (a[6] != Py_None) {  // may be wider, or longer
    const Tensor* t = tensor_of(a[6]);
    if (t == nullptr || t->scalar_type() != at::kInt || t->device() != dev || t->dim() != 2 ||
        t->size(0) < in.batch || t->size(1) < in.g + 1 || !rows_ok(*t))
      refuse("out_tokens", t, at::kInt, {in.batch, in.g + 1}, kRowsText);
    out = *t;
  } else {
    out = make({in.batch, in.g + 1}, at::kInt, dev);
  }
  if (a[7] != Py_None) {
    const Tensor* t = tensor_of(a[7]);
    if (t == nullptr || t->scalar_type() != at::kInt || t->device() != dev || t->dim() != 1 ||
        t->size(0) < in.batch || (t->stride(0) != 1 && t->size(0) != 1))
      refuse("out_accepted", t, at::kInt, {in.batch}, " contiguous");
    accepted = *t;
  } else {
    accepted = make({in.batch}, at::kInt, dev);
  }
  const int rc = lib.verify(&in, out.data_ptr<int32_t>(), out.size(0) > 1 ? out.stride(0) : out.size(1),
                            accepted.data_ptr<int32_t>(), &call.ex);
  if (rc != NVFP4_OK) return fail("spec_verify", rc);
  return Py_BuildValue("(NN)", a[6] != Py_None ? Py_NewRef(a[6]) : wrap(out),
                       a[7] != Py_None ? Py_NewRef(a[7]) : wrap(accepted));
  CALL_END
}

// bind(quantize, rmsnorm, gemm, verify, error): the library's functions by address
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses and an exception class");
    return nullptr;
  }
  void* f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (f[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  lib.quantize = reinterpret_cast<decltype(lib.quantize)>(f[0]);
  lib.rmsnorm = reinterpret_cast<decltype(lib.rmsnorm)>(f[1]);
  lib.gemm = reinterpret_cast<decltype(lib.gemm)>(f[2]);
  lib.verify = reinterpret_cast<decltype(lib.verify)>(f[3]);
  Py_XDECREF(lib.error);
  lib.error = Py_NewRef(a[4]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                         {"quantize", FAST(quantize), METH_FASTCALL, nullptr},
                         {"rmsnorm", FAST(rmsnorm), METH_FASTCALL, nullptr},
                         {"gemm", FAST(gemm), METH_FASTCALL, nullptr},
                         {"verify", FAST(verify), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  s_codes = PyUnicode_InternFromString("codes");
  s_scales = PyUnicode_InternFromString("scales");
  s_m = PyUnicode_InternFromString("m");
  s_n = PyUnicode_InternFromString("n");
  s_k = PyUnicode_InternFromString("k");
  return PyModule_Create(&module);
}
