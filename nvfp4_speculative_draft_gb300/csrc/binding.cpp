// binding.cpp -- native argument marshalling of the verify step's and the attention step's calls.
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

#include <cmath>
#include <cstdint>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <utility>

#include "nvfp4draft.h"

namespace {

using at::Tensor;

constexpr int64_t kBlock = 128;

struct Library {
  decltype(&::fp8b_quantize) quantize = nullptr;
  decltype(&::fp8b_rmsnorm) rmsnorm = nullptr;
  decltype(&::fp8b_gemm) gemm = nullptr;
  decltype(&::spec_verify) verify = nullptr;
  decltype(&::kv_plan) plan = nullptr;
  decltype(&::rope_kv_write) rope = nullptr;
  decltype(&::prompt_attention) prompt = nullptr;
  decltype(&::paged_attention) paged = nullptr;
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
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
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

// ------------------------------------------------------------ attention step

// [tokens, heads, dim] BF16 rows with unit stride along dim.
const Tensor& need_heads(PyObject* o, const char* name, at::Device dev, int64_t tokens, int64_t heads, int64_t dim) {
  const Tensor* t = tensor_of(o);
  if (!is(t, at::kBFloat16, dev, {tokens, heads, dim}) || (t->stride(2) != 1 && dim != 1))
    refuse(name, t, at::kBFloat16, {tokens, heads, dim}, " with unit stride along the last axis");
  return *t;
}
// The first tensor of a call, which gives its sizes.
const Tensor& first_heads(PyObject* o, const char* name) {
  const Tensor& t = *tensor_of(o);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || (t.stride(2) != 1 && t.size(2) != 1))
    refuse(name, &t, at::kBFloat16, {-1, -1, -1}, " with unit stride along the last axis");
  return t;
}
// Strides for the library: those of an extent of 1 are arbitrary in torch.
attn_rows rows_of(const Tensor& t) {
  attn_rows r{t.data_ptr(), t.stride(0), t.stride(1)};
  if (t.size(1) <= 1) r.ld_head = (t.size(2) + 7) / 8 * 8;
  if (t.size(0) <= 1) r.ld_token = t.size(1) <= 1 ? r.ld_head : t.size(1) * r.ld_head;
  return r;
}
// What is written to: no element twice.
void need_distinct(const Tensor& t, const char* name) {
  int64_t order[4], n = 0;
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) != 1) order[n++] = i;
  for (int64_t i = 1; i < n; ++i)
    for (int64_t j = i; j > 0 && t.stride(order[j]) < t.stride(order[j - 1]); --j) std::swap(order[j], order[j - 1]);
  int64_t reach = 1;  // elements up to the last of the axes so far
  for (int64_t i = 0; i < n; ++i) {
    if (t.stride(order[i]) < reach) throw Refusal(std::string(name) + " must not overlap itself");
    reach += (t.size(order[i]) - 1) * t.stride(order[i]);
  }
}
const Tensor& need_pages(PyObject* o, const char* name, at::Device dev, at::IntArrayRef shape) {
  const Tensor* t = tensor_of(o);
  const bool any = shape.empty();  // the first of the two
  if (t == nullptr || t->scalar_type() != at::kBFloat16 || t->device() != dev || t->dim() != 4 ||
      (!any && t->sizes() != shape) || (t->stride(3) != 1 && t->size(3) != 1))
    refuse(name, t, at::kBFloat16, any ? at::IntArrayRef({-1, -1, -1, -1}) : shape,
           " [pages, page size, heads, dim] with unit stride along the last axis");
  return *t;
}
kv_pages pages_of(const Tensor& t) {
  kv_pages r{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
  if (t.size(2) <= 1) r.ld_head = (t.size(3) + 7) / 8 * 8;
  if (t.size(1) <= 1) r.ld_token = t.size(2) <= 1 ? r.ld_head : t.size(2) * r.ld_head;
  if (t.size(0) <= 1) r.ld_page = t.size(1) <= 1 ? r.ld_token : t.size(1) * r.ld_token;
  return r;
}
int64_t number(PyObject* o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}
// int32 vectors, given or made: those that are made share one allocation, 64 bytes aligned.
struct Vectors {
  static constexpr int64_t kAlign = 16;
  int64_t words = 0;
  Tensor all;
  int64_t add(PyObject* o, const char* name, at::Device dev, int64_t n) {
    if (o != Py_None) {
      need_vector(o, name, at::kInt, dev, n);
      return -1;
    }
    const int64_t at = words;
    words += (n + kAlign - 1) / kAlign * kAlign;
    return at;
  }
  Tensor get(PyObject* o, int64_t at, int64_t n) const {
    if (at < 0) return *tensor_of(o);
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
  }
};

// plan(lens, num_new, block_table, free_pages, free_count, page_size, tokens, held | None,
//      cu_new | None, kv_lens | None, positions | None, slots | None, held_out | None,
//      free_count_out | None, stream, dev_status) -> six tensors
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(16)
  const at::Device dev = device_of(a[0], "lens");
  const Tensor& lens = *tensor_of(a[0]);
  if (lens.dim() != 1) refuse("lens", &lens, at::kInt, {-1}, "");
  kv_plan_input in{};
  in.batch = lens.size(0);
  in.lens = need_vector(a[0], "lens", at::kInt, dev, in.batch).data_ptr<int32_t>();
  in.num_new = need_vector(a[1], "num_new", at::kInt, dev, in.batch).data_ptr<int32_t>();
  const Tensor* table = tensor_of(a[2]);
  if (table == nullptr || table->dim() != 2) refuse("block_table", table, at::kInt, {in.batch, -1}, kRowsText);
  need_rows(a[2], "block_table", at::kInt, dev, {in.batch, table->size(1)});
  in.block_table = table->data_ptr<int32_t>();
  in.max_pages = table->size(1);
  in.ld_table = in.batch > 1 ? table->stride(0) : in.max_pages;
  const Tensor* free = tensor_of(a[3]);
  if (free == nullptr || free->dim() != 1) refuse("free_pages", free, at::kInt, {-1}, " contiguous");
  in.free_capacity = free->size(0);
  in.free_pages = need_vector(a[3], "free_pages", at::kInt, dev, in.free_capacity).data_ptr<int32_t>();
  in.free_count = need_vector(a[4], "free_count", at::kInt, dev, 1).data_ptr<int32_t>();
  in.page_size = number(a[5]);
  in.tokens = number(a[6]);
  if (in.tokens < 0 || in.tokens > 0x7FFFFFFF) throw Refusal("tokens must be in 0 .. 2^31 - 1");
  if (a[7] != Py_None) in.held = need_vector(a[7], "held", at::kInt, dev, in.batch).data_ptr<int32_t>();
  const Call call(dev, a[14], a[15]);
  const char* names[6] = {"cu_new", "kv_lens", "positions", "slots", "held_out", "free_count_out"};
  const int64_t sizes[6] = {in.batch + 1, in.batch, in.tokens, in.tokens, in.batch, 1};
  Vectors made;
  int64_t where[6];
  for (int i = 0; i < 6; ++i) where[i] = made.add(a[8 + i], names[i], dev, sizes[i]);
  if (made.words > 0) made.all = make({made.words}, at::kInt, dev);
  Tensor v[6];
  for (int i = 0; i < 6; ++i) v[i] = made.get(a[8 + i], where[i], sizes[i]);
  const Tensor &cu = v[0], &kv = v[1], &positions = v[2], &slots = v[3], &held = v[4], &count = v[5];
  const kv_plan_output out{cu.data_ptr<int32_t>(),    kv.data_ptr<int32_t>(),   positions.data_ptr<int32_t>(),
                           slots.data_ptr<int32_t>(), held.data_ptr<int32_t>(), count.data_ptr<int32_t>()};
  const int rc = lib.plan(&in, &out, &call.ex);
  if (rc != NVFP4_OK) return fail("kv_plan", rc);
  return Py_BuildValue("(NNNNNN)", wrap(cu), wrap(kv), wrap(positions), wrap(slots), wrap(held), wrap(count));
  CALL_END
}

// rope(q, k, v | None, positions, turns, axis, axes, k_cache | None, v_cache | None, slots | None,
//      q_out | None, k_out | None, stream, dev_status) -> (q, k | None)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(14)
  const at::Device dev = device_of(a[0], "q");
  const Tensor& q = first_heads(a[0], "q");
  rope_kv_input in{};
  rope_kv_output out{};
  in.tokens = q.size(0);
  in.heads = q.size(1);
  in.dim = q.size(2);
  const Tensor* kt = tensor_of(a[1]);
  in.kv_heads = kt != nullptr && kt->dim() == 3 ? kt->size(1) : 1;
  const Tensor& k = need_heads(a[1], "k", dev, in.tokens, in.kv_heads, in.dim);
  in.q = rows_of(q);
  in.k = rows_of(k);
  in.axes = number(a[6]);
  const Tensor* pos = tensor_of(a[3]);
  if (pos != nullptr && pos->dim() == 2) {
    need_rows(a[3], "positions", at::kInt, dev, {in.axes, in.tokens});
    in.ld_positions = in.axes > 1 ? pos->stride(0) : in.tokens;
  } else {  // one row for all axes
    need_vector(a[3], "positions", at::kInt, dev, in.tokens);
  }
  in.positions = pos->data_ptr<int32_t>();
  const Tensor* turns = tensor_of(a[4]);
  if (turns == nullptr || turns->dim() != 1) refuse("rotary.turns", turns, at::kLong, {-1}, " contiguous");
  const int64_t pairs = turns->size(0);
  in.rot_dim = 2 * pairs;
  if (in.rot_dim > in.dim) throw Refusal("the rotary table has more pairs than a head");
  in.turns = reinterpret_cast<const uint64_t*>(need_vector(a[4], "rotary.turns", at::kLong, dev, pairs).data_ptr());
  in.axis = need_vector(a[5], "rotary.axis", at::kByte, dev, pairs).data_ptr<uint8_t>();
  const bool cached = a[7] != Py_None;
  if (cached != (a[8] != Py_None) || cached != (a[9] != Py_None))
    throw Refusal("k_cache, v_cache and slots go together");
  if (cached) {
    const Tensor& kc = need_pages(a[7], "k_cache", dev, {});
    if (kc.size(2) != in.kv_heads || kc.size(3) != in.dim) throw Refusal("k_cache must have the heads of k");
    const Tensor& vc = need_pages(a[8], "v_cache", dev, kc.sizes());
    need_distinct(kc, "k_cache");
    need_distinct(vc, "v_cache");
    in.k_cache = pages_of(kc);
    in.v_cache = pages_of(vc);
    in.pages = kc.size(0);
    in.page_size = kc.size(1);
    in.v = rows_of(need_heads(a[2], "v", dev, in.tokens, in.kv_heads, in.dim));
    in.slots = need_vector(a[9], "slots", at::kInt, dev, in.tokens).data_ptr<int32_t>();
  }
  const Call call(dev, a[12], a[13]);
  const Tensor qo = a[10] != Py_None ? need_heads(a[10], "q_out", dev, in.tokens, in.heads, in.dim)
                                     : make({in.tokens, in.heads, in.dim}, at::kBFloat16, dev);
  need_distinct(qo, "q_out");
  out.q = rows_of(qo);
  Tensor ko;
  if (a[11] != Py_None) {
    ko = need_heads(a[11], "k_out", dev, in.tokens, in.kv_heads, in.dim);
    need_distinct(ko, "k_out");
  } else if (!cached) {
    ko = make({in.tokens, in.kv_heads, in.dim}, at::kBFloat16, dev);
  }
  if (ko.defined()) out.k = rows_of(ko);
  const int rc = lib.rope(&in, &out, &call.ex);
  if (rc != NVFP4_OK) return fail("rope_kv_write", rc);
  return Py_BuildValue("(NN)", a[10] != Py_None ? Py_NewRef(a[10]) : wrap(qo),
                       a[11] != Py_None ? Py_NewRef(a[11]) : ko.defined() ? wrap(ko) : Py_NewRef(Py_None));
  CALL_END
}

// scale | None: 1 / sqrt(dim)
float scale_of(PyObject* o, int64_t dim) {
  if (o == Py_None) return (float)(1.0 / std::sqrt((double)dim));
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)x;
}
// out | None, workspace | None -> the output and the call's workspace, which lives until the
// call's work is queued: the allocator hands its memory on in stream order.
struct AttentionOutputs {
  Tensor out, workspace;
  attn_rows rows;
  AttentionOutputs(PyObject* given, PyObject* ws, const Tensor& q, Call& call) {
    out = given != Py_None ? need_heads(given, "out", q.device(), q.size(0), q.size(1), q.size(2))
                           : make(q.sizes(), at::kBFloat16, q.device());
    need_distinct(out, "out");
    rows = rows_of(out);
    if (ws != Py_None) {
      const Tensor* t = tensor_of(ws);
      if (t == nullptr || t->device() != q.device() || !t->is_contiguous())
        throw Refusal("workspace must be a contiguous tensor on the call's device");
      workspace = *t;
    } else {
      workspace = make({(int64_t)ATTENTION_WS_BYTES}, at::kByte, q.device());
    }
    call.ex.workspace = workspace.data_ptr();
    call.ex.workspace_bytes = workspace.nbytes();
  }
};

// prompt(q, k, v, cu, scale | None, out | None, workspace | None, stream, dev_status) -> out
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(9)
  const at::Device dev = device_of(a[0], "q");
  const Tensor& q = first_heads(a[0], "q");
  prompt_attention_input in{};
  in.tokens = q.size(0);
  in.heads = q.size(1);
  in.dim = q.size(2);
  const Tensor* kt = tensor_of(a[1]);
  in.kv_heads = kt != nullptr && kt->dim() == 3 ? kt->size(1) : 1;
  in.q = rows_of(q);
  in.k = rows_of(need_heads(a[1], "k", dev, in.tokens, in.kv_heads, in.dim));
  in.v = rows_of(need_heads(a[2], "v", dev, in.tokens, in.kv_heads, in.dim));
  const Tensor* cu = tensor_of(a[3]);
  if (cu == nullptr || cu->dim() != 1 || cu->size(0) < 1) refuse("cu_seqlens", cu, at::kInt, {-1}, " contiguous");
  in.batch = cu->size(0) - 1;
  in.cu = need_vector(a[3], "cu_seqlens", at::kInt, dev, in.batch + 1).data_ptr<int32_t>();
  in.scale = scale_of(a[4], in.dim);
  Call call(dev, a[7], a[8]);
  const AttentionOutputs o(a[5], a[6], q, call);
  const int rc = lib.prompt(&in, &o.rows, &call.ex);
  if (rc != NVFP4_OK) return fail("prompt_attention", rc);
  return a[5] != Py_None ? Py_NewRef(a[5]) : wrap(o.out);
  CALL_END
}

// paged(q, k_cache, v_cache, block_table, kv_lens, cu_new, scale | None, out | None,
//       workspace | None, stream, dev_status) -> out
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  CALL_BEGIN(11)
  const at::Device dev = device_of(a[0], "q");
  const Tensor& q = first_heads(a[0], "q");
  paged_attention_input in{};
  in.tokens = q.size(0);
  in.heads = q.size(1);
  in.dim = q.size(2);
  in.q = rows_of(q);
  const Tensor& kc = need_pages(a[1], "k_cache", dev, {});
  if (kc.size(3) != in.dim) throw Refusal("k_cache must have heads of the size of q's");
  const Tensor& vc = need_pages(a[2], "v_cache", dev, kc.sizes());
  in.pages = kc.size(0);
  in.page_size = kc.size(1);
  in.kv_heads = kc.size(2);
  in.k = pages_of(kc);
  in.v = pages_of(vc);
  const Tensor* lens = tensor_of(a[4]);
  if (lens == nullptr || lens->dim() != 1) refuse("kv_lens", lens, at::kInt, {-1}, " contiguous");
  in.batch = lens->size(0);
  in.kv_lens = need_vector(a[4], "kv_lens", at::kInt, dev, in.batch).data_ptr<int32_t>();
  const Tensor* table = tensor_of(a[3]);
  if (table == nullptr || table->dim() != 2) refuse("block_table", table, at::kInt, {in.batch, -1}, kRowsText);
  need_rows(a[3], "block_table", at::kInt, dev, {in.batch, table->size(1)});
  in.block_table = table->data_ptr<int32_t>();
  in.max_pages = table->size(1);
  in.ld_table = in.batch > 1 ? table->stride(0) : in.max_pages;
  in.cu = need_vector(a[5], "cu_new", at::kInt, dev, in.batch + 1).data_ptr<int32_t>();
  in.scale = scale_of(a[6], in.dim);
  Call call(dev, a[9], a[10]);
  const AttentionOutputs o(a[7], a[8], q, call);
  const int rc = lib.paged(&in, &o.rows, &call.ex);
  if (rc != NVFP4_OK) return fail("paged_attention", rc);
  return a[7] != Py_None ? Py_NewRef(a[7]) : wrap(o.out);
  CALL_END
}

// bind(quantize, rmsnorm, gemm, verify, plan, rope, prompt, paged, error): the library's
// functions by address
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  constexpr int kCalls = 8;
  if (nargs != kCalls + 1) {
    PyErr_SetString(PyExc_TypeError, "bind takes eight addresses and an exception class");
    return nullptr;
  }
  void* f[kCalls];
  for (int i = 0; i < kCalls; ++i) {
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
  lib.plan = reinterpret_cast<decltype(lib.plan)>(f[4]);
  lib.rope = reinterpret_cast<decltype(lib.rope)>(f[5]);
  lib.prompt = reinterpret_cast<decltype(lib.prompt)>(f[6]);
  lib.paged = reinterpret_cast<decltype(lib.paged)>(f[7]);
  Py_XDECREF(lib.error);
  lib.error = Py_NewRef(a[kCalls]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                         {"quantize", FAST(quantize), METH_FASTCALL, nullptr},
                         {"rmsnorm", FAST(rmsnorm), METH_FASTCALL, nullptr},
                         {"gemm", FAST(gemm), METH_FASTCALL, nullptr},
                         {"verify", FAST(verify), METH_FASTCALL, nullptr},
                         {"plan", FAST(plan), METH_FASTCALL, nullptr},
                         {"rope", FAST(rope), METH_FASTCALL, nullptr},
                         {"prompt", FAST(prompt), METH_FASTCALL, nullptr},
                         {"paged", FAST(paged), METH_FASTCALL, nullptr},
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
