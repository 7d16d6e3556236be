// fused_binding.cpp -- the binding of the fused and grouped GEMMs: one CPython call that checks the tensors, allocates
// the output and calls the C ABI.  The smallest of these GEMMs take 6 to 12 us on the GPU; the same checks written in
// Python take 10.4 us a call, here 5.5 (2.5 of them the launch and its tensor maps).  Everything else of the package is
// bound through ctypes.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "bsp.h"

namespace {

// A refused argument: the message of a ValueError.
struct Refused {
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void want(bool ok, const char* name, const char* type, int64_t n) {
  if (!ok) refuse(std::string(name) + " must be a contiguous " + type + " tensor of " + std::to_string(n) + " elements");
}

// Elements between the first and one past the last of a row-major matrix.
int64_t span(const at::Tensor& t) { return (t.size(0) - 1) * t.stride(0) + t.size(1); }

// Whether two row-major matrices of one shape and type share an element.
bool overlap(const at::Tensor& a, const at::Tensor& b) {
  if (a.numel() == 0) return false;
  const int64_t size = a.element_size();
  const auto pa = reinterpret_cast<intptr_t>(a.data_ptr()), pb = reinterpret_cast<intptr_t>(b.data_ptr());
  if (pa >= pb + span(b) * size || pb >= pa + span(a) * size) return false;
  const int64_t ld = a.stride(0), cols = a.size(1);
  if (ld != b.stride(0) || ld < cols || (pb - pa) % size != 0) return true;
  const int64_t gap = (((pb - pa) / size) % ld + ld) % ld;  // column ranges modulo the common row stride
  return gap < cols || (ld - gap) % ld < cols;
}

// Other Python threads run while this one allocates and launches (either may block: a full launch queue waits for the
// stream, and a host function in the stream may wait for the interpreter).
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

struct Call {
  int64_t fp4, K, activation, gated;
  PyObject *ca, *sfa, *cb, *sfb, *offsets, *alpha, *row_scale, *bias, *f32, *out, *residual;
};

PyObject* run(const Call& c) {
  const at::Tensor &ca = tensor(c.ca, "A"), &sfa = tensor(c.sfa, "A's scales"), &cb = tensor(c.cb, "B"),
                   &sfb = tensor(c.sfb, "B's scales");
  const bool fp4 = c.fp4 != 0, grouped = c.offsets != Py_None;
  const int64_t K = c.K;
  // sizes; a hand-made operand whose buffers are smaller than they say would be read out of range
  const int64_t width = fp4 ? K / 2 : K, tiles = (K / (fp4 ? 16 : 32) + 3) / 4 * 512;  // scale bytes per 128 rows
  if (K < 0 || ca.dim() != 2 || ca.size(1) != width || ca.scalar_type() != at::kByte || !ca.is_contiguous())
    refuse("A: expected contiguous uint8 codes [M, " + std::to_string(width) + "]");
  if (cb.dim() != (grouped ? 3 : 2) || cb.size(-1) != width || cb.scalar_type() != at::kByte || !cb.is_contiguous())
    refuse(std::string("B: expected contiguous uint8 codes [") + (grouped ? "E, N, " : "N, ") + std::to_string(width) + "]");
  const int64_t M = ca.size(0), N = cb.size(-2), E = grouped ? cb.size(0) : 1;
  if (grouped && (E < 1 || E > BSP_MAX_EXPERTS))
    refuse("1 to " + std::to_string(BSP_MAX_EXPERTS) + " experts, got " + std::to_string(E));
  if (sfa.numel() != (M + 127) / 128 * tiles || sfa.scalar_type() != at::kByte || !sfa.is_contiguous())
    refuse("A: expected " + std::to_string((M + 127) / 128 * tiles) + " contiguous scale bytes");
  if (sfb.numel() != E * ((N + 127) / 128) * tiles || sfb.scalar_type() != at::kByte || !sfb.is_contiguous())
    refuse("B: expected " + std::to_string(E * ((N + 127) / 128) * tiles) + " contiguous scale bytes");
  if (c.gated && N % 2 != 0) refuse("a gated weight has an even number of rows");
  const int64_t cols = c.gated ? N / 2 : N;

  bsp_fused_gemm_desc d = {};
  bool cuda = ca.is_cuda() && sfa.is_cuda() && cb.is_cuda() && sfb.is_cuda();
  const c10::Device device = ca.device();
  bool same = sfa.device() == device && cb.device() == device && sfb.device() == device;
  auto add = [&](const at::Tensor& t) {
    cuda = cuda && t.is_cuda();
    same = same && t.device() == device;
    return t.data_ptr();
  };
  auto plain = [](const at::Tensor& t, at::ScalarType type, int64_t n) {
    return t.scalar_type() == type && t.numel() == n && t.is_contiguous();
  };
  if (grouped) {
    const at::Tensor& t = tensor(c.offsets, "offsets");
    want(t.dim() == 1 && plain(t, at::kInt, E + 1), "offsets", "int32", E + 1);
    d.offsets = static_cast<const int32_t*>(add(t));
  }
  if (c.alpha != Py_None) {
    const at::Tensor& t = tensor(c.alpha, "alpha");
    want(plain(t, at::kFloat, E), "alpha", "fp32", E);
    d.alpha = static_cast<const float*>(add(t));
  }
  if (c.row_scale != Py_None) {
    const at::Tensor& t = tensor(c.row_scale, "row_scale");
    want(plain(t, at::kFloat, M), "row_scale", "fp32", M);
    d.row_scale = static_cast<const float*>(add(t));
  }
  if (c.bias != Py_None) {
    const at::Tensor& t = tensor(c.bias, "bias");
    want(plain(t, at::kBFloat16, E * N), "bias", "bf16", E * N);
    d.bias = static_cast<const uint16_t*>(add(t));
  }
  const bool f32 = c.f32 == Py_True;
  const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
  auto matrix = [&](const at::Tensor& t) {
    return t.dim() == 2 && t.size(0) == M && t.size(1) == cols && t.stride(1) == 1 && t.scalar_type() == type;
  };
  if (c.out != Py_None) {
    const at::Tensor& t = tensor(c.out, "out");
    if (!matrix(t)) refuse("out must be a row-major [M, N] tensor of the output dtype");
    add(t);
  }
  if (c.residual != Py_None) {
    const at::Tensor& t = tensor(c.residual, "residual");
    if (!matrix(t)) refuse("residual must be a row-major tensor of the output's shape and dtype");
    d.residual = add(t);
    d.ld_residual = t.stride(0);
  }
  if (!cuda) refuse("libbsp runs on CUDA tensors only (no CPU path)");
  if (!same) refuse("operands on different devices");

  at::Tensor out;
  int status;
  {
    const Unlocked unlocked;
    // the launch goes to the operands' device and its current stream
    const c10::cuda::CUDAGuard guard(device);
    out = c.out != Py_None ? THPVariable_Unpack(c.out)
                           : at::empty({M, cols}, at::TensorOptions().dtype(type).device(device));
    d.D = out.data_ptr();
    d.ld_d = out.stride(0);
    if (M == 1) d.ld_d = d.ld_residual = (cols + 7) / 8 * 8;  // one row has no stride: a broadcast's or a slice's is anything
    if (d.residual != nullptr && (d.residual != d.D || d.ld_residual != d.ld_d)) {
      if (overlap(THPVariable_Unpack(c.residual), out))
        refuse("residual may be the output itself, but must not overlap it otherwise");
    }
    d.A = static_cast<const uint8_t*>(ca.data_ptr());
    d.sfA = static_cast<const uint8_t*>(sfa.data_ptr());
    d.B = static_cast<const uint8_t*>(cb.data_ptr());
    d.sfB = static_cast<const uint8_t*>(sfb.data_ptr());
    d.E = E;
    d.M = M;
    d.N = N;
    d.K = K;
    d.activation = c.activation;
    d.gated = c.gated;
    d.d_dtype = f32 ? BSP_OUT_F32 : BSP_OUT_BF16;
    const bsp_stream_t stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    status = fp4 ? nvfp4_gemm_fused(&d, stream) : mxfp8_gemm_fused(&d, stream);
  }
  if (status != BSP_OK) return PyLong_FromLong(status);
  if (c.out != Py_None) {
    Py_INCREF(c.out);
    return c.out;
  }
  return THPVariable_Wrap(out);
}

// fused_gemm(fp4, A, sfA, B, sfB, K, offsets, alpha, row_scale, bias, f32, out, activation, gated, residual):
// the output, or the status of a call that the library refused.
PyObject* fused_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15) {
    PyErr_SetString(PyExc_TypeError, "fused_gemm takes 15 arguments");
    return nullptr;
  }
  Call c = {};
  c.fp4 = PyObject_IsTrue(a[0]);
  c.ca = a[1], c.sfa = a[2], c.cb = a[3], c.sfb = a[4];
  c.K = PyLong_AsLongLong(a[5]);
  c.offsets = a[6], c.alpha = a[7], c.row_scale = a[8], c.bias = a[9], c.f32 = a[10], c.out = a[11];
  c.activation = PyLong_AsLongLong(a[12]);
  c.gated = PyObject_IsTrue(a[13]);
  c.residual = a[14];
  if (PyErr_Occurred()) return nullptr;
  try {
    return run(c);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (...) {  // torch's own type for each of its errors: out of memory is torch.OutOfMemoryError, as from torch.empty
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

PyMethodDef kMethods[] = {
    {"fused_gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fused_gemm)), METH_FASTCALL,
     "The fused and grouped GEMMs of libbsp on tensors."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fused_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fused_binding() {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", BSP_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
