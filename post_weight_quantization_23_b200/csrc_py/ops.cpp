// The Python entry of the adapter, checkpoint and input-gradient operators: checks
// every tensor's type, shape, strides and device, allocates what the caller did not
// pass, and calls the C ABI (include/gptq.h) on the current stream of the tensors'
// device.  For single tokens a call's host time counts as much as its kernel's, and these
// checks cost 5 us in Python against 0.5 us here.  Positional arguments only; the
// functions of the package document them.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/gptq.h"

namespace {

PyObject* g_error = nullptr;  // GptqError(status, where, detail)

struct Refused {
  gptq_status status;
  std::string detail;
};

[[noreturn]] void refuse(const std::string& detail, gptq_status st = GPTQ_ERR_INVALID_ARG) {
  throw Refused{st, detail};
}

PyObject* raise(const char* where, const Refused& r) {
  PyObject* e = PyObject_CallFunction(g_error, "iss", (int)r.status, where, r.detail.c_str());
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

std::string text(const at::Tensor& t) {
  std::string s = "(";
  for (auto d : t.sizes()) s += std::to_string(d) + ", ";
  return s + ") " + c10::toString(t.scalar_type());
}

// The device that every tensor of a call is on.
struct Device {
  int index = -1;
  void see(const char* name, const at::Tensor& t) {
    if (!t.is_cuda()) refuse(std::string(name) + ": tensor not on a CUDA device");
    const int d = t.get_device();
    if (index >= 0 && d != index) refuse(std::string(name) + ": tensors on different devices");
    index = d;
  }
};

const at::Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": not a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = optional(o, name);
  if (t == nullptr) refuse(std::string(name) + ": not a tensor");
  return *t;
}

// A (rows, cols) matrix of the type with unit column stride; its leading dimension.
int64_t matrix(const char* name, const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType dt,
               Device& dev) {
  if (t.scalar_type() != dt || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(std::string(name) + ": " + text(t) + ", want (" + std::to_string(rows) + ", " +
           std::to_string(cols) + ") " + c10::toString(dt));
  if (cols > 1 && t.stride(1) != 1) refuse(std::string(name) + ": unit column stride");
  dev.see(name, t);
  const int64_t ld = t.stride(0);
  return rows > 1 && cols > 0 ? ld : std::max<int64_t>({ld, cols, 1});
}

// A contiguous tensor of the type and sizes; its address.
template <typename P>
P* whole(const char* name, const at::Tensor& t, at::IntArrayRef sizes, at::ScalarType dt,
         Device& dev) {
  if (t.scalar_type() != dt || t.sizes() != sizes || !t.is_contiguous()) {
    std::string want;
    for (auto d : sizes) want += std::to_string(d) + ", ";
    refuse(std::string(name) + ": " + text(t) + ", want contiguous (" + want + ") " +
           c10::toString(dt));
  }
  dev.see(name, t);
  return static_cast<P*>(t.data_ptr());
}

gptq_dtype dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return GPTQ_F32;
    case at::kHalf: return GPTQ_F16;
    case at::kBFloat16: return GPTQ_BF16;
    default: refuse(std::string("dtype ") + c10::toString(t.scalar_type()));
  }
}

// A tensor of the caller's that the call writes.  The calls record nothing for autograd, so
// under grad mode an update of a tensor that requires grad would be missing from its gradients:
// refused, as torch refuses it for out= arguments.
const at::Tensor& target(const char* name, const at::Tensor& t) {
  if (c10::GradMode::is_enabled() && t.requires_grad())
    refuse(std::string(name) + ": written, and requires grad (call it under torch.no_grad() or "
           "inside an autograd.Function)");
  return t;
}
const at::Tensor* target(const char* name, const at::Tensor* t) {
  if (t != nullptr) target(name, *t);
  return t;
}

// Such a tensor has changed: an autograd graph that saved it finds out.  (An inference tensor
// has no version.)
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void changed(const at::Tensor* t) {
  if (t != nullptr) changed(*t);
}

at::Tensor make(at::IntArrayRef sizes, const at::Tensor& like, at::ScalarType dt) {
  return at::empty(sizes, like.options().dtype(dt).requires_grad(false));
}

// Runs fn(stream) with the tensors' device current.
template <typename F>
void launch(const Device& dev, F fn) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != dev.index) guard.set_index(dev.index);
  const gptq_status st =
      fn(reinterpret_cast<gptq_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index).stream()));
  if (st != GPTQ_OK) refuse("", st);
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(std::to_string(n) + " arguments, want " + std::to_string(want));
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + ": not an integer");
  }
  return v;
}

struct Adapters {
  int64_t na, r, k, n, nreq;
  const void *A, *B;
  const float* scaling;
  const int32_t *starts, *adapter;
};

Adapters adapters(PyObject* const* o, at::ScalarType dt, Device& dev) {
  const at::Tensor &A = tensor(o[0], "A"), &B = tensor(o[1], "B"), &sc = tensor(o[2], "scaling"),
                   &st = tensor(o[3], "starts"), &ad = tensor(o[4], "adapter");
  if (A.dim() != 3 || B.dim() != 3 || ad.dim() != 1)
    refuse("A (na, rank, k), B (na, n, rank), adapter (requests,)");
  Adapters a;
  a.na = A.size(0), a.r = A.size(1), a.k = A.size(2), a.n = B.size(1), a.nreq = ad.size(0);
  a.A = whole<void>("A", A, {a.na, a.r, a.k}, dt, dev);
  a.B = whole<void>("B", B, {a.na, a.n, a.r}, dt, dev);
  a.scaling = whole<float>("scaling", sc, {a.na}, at::kFloat, dev);
  a.starts = whole<int32_t>("starts", st, {a.nreq + 1}, at::kInt, dev);
  a.adapter = whole<int32_t>("adapter", ad, {a.nreq}, at::kInt, dev);
  return a;
}

PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}

#define GPTQ_ENTRY(name, where)                                                  \
  PyObject* name##_impl(PyObject* const* a, Py_ssize_t n);                       \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {                  \
    HANDLE_TH_ERRORS                                                             \
    try {                                                                        \
      return name##_impl(a, n);                                                  \
    } catch (const Refused& r) {                                                 \
      return raise(where, r);                                                    \
    }                                                                            \
    END_HANDLE_TH_ERRORS                                                         \
  }                                                                              \
  PyObject* name##_impl(PyObject* const* a, Py_ssize_t n)

// Y, X, A, B, scaling, starts, adapter, out, V -> the updated tensor
GPTQ_ENTRY(lora_add, "gptq_lora_add") {
  count(n, 9);
  Device dev;
  const at::Tensor &X = tensor(a[1], "X"), *Y = optional(a[0], "Y"),
                   *V = target("V", optional(a[8], "V"));
  PyObject* to = a[7] != Py_None ? a[7] : a[0];
  const at::Tensor& out = target("Y or out", tensor(to, "Y or out"));
  const at::ScalarType dt = X.scalar_type();
  const gptq_dtype code = dtype_code(X);
  const Adapters d = adapters(a + 2, dt, dev);
  if (X.dim() != 2) refuse("X: (m, k)");
  const int64_t m = X.size(0);
  const int64_t ldx = matrix("X", X, m, d.k, dt, dev), ldo = matrix("out", out, m, d.n, dt, dev);
  const int64_t ldy = Y != nullptr ? matrix("Y", *Y, m, d.n, dt, dev) : 0;
  float* pv = V != nullptr ? whole<float>("V", *V, {m, d.r}, at::kFloat, dev) : nullptr;
  launch(dev, [&](gptq_stream_t s) {
    return gptq_lora_add(Y != nullptr ? Y->data_ptr() : nullptr, ldy, X.data_ptr(), code, m, d.k, ldx,
                         d.A, d.B, d.scaling, d.na, (int)d.r, d.starts, d.adapter, d.nreq, d.n,
                         out.data_ptr(), ldo, pv, s);
  });
  changed(out);
  changed(V);
  return given(to);
}

// dY, X, V, A, B, scaling, starts, adapter, dX, x_scales, out, dA, dB, ws -> (out, dA, dB)
GPTQ_ENTRY(lora_backward, "gptq_lora_backward") {
  count(n, 14);
  Device dev;
  const at::Tensor &dY = tensor(a[0], "dY"), &X = tensor(a[1], "X"), &V = tensor(a[2], "V");
  const at::Tensor *dX = optional(a[8], "dX"), *xs = optional(a[9], "x_scales");
  PyObject* to = a[10] != Py_None ? a[10] : a[8];
  const at::Tensor* out = target("dX or out", optional(to, "out"));
  const at::ScalarType dt = dY.scalar_type();
  const gptq_dtype code = dtype_code(dY);
  const Adapters d = adapters(a + 3, dt, dev);
  if (dY.dim() != 2) refuse("dY: (m, n)");
  const int64_t m = dY.size(0);
  const int64_t ldy = matrix("dY", dY, m, d.n, dt, dev);
  const int64_t ldx = matrix("X", X, m, d.k, xs != nullptr ? at::kChar : dt, dev);
  const float* pxs =
      xs != nullptr ? whole<float>("x_scales", *xs, {m, (d.k + 127) / 128}, at::kFloat, dev) : nullptr;
  const float* pv = whole<float>("V", V, {m, d.r}, at::kFloat, dev);
  const int64_t ldo = out != nullptr ? matrix("out", *out, m, d.k, dt, dev) : 0;
  const int64_t ldd = out != nullptr && dX != nullptr ? matrix("dX", *dX, m, d.k, dt, dev) : 0;
  const at::Tensor *gA = target("dA", optional(a[11], "dA")),
                   *gB = target("dB", optional(a[12], "dB")), *ws = target("ws", optional(a[13], "ws"));
  const at::Tensor dA = gA != nullptr ? *gA : make({d.na, d.r, d.k}, dY, dt);
  const at::Tensor dB = gB != nullptr ? *gB : make({d.na, d.n, d.r}, dY, dt);
  void* pa = whole<void>("dA", dA, {d.na, d.r, d.k}, dt, dev);
  void* pb = whole<void>("dB", dB, {d.na, d.n, d.r}, dt, dev);
  const int64_t need = (int64_t)gptq_workspace_size(GPTQ_OP_LORA_BACKWARD, d.r, 0, m, nullptr);
  const at::Tensor w = ws != nullptr ? *ws : make({std::max<int64_t>(need, 1)}, dY, at::kByte);
  dev.see("ws", w);
  if (!w.is_contiguous()) refuse("ws: contiguous");
  launch(dev, [&](gptq_stream_t s) {
    return gptq_lora_backward(
        dY.data_ptr(), code, m, d.n, ldy, X.data_ptr(), ldx, pxs, d.k, pv, d.A, d.B, d.scaling, d.na,
        (int)d.r, d.starts, d.adapter, d.nreq,
        out != nullptr && dX != nullptr ? dX->data_ptr() : nullptr, ldd,
        out != nullptr ? out->data_ptr() : nullptr, ldo, pa, pb, w.data_ptr(), w.nbytes(), s);
  });
  changed(out);
  changed(gA);
  changed(gB);
  changed(ws);
  PyObject* res = PyTuple_New(3);
  if (res == nullptr) return nullptr;
  PyTuple_SET_ITEM(res, 0, given(to));
  PyTuple_SET_ITEM(res, 1, gA != nullptr ? given(a[11]) : THPVariable_Wrap(dA));
  PyTuple_SET_ITEM(res, 2, gB != nullptr ? given(a[12]) : THPVariable_Wrap(dB));
  return res;
}

// X, codes, scales -> (codes, scales)
GPTQ_ENTRY(act_checkpoint, "gptq_act_checkpoint") {
  count(n, 3);
  Device dev;
  const at::Tensor& X = tensor(a[0], "X");
  const at::Tensor *gc = target("codes", optional(a[1], "codes")),
                   *gs = target("scales", optional(a[2], "scales"));
  const gptq_dtype code = dtype_code(X);
  if (X.dim() != 2) refuse("X: (m, k)");
  const int64_t m = X.size(0), k = X.size(1), nb = (k + 127) / 128;
  const int64_t ldx = matrix("X", X, m, k, X.scalar_type(), dev);
  const at::Tensor codes = gc != nullptr ? *gc : make({m, k}, X, at::kChar);
  const at::Tensor scales = gs != nullptr ? *gs : make({m, nb}, X, at::kFloat);
  const int64_t ldc = matrix("codes", codes, m, k, at::kChar, dev);
  float* ps = whole<float>("scales", scales, {m, nb}, at::kFloat, dev);
  launch(dev, [&](gptq_stream_t s) {
    return gptq_act_checkpoint(X.data_ptr(), code, m, k, ldx,
                               static_cast<int8_t*>(codes.data_ptr()), ldc, ps, s);
  });
  changed(gc);
  changed(gs);
  PyObject* res = PyTuple_New(2);
  if (res == nullptr) return nullptr;
  PyTuple_SET_ITEM(res, 0, gc != nullptr ? given(a[1]) : THPVariable_Wrap(codes));
  PyTuple_SET_ITEM(res, 1, gs != nullptr ? given(a[2]) : THPVariable_Wrap(scales));
  return res;
}

// codes, scales, dtype, out -> the activations
GPTQ_ENTRY(act_restore, "gptq_act_restore") {
  count(n, 4);
  Device dev;
  const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
  const at::Tensor* go = target("out", optional(a[3], "out"));
  if (codes.dim() != 2) refuse("codes: (m, k)");
  if (go == nullptr && !THPDtype_Check(a[2])) refuse("dtype: not a torch.dtype");
  const int64_t m = codes.size(0), k = codes.size(1);
  const int64_t ldc = matrix("codes", codes, m, k, at::kChar, dev);
  const float* ps = whole<float>("scales", scales, {m, (k + 127) / 128}, at::kFloat, dev);
  const at::Tensor out =
      go != nullptr ? *go : make({m, k}, codes, reinterpret_cast<THPDtype*>(a[2])->scalar_type);
  const gptq_dtype code = dtype_code(out);
  const int64_t ldo = matrix("out", out, m, k, out.scalar_type(), dev);
  launch(dev, [&](gptq_stream_t s) {
    return gptq_act_restore(static_cast<const int8_t*>(codes.data_ptr()), ldc, ps, m, k, code,
                            out.data_ptr(), ldo, s);
  });
  changed(go);
  return go != nullptr ? given(a[3]) : THPVariable_Wrap(out);
}

// dY, qweight, scales, zeros, bits, group_size, k, g_idx, out -> dX
GPTQ_ENTRY(gemm_dgrad, "gptq_gemm_dgrad") {
  count(n, 9);
  Device dev;
  const at::Tensor &dY = tensor(a[0], "dY"), &qw = tensor(a[1], "qweight"),
                   &sc = tensor(a[2], "scales"), &ze = tensor(a[3], "zeros");
  const int64_t bits = integer(a[4], "bits"), group = integer(a[5], "group_size"),
                k = integer(a[6], "k");
  const at::Tensor *gi = optional(a[7], "g_idx"), *go = target("out", optional(a[8], "out"));
  const gptq_dtype code = dtype_code(dY);
  if (dY.dim() != 2 || sc.dim() != 2) refuse("dY (m, n), scales (n, ngroups)");
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8)
    refuse("bits " + std::to_string(bits), GPTQ_ERR_UNSUPPORTED);
  if (k < 0 || group < -1 || group > INT32_MAX) refuse("k, group_size");
  const int64_t m = dY.size(0), nn = dY.size(1), ng = sc.size(1);
  const int64_t ldy = matrix("dY", dY, m, nn, dY.scalar_type(), dev);
  const int32_t* pq = whole<int32_t>("qweight", qw, {nn, k * bits / 32}, at::kInt, dev);
  const float* ps = whole<float>("scales", sc, {nn, ng}, at::kFloat, dev);
  const int32_t* pz = whole<int32_t>("zeros", ze, {nn, ng}, at::kInt, dev);
  const int32_t* pg = gi != nullptr ? whole<int32_t>("g_idx", *gi, {k}, at::kInt, dev) : nullptr;
  const at::Tensor out = go != nullptr ? *go : make({m, k}, dY, dY.scalar_type());
  const int64_t ldx = matrix("out", out, m, k, dY.scalar_type(), dev);
  launch(dev, [&](gptq_stream_t s) {
    return gptq_gemm_dgrad(dY.data_ptr(), code, m, nn, ldy, pq, ps, pz, pg, k, (int)bits, (int)group,
                           ng, out.data_ptr(), ldx, s);
  });
  changed(go);
  return go != nullptr ? given(a[8]) : THPVariable_Wrap(out);
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XINCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"lora_add", (PyCFunction)(void (*)(void))lora_add, METH_FASTCALL, nullptr},
    {"lora_backward", (PyCFunction)(void (*)(void))lora_backward, METH_FASTCALL, nullptr},
    {"act_checkpoint", (PyCFunction)(void (*)(void))act_checkpoint, METH_FASTCALL, nullptr},
    {"act_restore", (PyCFunction)(void (*)(void))act_restore, METH_FASTCALL, nullptr},
    {"gemm_dgrad", (PyCFunction)(void (*)(void))gemm_dgrad, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&g_module); }
