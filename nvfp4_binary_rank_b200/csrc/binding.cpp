// Fast path of the FP8 operators' Python calls.
//
// A decode step makes these calls once per layer with a few microseconds of GPU work in
// each, and marshalling them through ctypes, with outputs allocated from Python, took
// longer than the work (block norm of one token: 14 us a call).  These functions check a
// plain call (contiguous tensors of one device, which is the current one, on the current
// stream), allocate its outputs and call the C ABI.  They return the outputs, an int (the
// C ABI's status), or None for any call that is not plain: _fp8.py then checks it operand
// by operand and makes it, or says what is wrong with it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/biloco.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr ScalarType kBf16 = ScalarType::BFloat16, kF32 = ScalarType::Float, kFp8 = ScalarType::Float8_e4m3fn;

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous tensor of that type on CUDA device `dev`, with `dim` dimensions.
bool dense(const Tensor* t, ScalarType type, int dev, int64_t dim) {
  return t && t->defined() && t->is_cuda() && t->scalar_type() == type && t->get_device() == dev && t->dim() == dim &&
         t->is_contiguous();
}
bool is_real(ScalarType t) { return t == kBf16 || t == kF32; }
int type_code(ScalarType t) { return t == kBf16 ? BILOCO_TYPE_BF16 : BILOCO_TYPE_F32; }
int64_t blocks(int64_t n) { return (n + 127) / 128; }
bool small(int64_t n) { return n <= 0x7FFFFFFF; }

Tensor make(at::IntArrayRef shape, ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}
biloco_stream_t stream_of(int dev) {
  return reinterpret_cast<biloco_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}
// The CUDA device of a tensor if it is the current one, else -1.
int device_of(const Tensor* t) {
  if (!t || !t->defined() || !t->is_cuda()) return -1;
  const int dev = t->get_device();
  return dev == c10::cuda::current_device() ? dev : -1;
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* status(int st) { return PyLong_FromLong(st); }
PyObject* give(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// quant_act(x)
PyObject* quant_act(const Tensor* x) {
  const int dev = device_of(x);
  if (dev < 0 || !dense(x, kBf16, dev, 2) || !small(x->size(0)) || !small(x->size(1))) return none();
  const int64_t M = x->size(0), K = x->size(1);
  Tensor codes = make({M, K}, kFp8, dev), scales = make({blocks(K), M}, kF32, dev);
  const int st = biloco_fp8_quant_act(x->data_ptr(), K, static_cast<int>(M), static_cast<int>(K),
                                      static_cast<uint8_t*>(codes.data_ptr()), static_cast<float*>(scales.data_ptr()),
                                      stream_of(dev));
  return st ? status(st) : give({codes, scales});
}

// gemm(x_codes, x_scales, w_codes, w_scales, out or None, f32)
PyObject* gemm(PyObject* const* a) {
  const Tensor *x = tensor(a[0]), *xs = tensor(a[1]), *w = tensor(a[2]), *ws = tensor(a[3]);
  const int dev = device_of(x);
  if (dev < 0 || !dense(x, kFp8, dev, 2) || !dense(xs, kF32, dev, 2) || !dense(w, kFp8, dev, 2) || !dense(ws, kF32, dev, 2))
    return none();
  const int64_t M = x->size(0), K = x->size(1), N = w->size(0);
  if (w->size(1) != K || xs->size(0) != blocks(K) || xs->size(1) != M || ws->size(0) != blocks(N) ||
      ws->size(1) != blocks(K) || !small(M) || !small(N) || !small(K))
    return none();
  const bool f32 = a[5] == Py_True;
  Tensor y;
  if (a[4] == Py_None) {
    y = make({M, N}, f32 ? kF32 : kBf16, dev);
  } else {
    const Tensor* out = tensor(a[4]);
    if (!dense(out, f32 ? kF32 : kBf16, dev, 2) || out->size(0) != M || out->size(1) != N) return none();
    y = *out;
  }
  const int st = biloco_fp8_gemm(static_cast<const uint8_t*>(x->data_ptr()), static_cast<const float*>(xs->data_ptr()),
                                 static_cast<const uint8_t*>(w->data_ptr()), static_cast<const float*>(ws->data_ptr()),
                                 y.data_ptr(), f32 ? BILOCO_TYPE_F32 : BILOCO_TYPE_BF16, static_cast<int>(M),
                                 static_cast<int>(N), static_cast<int>(K), stream_of(dev));
  if (st) return status(st);
  if (a[4] != Py_None) {
    Py_INCREF(a[4]);
    return a[4];
  }
  return THPVariable_Wrap(y);
}

// norm(y, h, post_weight, pre_weight, gate, res_scale, offset, eps, quant)
PyObject* norm(PyObject* const* a) {
  const Tensor* t[5];
  for (int i = 0; i < 5; ++i) {
    t[i] = tensor(a[i]);
    if (!t[i] && a[i] != Py_None) return none();
  }
  const Tensor *y = t[0], *h = t[1], *post = t[2], *pre = t[3], *gate = t[4];
  const int dev = device_of(y ? y : h);
  if (dev < 0 || !pre || !y || !dense(y, kBf16, dev, 2)) return none();
  const int64_t M = y->size(0), D = y->size(1);
  const ScalarType ht = h ? h->scalar_type() : kBf16, wt = pre->scalar_type();
  if (!small(M) || !small(D) || !is_real(ht) || !is_real(wt)) return none();
  if (h && (!dense(h, ht, dev, 2) || h->size(0) != M || h->size(1) != D)) return none();
  if (!dense(pre, wt, dev, 1) || pre->size(0) != D) return none();
  if (post && (!dense(post, wt, dev, 1) || post->size(0) != D)) return none();
  int64_t G = 1;
  if (gate) {
    if (!is_real(gate->scalar_type()) || gate->dim() < 1 || gate->dim() > 2 ||
        !dense(gate, gate->scalar_type(), dev, gate->dim()) || gate->size(-1) != D)
      return none();
    G = gate->dim() == 2 ? gate->size(0) : 1;
    if (G < 1 || M % G) return none();
  }
  const double res = PyFloat_AsDouble(a[5]), offset = PyFloat_AsDouble(a[6]), eps = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  const bool quant = a[8] == Py_True;
  Tensor h2 = make({M, D}, ht, dev), x = make({M, D}, quant ? kFp8 : kBf16, dev), scales;
  if (quant) scales = make({blocks(D), M}, kF32, dev);
  const int st = biloco_block_norm(
      y->data_ptr(), D, h ? h->data_ptr() : nullptr, h ? D : 0, type_code(ht), post ? post->data_ptr() : nullptr,
      pre->data_ptr(), type_code(wt), gate ? gate->data_ptr() : nullptr, gate ? type_code(gate->scalar_type()) : 0,
      static_cast<int>(G), static_cast<float>(res), static_cast<float>(offset), static_cast<float>(eps),
      static_cast<int>(M), static_cast<int>(D), h2.data_ptr(), D, quant ? nullptr : x.data_ptr(),
      quant ? static_cast<uint8_t*>(x.data_ptr()) : nullptr, quant ? static_cast<float*>(scales.data_ptr()) : nullptr,
      stream_of(dev));
  if (st) return status(st);
  return quant ? give({h2, x, scales}) : give({h2, x});
}

// moe(x, router, w13, w13_scales, w2, w2_scales, bias or None, top_k, score, renorm, route_scale)
PyObject* moe(PyObject* const* a) {
  const Tensor *x = tensor(a[0]), *router = tensor(a[1]), *w13 = tensor(a[2]), *s13 = tensor(a[3]), *w2 = tensor(a[4]),
               *s2 = tensor(a[5]), *bias = tensor(a[6]);
  const int dev = device_of(x);
  if (dev < 0 || !dense(x, kBf16, dev, 2) || !router || !is_real(router->scalar_type()) ||
      !dense(router, router->scalar_type(), dev, 2) || !dense(w13, kFp8, dev, 3) || !dense(s13, kF32, dev, 3) ||
      !dense(w2, kFp8, dev, 3) || !dense(s2, kF32, dev, 3) || (bias ? !dense(bias, kF32, dev, 1) : a[6] != Py_None))
    return none();
  const int64_t T = x->size(0), D = x->size(1), E = router->size(0), n = w13->size(0), F = w13->size(1) / 2;
  if (T < 1 || router->size(1) != D || w13->size(1) != 2 * F || w13->size(2) != D || s13->size(0) != n ||
      s13->size(1) != blocks(2 * F) || s13->size(2) != blocks(D) || w2->size(0) != n || w2->size(1) != D ||
      w2->size(2) != F || s2->size(0) != n || s2->size(1) != blocks(D) || s2->size(2) != blocks(F) || n < E ||
      (bias && bias->size(0) != E) || T > BILOCO_MOE_MAX_T || D > BILOCO_MOE_MAX_D || F > BILOCO_MOE_MAX_F ||
      E > BILOCO_MOE_MAX_E || n - E > BILOCO_MOE_MAX_SHARED)
    return none();
  const long k = PyLong_AsLong(a[7]), score = PyLong_AsLong(a[8]);
  const double scale = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  if (k < 1 || k > E || k > BILOCO_MOE_MAX_K) return none();
  const int t = static_cast<int>(T), d = static_cast<int>(D), f = static_cast<int>(F), sh = static_cast<int>(n - E);
  const size_t need = biloco_fp8_moe_workspace_bytes(t, d, f, static_cast<int>(k), sh);
  if (!need) return none();
  Tensor y = make({T, D}, kBf16, dev), ids = make({T, k}, ScalarType::Int, dev), w = make({T, k}, kF32, dev),
         ws = make({static_cast<int64_t>(need)}, ScalarType::Byte, dev);
  const int st = biloco_fp8_moe(
      x->data_ptr(), D, router->data_ptr(), type_code(router->scalar_type()),
      bias ? static_cast<const float*>(bias->data_ptr()) : nullptr, static_cast<const uint8_t*>(w13->data_ptr()),
      static_cast<const float*>(s13->data_ptr()), static_cast<const uint8_t*>(w2->data_ptr()),
      static_cast<const float*>(s2->data_ptr()), t, d, f, static_cast<int>(E), static_cast<int>(k), sh,
      static_cast<int>(score), a[9] == Py_True, static_cast<float>(scale), y.data_ptr(), static_cast<int*>(ids.data_ptr()),
      static_cast<float*>(w.data_ptr()), ws.data_ptr(), need, stream_of(dev));
  return st ? status(st) : give({y, ids, w});
}

// C++ exceptions (out of memory, a CUDA error) become Python ones, torch's own kind among them.
template <Py_ssize_t kArgs, typename Fn>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, Fn fn) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  HANDLE_TH_ERRORS
  return fn(args);
  END_HANDLE_TH_ERRORS
}

PyObject* py_quant_act(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded<1>(args, n, [](PyObject* const* a) { return quant_act(tensor(a[0])); });
}
PyObject* py_gemm(PyObject*, PyObject* const* args, Py_ssize_t n) { return guarded<6>(args, n, gemm); }
PyObject* py_norm(PyObject*, PyObject* const* args, Py_ssize_t n) { return guarded<9>(args, n, norm); }
PyObject* py_moe(PyObject*, PyObject* const* args, Py_ssize_t n) { return guarded<11>(args, n, moe); }

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {{"quant_act", fast(py_quant_act), METH_FASTCALL, nullptr},
                          {"gemm", fast(py_gemm), METH_FASTCALL, nullptr},
                          {"norm", fast(py_norm), METH_FASTCALL, nullptr},
                          {"moe", fast(py_moe), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* m = PyModule_Create(&kModule);
  // the PyTorch whose headers this was compiled against: its tensors' layout is no other's
  if (m && PyModule_AddStringConstant(m, "torch_version", BILOCO_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
