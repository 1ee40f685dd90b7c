// torch_calls.cpp -- the Python binding's calls of the int8 and gated entry points
// (include/bq.h) on torch tensors: checks, output tensors, the library call.
//
// They are the calls of a decode step, where the host bounds the rate: the launch
// itself takes 2.1 us, and the same work through ctypes and torch's Python functions
// took another 7 (1.5 an output, 1 for the argument conversion, 3 for the checks).
// The functions take every argument by position; None stands for what is left out.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <stdexcept>
#include <string>

#include "bq.h"

namespace {

using at::ScalarType;
using at::Tensor;
using Wide = __int128;  // element counts of the callers' numbers, without overflow

PyObject *g_error = nullptr;  // the binding's BqError

// The library's functions, by the addresses that the binding loaded.
struct Library {
  decltype(&bq_act_quant_int8) act_quant_int8;
  decltype(&bq_gemm_int8_int8_epilogue) gemm_int8_int8;
  decltype(&bq_gemm_gated) gemm_gated;
  decltype(&bq_gated_grad_quant) gated_grad_quant;
} g_lib;

// An argument error, or (raised) one that Python already holds.
struct Refusal : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Raised {};

// A tensor argument, or nullptr for None.
const Tensor *tensor(PyObject *o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor");
    throw Raised{};
  }
  return &THPVariable_Unpack(o);
}

// One that may not be left out.
const Tensor &need_tensor(PyObject *o) {
  const Tensor *t = tensor(o);
  if (!t) {
    PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor, not None");
    throw Raised{};
  }
  return *t;
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// The calls run on the current stream of the current device, where their tensors live.
struct Here {
  int device = -1;
  void on(const Tensor *t) {
    if (!t) return;
    if (!t->is_cuda()) throw Refusal("libbq works on CUDA tensors only");
    if (device < 0) device = c10::cuda::current_device();
    if (t->get_device() != device) throw Refusal("tensors must be on the current CUDA device");
  }
  void on(const Tensor &t) { on(&t); }
  bq_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
  Tensor empty(at::IntArrayRef size, ScalarType type) const {
    return Tensor(at::detail::empty_cuda(
        size, type, at::Device(at::kCUDA, static_cast<at::DeviceIndex>(device)), std::nullopt));
  }
};

const char *type_name(ScalarType t) {
  return t == at::kChar       ? "torch.int8"
         : t == at::kByte     ? "torch.uint8"
         : t == at::kBFloat16 ? "torch.bfloat16"
                              : "torch.float32";
}

void need(const Tensor &t, ScalarType type, Wide count, const char *what) {
  if (t.scalar_type() != type || t.numel() < count || !t.is_contiguous())
    throw Refusal(std::string(what) + " must be a contiguous " + type_name(type) +
                  " tensor of at least " +
                  std::to_string(static_cast<long long>(std::min<Wide>(count, INT64_MAX))) +
                  " elements");
}

// The word that a quantizer reports a NaN or Inf in.
void need_status(const Tensor *t) {
  if (t && (t->scalar_type() != at::kInt || t->numel() < 1))
    throw Refusal("status must be a torch.int32 tensor of at least 1 element");
}

// bf16 [rows, cols] with unit column stride (the row stride may exceed cols).
void need_rows(const Tensor &t, int64_t rows, int64_t cols, const char *what) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || t.size(0) != rows ||
      t.size(1) != cols || (cols > 1 && t.stride(1) != 1))
    throw Refusal(std::string(what) + " must be a bf16 [" + std::to_string(rows) + ", " +
                  std::to_string(cols) + "] tensor with unit column stride");
}

// Row stride of a tensor's last two dimensions (one row has none of its own).
int64_t row_stride(const Tensor &t) {
  return t.size(-2) > 1 ? t.stride(-2) : std::max(t.stride(-2), t.size(-1));
}

// bf16 rows of unit column stride for a batch whose last problem begins
// `last` elements behind the first: the strides are the
// caller's, so what counts is what the storage holds.
void need_batch_rows(const Tensor &t, int64_t rows, int64_t cols, Wide last, const char *what) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() < 2 || t.size(-2) < rows || t.size(-1) < cols ||
      (cols > 1 && t.stride(-1) != 1))
    throw Refusal(std::string(what) + " must be bf16 [.., " + std::to_string(rows) + ", " +
                  std::to_string(cols) + "] with unit column stride");
  const Wide held = Wide(t.storage().nbytes() / t.element_size()) - t.storage_offset();
  if (rows > 0 && cols > 0 && last + Wide(rows - 1) * row_stride(t) + cols > held)
    throw Refusal(std::string(what) + " does not reach the last problem's last row");
}

void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
void *ptr(const Tensor &t) { return t.data_ptr(); }

// A given output, checked, or a new one.
template <class F>
Tensor output(const Tensor *given, ScalarType type, Wide count, const char *what, F make) {
  if (!given) return make();
  need(*given, type, count, what);
  return *given;
}

// The library's call, without the interpreter lock; its status as the binding's error.
template <class F>
void call(const char *name, F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  if (st == BQ_OK) return;
  PyObject *e = PyObject_CallFunction(g_error, "is", st, name);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// The results as a tuple; an undefined tensor is None.
PyObject *tuple(std::initializer_list<Tensor> ts) {
  PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const Tensor &t : ts) {
    PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Nothing leaves as a C++ exception: refusals are ValueErrors, torch's own errors
// (an allocation that failed) what torch makes of them.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Raised &) {
    return nullptr;
  } catch (const Refusal &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (x, q, scale, status) -> (q, scale)
PyObject *act_quant_int8(PyObject *const *a) {
  const Tensor &x = need_tensor(a[0]);
  const Tensor *q_in = tensor(a[1]), *scale_in = tensor(a[2]), *status = tensor(a[3]);
  need_status(status);
  Here here;
  here.on(x);
  here.on(q_in);
  here.on(scale_in);
  here.on(status);
  if (x.scalar_type() != at::kBFloat16 || x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
    throw Refusal("x must be a bf16 [M, K] tensor with unit column stride");
  const int64_t M = x.size(0), K = x.size(1);
  Tensor q = output(q_in, at::kChar, Wide(M) * K, "q", [&] { return here.empty({M, K}, at::kChar); });
  Tensor scale =
      output(scale_in, at::kFloat, M, "scale", [&] { return here.empty({M}, at::kFloat); });
  const bq_stream_t stream = here.stream();
  call("bq_act_quant_int8", [&] {
    return g_lib.act_quant_int8(ptr(x), M, K, row_stride(x), ptr(q),
                                static_cast<float *>(ptr(scale)), static_cast<int *>(ptr(status)),
                                stream);
  });
  return tuple({q, scale});
}

// (a_q, a_scale, b, b_scale, M, N, K, y, bias, residual, alpha, act, batch, config) -> y;
// batch: the seven numbers of bq_batch, config: the address of a bq_gemm_config
PyObject *gemm_int8_int8(PyObject *const *a) {
  const Tensor &aq = need_tensor(a[0]), &as = need_tensor(a[1]), &b = need_tensor(a[2]),
               &bs = need_tensor(a[3]);
  const int64_t M = integer(a[4]), N = integer(a[5]), K = integer(a[6]);
  const Tensor *y_in = tensor(a[7]), *bias = tensor(a[8]), *res = tensor(a[9]);
  bq_epilogue epi = {};
  epi.alpha = static_cast<float>(number(a[10]));
  epi.act = static_cast<int>(integer(a[11]));
  bq_batch batch = {1, 0, 0, 0, 0, 0, 0};
  const bool batched = a[12] != Py_None;
  if (batched) {
    int64_t *field[7] = {&batch.count,       &batch.stride_a, &batch.stride_a_sf, &batch.stride_b,
                         &batch.stride_b_sf, &batch.stride_y, &batch.stride_res};
    for (int i = 0; i < 7; ++i) {
      PyObject *o = PyTuple_GetItem(a[12], i);
      if (!o) throw Raised{};
      *field[i] = integer(o);
    }
  }
  const bq_gemm_config *config = nullptr;
  if (a[13] != Py_None)
    config = reinterpret_cast<const bq_gemm_config *>(static_cast<intptr_t>(integer(a[13])));
  const Wide more = M && N ? std::max<int64_t>(batch.count - 1, 0) : 0;
  need(aq, at::kChar, Wide(M) * K + more * batch.stride_a, "a_q");
  need(b, at::kChar, Wide(N) * K + more * batch.stride_b, "b");
  need(as, at::kFloat, M + more * (batch.stride_a_sf / 4), "a_scale");
  need(bs, at::kFloat, N + more * (batch.stride_b_sf / 4), "b_scale");
  if (bias) {
    need(*bias, at::kBFloat16, N, "bias");
    epi.bias = ptr(bias);
  }
  if (res) {
    if (batched)
      need_batch_rows(*res, M, N, more * (batch.stride_res / 2), "residual");
    else
      need_rows(*res, M, N, "residual");
    epi.ld_residual = row_stride(*res);
    epi.residual = ptr(res);
  }
  if (!y_in && more > 0 && Wide(batch.stride_y) > Wide(M) * N * 2)
    throw Refusal("a batch with gaps between its outputs (stride_y) needs y");
  Here here;
  for (const Tensor *t : {&aq, &as, &b, &bs, y_in, bias, res}) here.on(t);
  Tensor y = output(y_in, at::kBFloat16, Wide(M) * N + more * (batch.stride_y / 2), "y", [&] {
    return M < 0 || N < 0 || batch.count < 0 ? Tensor()  // refused below
           : batched                         ? here.empty({batch.count, M, N}, at::kBFloat16)
                                             : here.empty({M, N}, at::kBFloat16);
  });
  const bq_stream_t stream = here.stream();
  call("bq_gemm_int8_int8_epilogue", [&] {
    return g_lib.gemm_int8_int8(ptr(aq), static_cast<float *>(ptr(as)), ptr(b),
                                static_cast<float *>(ptr(bs)), M, N, K,
                                y.defined() ? ptr(y) : nullptr, &epi, &batch, config, stream);
  });
  return THPVariable_Wrap(y);
}

// (weight_kind, a_q, a_sf, b_gate, gate_sf, b_up, up_sf, M, N, K, y, act, alpha,
// keep_projections, gu, quantize_out, write_y, q_out, sf_out, config) -> (y, q, sf, gu)
PyObject *gemm_gated(PyObject *const *a) {
  const int64_t kind = integer(a[0]);
  const Tensor &aq = need_tensor(a[1]), &as = need_tensor(a[2]), &wg = need_tensor(a[3]),
               &sg = need_tensor(a[4]), &wu = need_tensor(a[5]), &su = need_tensor(a[6]);
  const int64_t M = integer(a[7]), N = integer(a[8]), K = integer(a[9]);
  const Tensor *y_in = tensor(a[10]), *gu_in = tensor(a[14]), *q_in = tensor(a[17]),
               *sf_in = tensor(a[18]);
  bq_gated_epilogue epi = {};
  epi.act = static_cast<int>(integer(a[11]));
  epi.alpha = static_cast<float>(number(a[12]));
  const bool keep = truth(a[13]), quantize = truth(a[15]), write = truth(a[16]);
  Here here;
  for (const Tensor *t : {&aq, &as, &wg, &sg, &wu, &su, y_in, gu_in, q_in, sf_in}) here.on(t);
  if (!write && !quantize) throw Refusal("write_y=False needs quantize_out=True");
  const bq_gemm_config *config = nullptr;
  if (a[19] != Py_None)
    config = reinterpret_cast<const bq_gemm_config *>(static_cast<intptr_t>(integer(a[19])));
  auto bands = [](int64_t n) { return (Wide(n) + 127) / 128; };
  const bool i8 = kind == 6;
  const ScalarType code = i8 ? at::kChar : at::kByte, scale = i8 ? at::kFloat : at::kByte;
  const Wide na = i8 ? Wide(M) : bands(M) * bands(K) * 512,
             ns = i8 ? Wide(N) : bands(N) * bands(K) * 512,
             nw = Wide(N) * K / (kind == 0 ? 2 : 1), mn = Wide(M) * N;
  need(aq, code, Wide(M) * K, "a_q");
  need(as, scale, na, "a_sf");
  need(wg, code, nw, "b_gate");
  need(sg, scale, ns, "gate_sf");
  need(wu, code, nw, "b_up");
  need(su, scale, ns, "up_sf");
  const bool sizes = M >= 0 && N >= 0;  // else refused by the library
  auto fresh = [&](std::initializer_list<int64_t> size, ScalarType type) {
    return sizes ? here.empty(at::IntArrayRef(size), type) : Tensor();
  };
  Tensor y, gu, q, sf;
  if (write)
    y = output(y_in, at::kBFloat16, mn, "y", [&] { return fresh({M, N}, at::kBFloat16); });
  if (gu_in || keep)
    gu = output(gu_in, at::kBFloat16, 2 * mn, "gu",
                [&] { return fresh({M, 2 * N}, at::kBFloat16); });
  if (quantize) {
    const int64_t nsf = sizes ? static_cast<int64_t>(bands(M) * bands(N) * 512) : 0;
    q = output(q_in, at::kByte, mn, "q_out", [&] { return fresh({M, N}, at::kByte); });
    sf = output(sf_in, at::kByte, nsf, "sf_out",
                [&] { return fresh({std::max<int64_t>(nsf, 1)}, at::kByte); });
  }
  auto at_of = [](const Tensor &t) { return t.defined() ? ptr(t) : nullptr; };
  epi.gu_out = at_of(gu);
  epi.q_out = at_of(q);
  epi.sf_out = at_of(sf);
  const bq_stream_t stream = here.stream();
  call("bq_gemm_gated", [&] {
    return g_lib.gemm_gated(static_cast<int>(kind), ptr(aq), ptr(as), ptr(wg), ptr(sg), ptr(wu),
                            ptr(su), M, N, K, at_of(y), &epi, config, stream);
  });
  return tuple({y, q, sf, gu});
}

// (dh, gu, act, rounding, seed, q_row, sf_row, q_t, sf_t, d, status)
// -> (q_row, sf_row, q_t, sf_t)
PyObject *gated_grad_quant(PyObject *const *a) {
  const Tensor &dh = need_tensor(a[0]), &gu = need_tensor(a[1]);
  const int act = static_cast<int>(integer(a[2])), rounding = static_cast<int>(integer(a[3]));
  const uint64_t seed = PyLong_AsUnsignedLongLongMask(a[4]);
  if (PyErr_Occurred()) throw Raised{};
  const Tensor *out[4] = {tensor(a[5]), tensor(a[6]), tensor(a[7]), tensor(a[8])};
  const Tensor *d = tensor(a[9]), *status = tensor(a[10]);
  need_status(status);
  Here here;
  here.on(dh);
  here.on(gu);
  for (const Tensor *t : out) here.on(t);
  here.on(d);
  here.on(status);
  if (dh.dim() != 2) throw Refusal("dh must be a bf16 [M, N] tensor");
  const int64_t M = dh.size(0), N = dh.size(1);
  need_rows(dh, M, N, "dh");
  need_rows(gu, M, 2 * N, "gu");
  // both scale buffers have as many atoms
  const int64_t nsf = std::max<int64_t>((M + 127) / 128 * ((2 * N + 127) / 128) * 512, 1);
  auto bytes = [&](std::initializer_list<int64_t> size) {
    return here.empty(at::IntArrayRef(size), at::kByte);
  };
  const Wide count = Wide(2) * M * N;
  Tensor q_row = output(out[0], at::kByte, count, "q_row", [&] { return bytes({M, 2 * N}); });
  Tensor sf_row = output(out[1], at::kByte, nsf, "sf_row", [&] { return bytes({nsf}); });
  Tensor q_t = output(out[2], at::kByte, count, "q_t", [&] { return bytes({2 * N, M}); });
  Tensor sf_t = output(out[3], at::kByte, nsf, "sf_t", [&] { return bytes({nsf}); });
  if (d) need(*d, at::kBFloat16, count, "d");
  const bq_stream_t stream = here.stream();
  call("bq_gated_grad_quant", [&] {
    return g_lib.gated_grad_quant(ptr(dh), row_stride(dh), ptr(gu), row_stride(gu), M, N, act,
                                  rounding, seed, ptr(q_row), ptr(sf_row), ptr(q_t), ptr(sf_t),
                                  ptr(d), static_cast<int *>(ptr(status)), stream);
  });
  return tuple({q_row, sf_row, q_t, sf_t});
}

// (BqError, addresses of the library's functions in Library's order)
PyObject *init(PyObject *const *a) {
  void *f[4];
  for (int i = 0; i < 4; ++i) {
    f[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) throw Raised{};
  }
  g_lib = {reinterpret_cast<decltype(g_lib.act_quant_int8)>(f[0]),
           reinterpret_cast<decltype(g_lib.gemm_int8_int8)>(f[1]),
           reinterpret_cast<decltype(g_lib.gemm_gated)>(f[2]),
           reinterpret_cast<decltype(g_lib.gated_grad_quant)>(f[3])};
  Py_XDECREF(g_error);
  g_error = Py_NewRef(a[0]);
  return Py_NewRef(Py_None);
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<init, 5>("init"),
    method<act_quant_int8, 4>("act_quant_int8"),
    method<gemm_int8_int8, 14>("gemm_int8_int8"),
    method<gemm_gated, 20>("gemm_gated"),
    method<gated_grad_quant, 11>("gated_grad_quant"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
