// binding.cpp -- the torch side of the routing and adapter operators: tensors
// to wqmm_tensor descriptors, outputs and workspaces from torch's allocator,
// both phases on the current stream.  Marshalling only; every check of shapes
// and dtypes is phase 1's.
//
// It is compiled because a call at a few tokens is bound by the host: through
// ctypes a combine of 16 tokens took 12 us of host time for 2 us of GPU time.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/wqmm.h"

namespace {

PyObject* g_error = nullptr;  // WqmmError

struct Failed {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const char* msg) {
  PyErr_SetString(type, msg);
  throw Failed();
}

void check(wqmm_status st) {
  if (st == WQMM_SUCCESS) return;
  PyObject* args = Py_BuildValue("(is)", static_cast<int>(st), wqmm_last_error());
  if (args) {
    PyErr_SetObject(g_error, args);
    Py_DECREF(args);
  }
  throw Failed();
}

int code(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return WQMM_DT_F16;
    case at::kBFloat16: return WQMM_DT_BF16;
    case at::kFloat: return WQMM_DT_F32;
    case at::kChar: return WQMM_DT_I8;
    case at::kInt: return WQMM_DT_I32;
    case at::kFloat8_e4m3fn: return WQMM_DT_FP8E4M3;
    case at::kLong: return WQMM_DT_I64;
    default: raise(PyExc_TypeError, "no wqmm dtype for this tensor's dtype");
  }
}

// A tensor argument; None where `optional`.
const at::Tensor* tensor(PyObject* o, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "a torch tensor is expected");
  return &THPVariable_Unpack(o);
}

bool truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw Failed();
  return t == 1;
}

struct Desc {
  wqmm_tensor d{};
  const wqmm_tensor* p = nullptr;
  explicit Desc(const at::Tensor* t) {
    if (!t) return;
    const int64_t nd = t->dim();
    if (nd < 1 || nd > 3) raise(PyExc_ValueError, "a tensor of 1 to 3 dimensions is expected");
    d.data = t->data_ptr();
    d.dtype = code(t->scalar_type());
    d.ndim = static_cast<int32_t>(nd);
    for (int64_t i = 0; i < nd; ++i) {
      d.shape[i] = t->size(i);
      d.strides[i] = t->stride(i);
    }
    d.format = WQMM_FORMAT_ND;
    p = &d;
  }
  explicit Desc(const at::Tensor& t) : Desc(&t) {}
  operator const wqmm_tensor*() const { return p; }
};

// The one CUDA device of all tensors given, made current for the call.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(std::initializer_list<const at::Tensor*> ts) {
    int dev = -1;
    for (const at::Tensor* t : ts) {
      if (!t) continue;
      if (!t->is_cuda()) raise(PyExc_ValueError, "every tensor must be a CUDA tensor");
      const int d = t->device().index();
      if (dev >= 0 && d != dev) raise(PyExc_ValueError, "tensors of two devices: one device is expected");
      dev = d;
    }
    guard.set_index(dev);
  }
};

// A contiguous tensor beside `like`, straight from the allocator (0.3 us less of the host than by at::empty).
at::Tensor make(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
at::Tensor make(at::IntArrayRef shape, const at::Tensor& like) { return make(shape, like, like.scalar_type()); }

using Run = wqmm_status (*)(void*, uint64_t, wqmm_executor*, wqmm_stream);

// The workspace and phase 2 of an executor phase 1 has handed out.
void finish(wqmm_status st, uint64_t size, wqmm_executor* ex, Run run, const at::Tensor& like) {
  check(st);
  at::Tensor space;
  if (size) {
    try {
      space = make({static_cast<int64_t>(size)}, like, at::kByte);
    } catch (...) {
      wqmm_executor_destroy(ex);
      throw;
    }
  }
  const cudaStream_t s = c10::cuda::getCurrentCUDAStream().stream();
  check(run(size ? space.data_ptr() : nullptr, size, ex, reinterpret_cast<wqmm_stream>(s)));
}


void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
}

#define BEGIN \
  HANDLE_TH_ERRORS try {
#define END          \
  }                  \
  catch (Failed&) {  \
    return nullptr;  \
  }                  \
  END_HANDLE_TH_ERRORS

// (expert_ids, num_experts) -> (offsets, source, position)
PyObject* sort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN count(n, 2);
  const at::Tensor* ids = tensor(a[0]);
  const int64_t experts = PyLong_AsLongLong(a[1]);
  if (experts == -1 && PyErr_Occurred()) throw Failed();
  OnDevice on({ids});
  at::Tensor offsets = make({experts < 0 ? 1 : experts < 65536 ? experts + 1 : 1}, *ids, at::kInt);
  at::Tensor source = make({ids->numel()}, *ids, at::kInt), position = make(ids->sizes(), *ids, at::kInt);
  uint64_t size = 0;
  wqmm_executor* ex = nullptr;
  const wqmm_status st = route_sort_get_workspace_size(Desc(ids), experts, Desc(offsets), Desc(source), Desc(position),
                                                       &size, &ex);
  finish(st, size, ex, route_run, *ids);
  return Py_BuildValue("(NNN)", THPVariable_Wrap(offsets), THPVariable_Wrap(source), THPVariable_Wrap(position));
  END
}

// (x, position, out) -> out
PyObject* dispatch_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN count(n, 3);
  const at::Tensor *x = tensor(a[0]), *position = tensor(a[1]), *given = tensor(a[2], true);
  OnDevice on({x, position, given});
  if (x->dim() < 1) raise(PyExc_ValueError, "x must be (T, hidden) or (b, s, hidden)");
  at::Tensor out = given ? *given : make({position->numel(), x->size(-1)}, *x);
  uint64_t size = 0;
  wqmm_executor* ex = nullptr;
  const wqmm_status st = route_dispatch_get_workspace_size(Desc(x), Desc(position), Desc(out), &size, &ex);
  finish(st, size, ex, route_run, *x);
  return THPVariable_Wrap(out);
  END
}

// (x_sorted, position, weights, x3, out) -> out
PyObject* combine_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN count(n, 5);
  const at::Tensor *xs = tensor(a[0]), *position = tensor(a[1]), *weights = tensor(a[2], true),
                   *x3 = tensor(a[3], true), *given = tensor(a[4], true);
  OnDevice on({xs, position, weights, x3, given});
  at::Tensor out;
  if (given) {
    out = *given;
  } else if (x3) {
    out = make(x3->sizes(), *xs);
  } else {
    if (xs->dim() != 2 || position->dim() < 1) raise(PyExc_ValueError, "x_sorted must be (rows, hidden), position (T, K)");
    auto shape = position->sizes().vec();
    if (shape.size() > 1) shape.pop_back();
    shape.push_back(xs->size(1));
    out = make(shape, *xs);
  }
  uint64_t size = 0;
  wqmm_executor* ex = nullptr;
  const wqmm_status st = route_combine_get_workspace_size(Desc(xs), Desc(position), Desc(weights), Desc(x3), Desc(out),
                                                          &size, &ex);
  finish(st, size, ex, route_run, *xs);
  return THPVariable_Wrap(out);
  END
}

// (grad, x_sorted, position, weights, out) -> (grad_sorted, grad_weights)
PyObject* combine_tokens_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN count(n, 5);
  const at::Tensor *grad = tensor(a[0]), *xs = tensor(a[1]), *position = tensor(a[2]), *weights = tensor(a[3]),
                   *given = tensor(a[4], true);
  OnDevice on({grad, xs, position, weights, given});
  at::Tensor out = given ? *given : make(xs->sizes(), *xs), gw = make(weights->sizes(), *weights);
  uint64_t size = 0;
  wqmm_executor* ex = nullptr;
  const wqmm_status st = route_combine_grad_get_workspace_size(Desc(grad), Desc(xs), Desc(position), Desc(weights),
                                                               Desc(out), Desc(gw), &size, &ex);
  finish(st, size, ex, route_run, *xs);
  return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(gw));
  END
}

// (x1, lora_a, lora_b, scale, offsets, source, y, out) -> out
PyObject* lora_add(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN count(n, 8);
  const at::Tensor *x = tensor(a[0]), *la = tensor(a[1]), *lb = tensor(a[2]), *scale = tensor(a[3], true),
                   *offsets = tensor(a[4]), *source = tensor(a[5]), *y = tensor(a[6], true), *given = tensor(a[7], true);
  OnDevice on({x, la, lb, scale, offsets, source, y, given});
  at::Tensor out;
  if (given) {
    out = *given;
  } else {
    if (x->dim() < 1 || lb->dim() != 3) raise(PyExc_ValueError, "x1 must be (m, k) or (b, s, k), lora_b (adapters, n, rank)");
    auto shape = x->sizes().vec();
    shape.back() = lb->size(1);
    out = make(shape, *x);
  }
  uint64_t size = 0;
  wqmm_executor* ex = nullptr;
  const wqmm_status st = lora_get_workspace_size(Desc(x), Desc(la), Desc(lb), Desc(scale), Desc(offsets), Desc(source),
                                                 Desc(y), Desc(out), &size, &ex);
  finish(st, size, ex, lora_run, *x);
  return THPVariable_Wrap(out);
  END
}

// (x1, lora_a, lora_b, scale, offsets, source, y, out) -> None: what lora_add would refuse of its arguments is refused
PyObject* check_lora_add(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN count(n, 8);
  const at::Tensor *x = tensor(a[0]), *la = tensor(a[1]), *lb = tensor(a[2]), *scale = tensor(a[3], true),
                   *offsets = tensor(a[4]), *source = tensor(a[5]), *y = tensor(a[6], true), *out = tensor(a[7]);
  uint64_t size = 0;
  wqmm_executor* ex = nullptr;
  check(lora_get_workspace_size(Desc(x), Desc(la), Desc(lb), Desc(scale), Desc(offsets), Desc(source), Desc(y),
                                Desc(out), &size, &ex));
  wqmm_executor_destroy(ex);
  Py_RETURN_NONE;
  END
}

// (grad, x1, lora_a, lora_b, scale, offsets, source, grad_x_in, need_grad_x, in_place) -> (grad_x, grad_a, grad_b)
PyObject* lora_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  BEGIN count(n, 10);
  const at::Tensor *grad = tensor(a[0]), *x = tensor(a[1]), *la = tensor(a[2]), *lb = tensor(a[3]),
                   *scale = tensor(a[4], true), *offsets = tensor(a[5]), *source = tensor(a[6]),
                   *gx_in = tensor(a[7], true);
  const bool need = truth(a[8]), in_place = truth(a[9]);
  OnDevice on({grad, x, la, lb, scale, offsets, source, gx_in});
  at::Tensor gx, ga = make(la->sizes(), *la), gb = make(lb->sizes(), *lb);
  if (need) gx = in_place && gx_in ? *gx_in : make(x->sizes(), *x);
  uint64_t size = 0;
  wqmm_executor* ex = nullptr;
  const wqmm_status st = lora_grad_get_workspace_size(Desc(grad), Desc(x), Desc(la), Desc(lb), Desc(scale),
                                                      Desc(offsets), Desc(source), Desc(gx_in),
                                                      Desc(need ? &gx : nullptr), Desc(ga), Desc(gb), &size, &ex);
  finish(st, size, ex, lora_run, *x);
  PyObject* first = need ? THPVariable_Wrap(gx) : Py_NewRef(Py_None);
  return Py_BuildValue("(NNN)", first, THPVariable_Wrap(ga), THPVariable_Wrap(gb));
  END
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(sort_tokens),         METHOD(dispatch_tokens), METHOD(combine_tokens),
                           METHOD(combine_tokens_grad), METHOD(lora_add),        METHOD(check_lora_add),
                           METHOD(lora_grad),           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* package = PyImport_ImportModule("weight_quantized_gemm_anti_b200");
  if (!package) return nullptr;
  g_error = PyObject_GetAttrString(package, "WqmmError");
  Py_DECREF(package);
  return g_error ? PyModule_Create(&g_module) : nullptr;
}
