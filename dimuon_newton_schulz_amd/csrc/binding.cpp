// Marshalling of the experts' calls without the interpreter: a short call's
// host time is the reading of its tensors' shapes, strides and addresses,
// 7 to 10 us in Python and well below 1 us here.
//
// Each function takes the ordinary case only: every tensor of the expected
// shape and dtype on the current GPU, rows' elements consecutive, the launch
// on the current stream.  For anything else it returns None, and the Python
// function of the same name goes on (it says what is wrong, or makes the
// call).  A failing status comes back as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "muon_mi355x.h"

namespace {

decltype(&expert_sort) f_sort = nullptr;
decltype(&expert_gather) f_gather = nullptr;
decltype(&expert_combine) f_combine = nullptr;
decltype(&expert_combine_grad) f_combine_grad = nullptr;
decltype(&linear_forward) f_linear = nullptr;
decltype(&linear_grad_workspace_bytes) f_grad_bytes = nullptr;
decltype(&linear_grad) f_grad = nullptr;

constexpr int64_t kSortAlone = 8192, kMaxExperts = 1024, kMaxStride = int64_t{1} << 20;

// The GPU that is current (-1: none), and whether a tensor argument lies on it.
int current_gpu() {
  int d = -1;
  return hipGetDevice(&d) == hipSuccess ? d : -1;
}

// A tensor on GPU `gpu`, or NULL.
const at::Tensor* tensor_on(PyObject* o, int gpu) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.get_device() == gpu ? &t : nullptr;
}

int dtype_of(const at::Tensor& t) {
  const auto s = t.scalar_type();
  return s == at::kFloat ? MUON_F32 : s == at::kBFloat16 ? MUON_BF16 : -1;
}

// Row stride of a rows x columns tensor of that dtype; -1: not the ordinary case.
int64_t row_stride(const at::Tensor* t, int64_t rows, int64_t columns, int dtype) {
  if (!t || t->dim() != 2 || t->size(0) != rows || t->size(1) != columns || dtype_of(*t) != dtype) return -1;
  const int64_t ld = t->stride(0);
  return t->stride(1) == 1 && ld >= columns && ld <= kMaxStride ? ld : -1;
}

bool ints(const at::Tensor* t, int64_t n) {
  return t && t->scalar_type() == at::kInt && t->numel() == n && t->is_contiguous();
}

void* stream_of(int gpu) { return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(gpu)).stream(); }

// The routes' tensors (offsets, order, place).
bool routes_of(PyObject* const* a, int gpu, expert_routes_t& r) {
  const at::Tensor *offsets = tensor_on(a[0], gpu), *order = tensor_on(a[1], gpu), *place = tensor_on(a[2], gpu);
  if (!place || place->dim() != 2 || !ints(place, place->numel()) || place->size(1) < 1) return false;
  if (!ints(order, place->numel()) || order->dim() != 1 || !offsets || offsets->dim() != 1 || offsets->numel() < 2 ||
      offsets->numel() > kMaxExperts + 1 || !ints(offsets, offsets->numel()) || place->size(1) > INT32_MAX)
    return false;
  r = {static_cast<int32_t*>(offsets->data_ptr()), static_cast<int32_t*>(order->data_ptr()),
       static_cast<int32_t*>(place->data_ptr()), place->size(0), static_cast<int32_t>(place->size(1)),
       static_cast<int32_t>(offsets->numel() - 1)};
  return true;
}

// Whether autograd would have to record a call on one of these arguments.
bool recorded(PyObject* const* a, Py_ssize_t n) {
  if (!c10::GradMode::is_enabled()) return false;
  for (Py_ssize_t i = 0; i < n; ++i)
    if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad()) return true;
  return false;
}

#define MUON_ORDINARY(cond) \
  do {                      \
    if (!(cond)) Py_RETURN_NONE; \
  } while (0)

template <typename F>
muon_status_t released(F&& f) {
  muon_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// The given output (a new reference), or a new tensor; `out` is set to it.
PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}

PyObject* py_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int gpu = current_gpu();
  MUON_ORDINARY(n == 2 && f_sort && PyLong_Check(a[1]));
  const at::Tensor* ids = tensor_on(a[0], gpu);
  const int64_t experts = PyLong_AsLongLong(a[1]);
  if (experts == -1 && PyErr_Occurred()) PyErr_Clear();
  MUON_ORDINARY(ids && ids->dim() == 2 && ids->is_contiguous() && experts >= 1 && experts <= kMaxExperts);
  const bool wide = ids->scalar_type() == at::kLong;
  const int64_t slots = ids->numel();
  MUON_ORDINARY((wide || ids->scalar_type() == at::kInt) && ids->size(1) >= 1 && slots <= kSortAlone);
  const at::Tensor flat = at::empty({experts + 1 + 2 * slots}, ids->options().dtype(at::kInt));
  // (Views of one allocation, made directly: narrow() costs three times as much.)
  const auto piece = [&](int64_t at, at::IntArrayRef sizes) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(flat.storage()), flat.key_set(), flat.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    return t;
  };
  const at::Tensor offsets = piece(0, {experts + 1}), order = piece(experts + 1, {slots});
  const at::Tensor place = piece(experts + 1 + slots, {ids->size(0), ids->size(1)});
  int32_t* p = static_cast<int32_t*>(flat.data_ptr());
  const expert_routes_t r{p, p + experts + 1, p + experts + 1 + slots, ids->size(0), static_cast<int32_t>(ids->size(1)),
                          static_cast<int32_t>(experts)};
  const void* from = ids->data_ptr();
  void* s = stream_of(gpu);
  const muon_status_t st = released([&] { return f_sort(from, wide ? 8 : 4, &r, nullptr, 0, s); });
  if (st != MUON_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(NNN)", THPVariable_Wrap(offsets), THPVariable_Wrap(order), THPVariable_Wrap(place));
  END_HANDLE_TH_ERRORS
}

// x, offsets, order, place, out or None
PyObject* py_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int gpu = current_gpu();
  expert_routes_t r;
  MUON_ORDINARY(n == 5 && f_gather && !recorded(a, n) && routes_of(a + 1, gpu, r));
  const at::Tensor* x = tensor_on(a[0], gpu);
  MUON_ORDINARY(x && x->dim() == 2 && dtype_of(*x) >= 0);
  const int64_t width = x->size(1), slots = r.tokens * r.top;
  const int dt = dtype_of(*x);
  const int64_t ld = row_stride(x, r.tokens, width, dt);
  MUON_ORDINARY(ld >= 0);
  PyObject* out = a[4] == Py_None ? THPVariable_Wrap(at::empty({slots, width}, x->options())) : given(a[4]);
  const at::Tensor* o = tensor_on(out, gpu);
  const int64_t ld_out = row_stride(o, slots, width, dt);
  if (ld_out < 0) {
    Py_DECREF(out);
    Py_RETURN_NONE;
  }
  const void* from = x->data_ptr();
  void *to = o->data_ptr(), *s = stream_of(gpu);
  const muon_status_t st =
      released([&] { return f_gather(from, ld, width, static_cast<muon_dtype_t>(dt), &r, to, ld_out, s); });
  if (st == MUON_OK) return out;
  Py_DECREF(out);
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// Weights (or their gradients) of every slot.
bool per_slot(const at::Tensor* t, const expert_routes_t& r, int& dt) {
  if (!t || t->dim() != 2 || t->size(0) != r.tokens || t->size(1) != r.top || !t->is_contiguous()) return false;
  dt = dtype_of(*t);
  return dt >= 0;
}

// ys, offsets, order, place, weights or None, residual or None, out or None
PyObject* py_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int gpu = current_gpu();
  expert_routes_t r;
  MUON_ORDINARY(n == 7 && f_combine && !recorded(a, n) && routes_of(a + 1, gpu, r));
  const at::Tensor* ys = tensor_on(a[0], gpu);
  MUON_ORDINARY(ys && ys->dim() == 2 && dtype_of(*ys) >= 0);
  const int64_t width = ys->size(1);
  const int dt = dtype_of(*ys);
  const int64_t ld = row_stride(ys, r.tokens * r.top, width, dt);
  MUON_ORDINARY(ld >= 0);
  const void *w = nullptr, *res = nullptr;
  int w_dt = MUON_F32;
  int64_t ld_res = 0;
  if (a[4] != Py_None) {
    const at::Tensor* t = tensor_on(a[4], gpu);
    MUON_ORDINARY(per_slot(t, r, w_dt));
    w = t->data_ptr();
  }
  if (a[5] != Py_None) {
    const at::Tensor* t = tensor_on(a[5], gpu);
    MUON_ORDINARY((ld_res = row_stride(t, r.tokens, width, dt)) >= 0);
    res = t->data_ptr();
  }
  PyObject* out = a[6] == Py_None ? THPVariable_Wrap(at::empty({r.tokens, width}, ys->options())) : given(a[6]);
  const at::Tensor* o = tensor_on(out, gpu);
  const int64_t ld_out = row_stride(o, r.tokens, width, dt);
  if (ld_out < 0) {
    Py_DECREF(out);
    Py_RETURN_NONE;
  }
  const void* from = ys->data_ptr();
  void *to = o->data_ptr(), *s = stream_of(gpu);
  const muon_status_t st = released([&] {
    return f_combine(from, ld, width, static_cast<muon_dtype_t>(dt), &r, w, static_cast<muon_dtype_t>(w_dt), res, ld_res,
                     to, ld_out, s);
  });
  if (st == MUON_OK) return out;
  Py_DECREF(out);
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// dy, ys, weights, offsets, order, place, dys, dweights
PyObject* py_combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int gpu = current_gpu();
  expert_routes_t r;
  MUON_ORDINARY(n == 8 && f_combine_grad && !recorded(a, 1) && routes_of(a + 3, gpu, r));
  const at::Tensor *dy = tensor_on(a[0], gpu), *ys = tensor_on(a[1], gpu), *w = tensor_on(a[2], gpu);
  const at::Tensor *dys = tensor_on(a[6], gpu), *dw = tensor_on(a[7], gpu);
  MUON_ORDINARY(ys && ys->dim() == 2 && dtype_of(*ys) >= 0);
  const int64_t width = ys->size(1), slots = r.tokens * r.top;
  const int dt = dtype_of(*ys);
  int w_dt, dw_dt;
  const int64_t ld = row_stride(ys, slots, width, dt), ld_dy = row_stride(dy, r.tokens, width, dt);
  const int64_t ld_dys = row_stride(dys, slots, width, dt);
  MUON_ORDINARY(ld >= 0 && ld_dy >= 0 && ld_dys >= 0 && per_slot(w, r, w_dt) && per_slot(dw, r, dw_dt) && w_dt == dw_dt);
  const void *p_dy = dy->data_ptr(), *p_ys = ys->data_ptr(), *p_w = w->data_ptr();
  void *p_dys = dys->data_ptr(), *p_dw = dw->data_ptr(), *s = stream_of(gpu);
  const muon_status_t st = released([&] {
    return f_combine_grad(p_dy, ld_dy, p_ys, ld, width, static_cast<muon_dtype_t>(dt), &r, p_w,
                          static_cast<muon_dtype_t>(w_dt), p_dys, ld_dys, p_dw, s);
  });
  if (st != MUON_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(OO)", a[6], a[7]);
  END_HANDLE_TH_ERRORS
}

// x, w, bias or None, activation, residual or None, offsets or None, pre or None, out or None
PyObject* py_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int gpu = current_gpu();
  MUON_ORDINARY(n == 8 && f_linear && !recorded(a, n) && PyLong_Check(a[3]));
  const at::Tensor *x = tensor_on(a[0], gpu), *w = tensor_on(a[1], gpu);
  MUON_ORDINARY(x && x->dim() == 2 && dtype_of(*x) >= 0 && w && (w->dim() == 2 || w->dim() == 3));
  const int dt = dtype_of(*x), d = static_cast<int>(w->dim());
  linear_args_t p{};
  p.rows = x->size(0);
  p.in = x->size(1);
  p.out = w->size(d - 2);
  p.groups = d == 3 ? w->size(0) : 1;
  p.dtype = dt;
  p.activation = static_cast<int32_t>(PyLong_AsLong(a[3]));
  p.x_stride = row_stride(x, p.rows, p.in, dt);
  MUON_ORDINARY(p.x_stride >= 0 && dtype_of(*w) == dt && w->size(d - 1) == p.in && w->stride(d - 1) == 1);
  p.w_stride = w->stride(d - 2);
  p.w_group_stride = d == 3 ? w->stride(0) : p.out * p.w_stride;
  MUON_ORDINARY(p.w_stride >= p.in && p.w_group_stride >= p.out * p.w_stride);
  if (a[2] != Py_None) {
    const at::Tensor* t = tensor_on(a[2], gpu);
    MUON_ORDINARY(t && dtype_of(*t) == dt && t->is_contiguous() && t->dim() == d - 1 && t->size(d - 2) == p.out &&
                  t->numel() == p.groups * p.out);
    p.bias = t->data_ptr();
  }
  if (a[4] != Py_None) {
    const at::Tensor* t = tensor_on(a[4], gpu);
    MUON_ORDINARY((p.residual_stride = row_stride(t, p.rows, p.out, dt)) >= 0);
    p.residual = t->data_ptr();
  }
  if (a[5] != Py_None) {
    const at::Tensor* t = tensor_on(a[5], gpu);
    MUON_ORDINARY(ints(t, p.groups + 1) && t->dim() == 1);
    p.offsets = static_cast<const int32_t*>(t->data_ptr());
  }
  if (a[6] != Py_None) {
    const at::Tensor* t = tensor_on(a[6], gpu);
    MUON_ORDINARY((p.pre_stride = row_stride(t, p.rows, p.out, dt)) >= 0);
    p.pre = t->data_ptr();
  }
  MUON_ORDINARY(p.offsets || p.groups == 1);
  PyObject* out = a[7] == Py_None ? THPVariable_Wrap(at::empty({p.rows, p.out}, x->options())) : given(a[7]);
  const at::Tensor* o = tensor_on(out, gpu);
  p.y_stride = row_stride(o, p.rows, p.out, dt);
  if (p.y_stride < 0) {
    Py_DECREF(out);
    Py_RETURN_NONE;
  }
  p.x = x->data_ptr();
  p.w = w->data_ptr();
  p.y = o->data_ptr();
  void* s = stream_of(gpu);
  const muon_status_t st = released([&] { return f_linear(&p, s); });
  if (st == MUON_OK) return out;
  Py_DECREF(out);
  return PyLong_FromLong(st);
  END_HANDLE_TH_ERRORS
}

// Row and group strides of a weight (or its gradient) of groups x out x in.
bool weight_strides(const at::Tensor* t, int dims, int64_t groups, int64_t out, int64_t in, int64_t& ld, int64_t& group) {
  if (!t || t->dim() != dims || t->size(dims - 2) != out || t->size(dims - 1) != in || t->stride(dims - 1) != 1 ||
      (dims == 3 && t->size(0) != groups))
    return false;
  ld = t->stride(dims - 2);
  group = dims == 3 ? t->stride(0) : out * ld;
  return ld >= in && group >= out * ld;
}

// dy, x, w, activation, pre, offsets, dx, dw, db (tensors or None), accumulate
// (bool), x_activation, x_pre, workspace (tensor or None)
PyObject* py_linear_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const int gpu = current_gpu();
  MUON_ORDINARY(n == 13 && f_grad && f_grad_bytes && !recorded(a, 1) && PyLong_Check(a[3]) && PyBool_Check(a[9]) && PyLong_Check(a[10]));
  const at::Tensor* dy = tensor_on(a[0], gpu);
  MUON_ORDINARY(dy && dy->dim() == 2 && dtype_of(*dy) >= 0);
  const int dt = dtype_of(*dy);
  linear_grad_args_t p{};
  p.rows = dy->size(0);
  p.out = dy->size(1);
  p.dtype = dt;
  p.grad_dtype = dt;
  p.activation = static_cast<int32_t>(PyLong_AsLong(a[3]));
  p.x_activation = static_cast<int32_t>(PyLong_AsLong(a[10]));
  p.accumulate = a[9] == Py_True;
  MUON_ORDINARY((p.dy_stride = row_stride(dy, p.rows, p.out, dt)) >= 0);
  p.dy = dy->data_ptr();
  // The weight, or its gradient, says what the groups and the columns are.
  const at::Tensor* weight = tensor_on(a[2] != Py_None ? a[2] : a[7], gpu);
  MUON_ORDINARY(weight && (weight->dim() == 2 || weight->dim() == 3));
  const int d = static_cast<int>(weight->dim());
  p.groups = d == 3 ? weight->size(0) : 1;
  p.in = weight->size(d - 1);
  if (a[5] != Py_None) {
    const at::Tensor* t = tensor_on(a[5], gpu);
    MUON_ORDINARY(ints(t, p.groups + 1) && t->dim() == 1);
    p.offsets = static_cast<const int32_t*>(t->data_ptr());
  }
  MUON_ORDINARY(p.offsets || p.groups == 1);
  if (p.activation) {
    const at::Tensor* t = tensor_on(a[4], gpu);
    MUON_ORDINARY((p.pre_stride = row_stride(t, p.rows, p.out, dt)) >= 0);
    p.pre = t->data_ptr();
  }
  if (a[6] != Py_None) {
    const at::Tensor *dx = tensor_on(a[6], gpu), *w = tensor_on(a[2], gpu);
    MUON_ORDINARY(weight_strides(w, d, p.groups, p.out, p.in, p.w_stride, p.w_group_stride) && dtype_of(*w) == dt &&
                  (p.dx_stride = row_stride(dx, p.rows, p.in, dt)) >= 0);
    p.w = w->data_ptr();
    p.dx = dx->data_ptr();
    if (p.x_activation) {
      const at::Tensor* t = tensor_on(a[11], gpu);
      MUON_ORDINARY((p.x_pre_stride = row_stride(t, p.rows, p.in, dt)) >= 0);
      p.x_pre = t->data_ptr();
    }
  }
  if (a[7] != Py_None) {
    const at::Tensor *dw = tensor_on(a[7], gpu), *x = tensor_on(a[1], gpu);
    MUON_ORDINARY(weight_strides(dw, d, p.groups, p.out, p.in, p.dw_stride, p.dw_group_stride) && dtype_of(*dw) >= 0 &&
                  (p.x_stride = row_stride(x, p.rows, p.in, dt)) >= 0);
    p.grad_dtype = dtype_of(*dw);
    p.x = x->data_ptr();
    p.dw = dw->data_ptr();
  }
  if (a[8] != Py_None) {
    const at::Tensor* db = tensor_on(a[8], gpu);
    MUON_ORDINARY(db && db->is_contiguous() && db->dim() == d - 1 && db->size(d - 2) == p.out &&
                  db->numel() == p.groups * p.out && dtype_of(*db) >= 0 && (!p.dw || dtype_of(*db) == p.grad_dtype));
    p.grad_dtype = dtype_of(*db);
    p.db = db->data_ptr();
  }
  MUON_ORDINARY(p.dx || p.dw || p.db);
  size_t bytes = 0;
  muon_status_t st = f_grad_bytes(&p, &bytes);
  MUON_ORDINARY(st == MUON_OK);
  // A new workspace belongs to the current stream, where the kernels run: the
  // allocator hands it out again behind them.
  at::Tensor ws;
  if (a[12] != Py_None) {
    const at::Tensor* t = tensor_on(a[12], gpu);
    MUON_ORDINARY(t && t->scalar_type() == at::kByte && t->is_contiguous());
    ws = *t;
  } else if (bytes) {
    ws = at::empty({static_cast<int64_t>(bytes)}, dy->options().dtype(at::kByte));
  }
  void *w_ptr = ws.defined() ? ws.data_ptr() : nullptr, *s = stream_of(gpu);
  const size_t w_bytes = ws.defined() ? static_cast<size_t>(ws.numel()) : 0;
  st = released([&] { return f_grad(&p, w_ptr, w_bytes, s); });
  if (st != MUON_OK) return PyLong_FromLong(st);
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// Addresses of the library's entry points, in this order: expert_sort,
// expert_gather, expert_combine, expert_combine_grad, linear_forward,
// linear_grad_workspace_bytes, linear_grad.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kEntries = 7;
  if (n != kEntries) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  void* p[kEntries];
  for (int i = 0; i < kEntries; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "address 0");
      return nullptr;
    }
  }
  f_sort = reinterpret_cast<decltype(f_sort)>(p[0]);
  f_gather = reinterpret_cast<decltype(f_gather)>(p[1]);
  f_combine = reinterpret_cast<decltype(f_combine)>(p[2]);
  f_combine_grad = reinterpret_cast<decltype(f_combine_grad)>(p[3]);
  f_linear = reinterpret_cast<decltype(f_linear)>(p[4]);
  f_grad_bytes = reinterpret_cast<decltype(f_grad_bytes)>(p[5]);
  f_grad = reinterpret_cast<decltype(f_grad)>(p[6]);
  Py_RETURN_NONE;
}

#define MUON_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MUON_METHOD(bind),         MUON_METHOD(sort),   MUON_METHOD(gather), MUON_METHOD(combine),
                         MUON_METHOD(combine_grad), MUON_METHOD(linear), MUON_METHOD(linear_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#define MUON_TEXT_OF(x) #x
#define MUON_TEXT(x) MUON_TEXT_OF(x)

// The caller compares the versions that this was compiled against with the running ones.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && (PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0 ||
            PyModule_AddStringConstant(m, "python_version", MUON_TEXT(PY_MAJOR_VERSION) "." MUON_TEXT(PY_MINOR_VERSION)) < 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
