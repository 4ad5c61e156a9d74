// The operators' Python calls, in C++: checks the tensors, allocates what is not given and
// calls the C ABI of include/moe.h.  It computes nothing.
//
// A call through ctypes with its checks in Python takes 6 to 10 us on the host (20 and more
// where it allocates several tensors), as long as or longer than the kernels of a decode
// step; here the same call takes 3 to 5 us, of which the launch itself is 2 to 3.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <climits>
#include <sstream>

#include "moe.h"

namespace {

PyObject* g_error = nullptr;  // MoeError of the package

struct Refused {  // a ValueError of the Python caller
  std::string why;
};
struct Pending {};  // a Python error is set already

template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused{s.str()};
}

std::string shape_of(const at::Tensor& t) {
  std::ostringstream s;
  s << toString(t.scalar_type()) << " " << t.sizes() << " on " << t.device();
  return s.str();
}

bool none(PyObject* o) { return o == Py_None; }

// Whether autograd records what is computed from t: the result would silently be cut off from it.
bool recorded(const at::Tensor& t) {
  if (!torch::autograd::impl::get_autograd_meta(t)) return false;  // most tensors
  if (c10::GradMode::is_enabled() && t.requires_grad()) return true;
  return c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  const at::Tensor& t = THPVariable_Unpack(o);
  // its memory holds the values with the other sign
  if (t.is_neg()) refuse(name, " is negated lazily: pass its resolve_neg()");
  if (recorded(t))
    refuse(name, " takes part in a gradient, which this call does not record: make it under torch.no_grad(), or in a "
                 "torch.autograd.Function whose backward makes the gradient's call");
  return t;
}

int32_t integer(PyObject* o, const char* name) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) throw Pending{};
  if (over || v > INT_MAX || v < INT_MIN) refuse(name, " does not fit 32 bits");
  return (int32_t)v;
}
int32_t extent(int64_t v, const char* name) {
  if (v > INT_MAX) refuse(name, " does not fit 32 bits");
  return (int32_t)v;
}

int32_t value_type(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_BF16;
    case at::kHalf: return MOE_F16;
    case at::kFloat: return MOE_F32;
    default: refuse(name, " must be bfloat16, float16 or float32, got ", toString(t.scalar_type()));
  }
}

struct Rows {
  void* p;
  int64_t ld;
};

// Device and stream of one call, taken from its first tensor; while it lives, that device is
// the current one, and so is the given stream (what the call allocates belongs to it).
struct Call {
  int dev;
  cudaStream_t stream;
  c10::cuda::OptionalCUDAGuard device_guard;
  c10::cuda::OptionalCUDAStreamGuard stream_guard;

  Call(const at::Tensor& first, PyObject* given) {
    if (!first.is_cuda()) refuse("operands must be cuda tensors");
    dev = first.get_device();
    if (c10::cuda::current_device() != dev) device_guard.set_index((c10::DeviceIndex)dev);
    if (none(given)) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    } else {
      int64_t v[3];
      const char* names[3] = {"stream_id", "device_index", "device_type"};
      for (int i = 0; i < 3; ++i) {
        PyObject* a = PyObject_GetAttrString(given, names[i]);
        if (!a) throw Pending{};
        v[i] = PyLong_AsLongLong(a);
        Py_DECREF(a);
        if (v[i] == -1 && PyErr_Occurred()) throw Pending{};
      }
      if (v[1] != dev) refuse("the stream is on cuda:", v[1], ", the operands on cuda:", dev);
      const auto s = c10::cuda::CUDAStream::unpack3(v[0], (c10::DeviceIndex)v[1], (c10::DeviceType)v[2]);
      stream_guard.reset_stream(s);
      stream = s.stream();
    }
  }

  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
  }

  // A matrix [R, F] with contiguous rows: pointer and pitch.
  Rows rows(const at::Tensor& t, const char* name, int64_t R, int64_t F, at::ScalarType type) const {
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.dim() != 2 || t.size(0) != R || t.size(1) != F)
      refuse(name, " must be ", toString(type), " [", R, ", ", F, "] on cuda:", dev, ", got ", shape_of(t));
    if (t.stride(1) != 1 && F > 1) refuse(name, " must have contiguous rows, got strides ", t.strides());
    return {t.data_ptr(), R > 1 ? t.stride(0) : F};
  }
  void* flat(const at::Tensor& t, const char* name, int64_t count, at::ScalarType type) const {
    if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.numel() != count || !t.is_contiguous())
      refuse(name, " must be ", count, " contiguous values of ", toString(type), " on cuda:", dev, ", got ", shape_of(t));
    return t.data_ptr();
  }
  void* flat(PyObject* o, const char* name, int64_t count, at::ScalarType type) const {
    return flat(tensor(o, name), name, count, type);
  }
  at::Tensor given_or_empty(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type) const {
    return none(o) ? empty(shape, type) : tensor(o, name);
  }
  // The workspace: `ws` if given, else `need` bytes held by `held` until the call returns
  // (the allocator hands them on in stream order).
  void* workspace(PyObject* ws, uint64_t need, at::Tensor& held, uint64_t* bytes) const {
    if (none(ws)) {
      *bytes = need;
      if (need == 0) return nullptr;
      held = empty({(int64_t)need}, at::kByte);
      return held.data_ptr();
    }
    held = tensor(ws, "ws");
    if (!held.is_cuda() || held.get_device() != dev || !held.is_contiguous())
      refuse("ws must be contiguous memory on cuda:", dev, ", got ", shape_of(held));
    *bytes = held.nbytes();
    return held.data_ptr();
  }
  const int32_t* limit(PyObject* o) const {
    return none(o) ? nullptr : (const int32_t*)flat(o, "rows", 1, at::kInt);
  }
};

void done(const char* name, moe_status rc) {
  if (rc == MOE_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "si", name, (int)rc);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Pending{};
}

// A call of the C ABI, during which other Python threads run: a launch waits where the
// device's queue is full.
template <typename F>
void run(const char* name, F call) {
  PyThreadState* held = PyEval_SaveThread();
  const moe_status rc = call();
  PyEval_RestoreThread(held);
  done(name, rc);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
// The caller's object if one was given, the new tensor otherwise.
PyObject* answer(PyObject* given, const at::Tensor& t) {
  return none(given) ? wrap(t) : Py_NewRef(given);
}

// An 8-bit checkpoint as Python holds it, its handle: (memory, offset, exponents or None,
// R, F).  With exponents None both parts lie in one piece of memory, as save makes it.
struct Ckpt {
  int8_t* q;
  uint8_t* e;
};
int64_t ckpt_codes(int64_t R, int64_t F) { return (R * F + 255) / 256 * 256; }
int64_t ckpt_bytes(int64_t R, int64_t F) { return ckpt_codes(R, F) + (R * ((F + 31) / 32) + 255) / 256 * 256; }

Ckpt ckpt(const Call& c, PyObject* o, int64_t R, int64_t F) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) refuse("not a checkpoint");
  const at::Tensor& mem = tensor(PyTuple_GET_ITEM(o, 0), "codes");
  const int64_t at = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1)), r = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 3)),
                f = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 4));
  if (PyErr_Occurred()) throw Pending{};
  if (r != R || f != F || !mem.is_cuda() || mem.get_device() != c.dev)
    refuse("the checkpoint must be of [", R, ", ", F, "] on cuda:", c.dev, ", is of [", r, ", ", f, "] on ", mem.device());
  PyObject* ex = PyTuple_GET_ITEM(o, 2);
  if (!none(ex))
    return {(int8_t*)c.flat(mem, "codes", R * F, at::kChar),
            (uint8_t*)c.flat(ex, "exps", R * ((F + 31) / 32), at::kByte)};
  if (mem.scalar_type() != at::kByte || !mem.is_contiguous() || at < 0 || at + ckpt_bytes(R, F) > mem.numel())
    refuse("not a checkpoint of [", R, ", ", F, "]: ", shape_of(mem));
  char* p = (char*)mem.data_ptr() + at;
  return {(int8_t*)p, (uint8_t*)p + ckpt_codes(R, F)};
}

// The handle of the checkpoint at `at` of mem, and its pointers.
PyObject* new_handle(const at::Tensor& mem, int64_t at, int64_t R, int64_t F, Ckpt* k) {
  char* p = (char*)mem.data_ptr() + at;
  *k = {(int8_t*)p, (uint8_t*)p + ckpt_codes(R, F)};
  return Py_BuildValue("(NLOLL)", wrap(mem), (long long)at, Py_None, (long long)R, (long long)F);
}
PyObject* const* pair(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) refuse("not the checkpoints of g and u");
  return &PyTuple_GET_ITEM(o, 0);
}

// ---------------------------------------------------------------- routes
struct Routes {
  int32_t *perm, *inv, *offsets;
};
Routes routes(const Call& c, PyObject* perm, PyObject* inv, PyObject* offsets, int64_t R, int64_t E) {
  return {(int32_t*)c.flat(perm, "perm", R, at::kInt), (int32_t*)c.flat(inv, "inv", R, at::kInt),
          (int32_t*)c.flat(offsets, "offsets", E + 1, at::kInt)};
}

void entries(const at::Tensor& idx, int32_t* T, int32_t* k) {
  if (idx.dim() != 1 && idx.dim() != 2) refuse("idx must be [T] or [T, k], got ", idx.sizes());
  *T = extent(idx.size(0), "T");
  *k = idx.dim() == 2 ? extent(idx.size(1), "k") : 1;
}

// New routes: (perm, inv, offsets)
PyObject* new_routes(const Call& c, int64_t R, int64_t E, Routes* r) {
  if (E < 0) refuse("E must not be negative, got ", E);
  const at::Tensor perm = c.empty({R}, at::kInt), inv = c.empty({R}, at::kInt), offsets = c.empty({E + 1}, at::kInt);
  *r = {(int32_t*)perm.data_ptr(), (int32_t*)inv.data_ptr(), (int32_t*)offsets.data_ptr()};
  return Py_BuildValue("(NNN)", wrap(perm), wrap(inv), wrap(offsets));
}

// sort(idx, E, perm, inv, offsets, ws, stream): None, or (perm, inv, offsets) where perm is None
PyObject* do_sort(PyObject* const* a) {
  const at::Tensor& idx = tensor(a[0], "idx");
  const Call c(idx, a[6]);
  int32_t T, k;
  entries(idx, &T, &k);
  const int32_t E = integer(a[1], "E");
  const int64_t R = (int64_t)T * k;
  const int32_t* ip = (const int32_t*)c.flat(idx, "idx", R, at::kInt);
  uint64_t need = 0, bytes = 0;
  done("moe_sort", moe_sort(nullptr, T, k, E, nullptr, nullptr, nullptr, nullptr, 0, &need, nullptr));
  Routes r;
  PyObject* made = none(a[2]) ? new_routes(c, R, E, &r) : (r = routes(c, a[2], a[3], a[4], R, E), Py_NewRef(Py_None));
  if (!made) throw Pending{};
  THPObjectPtr hold(made);
  at::Tensor held;
  void* ws = c.workspace(a[5], need, held, &bytes);
  run("moe_sort", [&] { return moe_sort(ip, T, k, E, r.perm, r.inv, r.offsets, ws, bytes, nullptr, c.stream); });
  return hold.release();
}

// dispatch(x, idx, E, xs, perm, inv, offsets, ws, stream): (xs, routes or None)
PyObject* do_dispatch(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &idx = tensor(a[1], "idx");
  const Call c(x, a[8]);
  const int32_t dt = value_type(x, "x");
  int32_t T, k;
  entries(idx, &T, &k);
  const int32_t E = integer(a[2], "E");
  const int64_t R = (int64_t)T * k;
  if (x.dim() != 2) refuse("x must be a matrix, got ", x.sizes());
  const int32_t H = extent(x.size(1), "H");
  const Rows xr = c.rows(x, "x", T, H, x.scalar_type());
  const int32_t* ip = (const int32_t*)c.flat(idx, "idx", R, at::kInt);
  uint64_t need = 0, bytes = 0;
  done("moe_dispatch", moe_sort(nullptr, T, k, E, nullptr, nullptr, nullptr, nullptr, 0, &need, nullptr));
  const at::Tensor xs = c.given_or_empty(a[3], "xs", {R, H}, x.scalar_type());
  const Rows xsr = c.rows(xs, "xs", R, H, x.scalar_type());
  Routes r;
  PyObject* made = none(a[4]) ? new_routes(c, R, E, &r) : (r = routes(c, a[4], a[5], a[6], R, E), Py_NewRef(Py_None));
  if (!made) throw Pending{};
  THPObjectPtr hold(made);
  at::Tensor held;
  void* ws = c.workspace(a[7], need, held, &bytes);
  run("moe_dispatch", [&] {
    return moe_dispatch(xr.p, xr.ld, dt, ip, T, k, E, H, xsr.p, xsr.ld, r.perm, r.inv, r.offsets, ws, bytes, nullptr,
                        c.stream);
  });
  return Py_BuildValue("(NN)", answer(a[3], xs), hold.release());
}

// collect(o, w or None, inv, T, k, y, stream): y.  Without weights: the gradient of dispatch.
PyObject* collect(PyObject* const* a, bool weighted) {
  const at::Tensor& o = tensor(a[0], weighted ? "o" : "dxs");
  const Call c(o, a[6]);
  const int32_t dt = value_type(o, weighted ? "o" : "dxs");
  const int32_t T = integer(a[3], "T"), k = integer(a[4], "k");
  const int64_t R = (int64_t)T * k;
  if (o.dim() != 2) refuse(weighted ? "o" : "dxs", " must be a matrix, got ", o.sizes());
  const int32_t H = extent(o.size(1), "H");
  const Rows r = c.rows(o, weighted ? "o" : "dxs", R, H, o.scalar_type());
  const float* w = weighted ? (const float*)c.flat(a[1], "w", R, at::kFloat) : nullptr;
  const int32_t* inv = (const int32_t*)c.flat(a[2], "inv", R, at::kInt);
  const at::Tensor y = c.given_or_empty(a[5], weighted ? "y" : "dx", {T, H}, o.scalar_type());
  const Rows yr = c.rows(y, weighted ? "y" : "dx", T, H, o.scalar_type());
  if (weighted)
    run("moe_collect", [&] { return moe_collect(r.p, r.ld, dt, w, inv, T, k, H, yr.p, yr.ld, c.stream); });
  else
    run("moe_dispatch_backward",
        [&] { return moe_dispatch_backward(r.p, r.ld, dt, inv, T, k, H, yr.p, yr.ld, c.stream); });
  return answer(a[5], y);
}
PyObject* do_collect(PyObject* const* a) { return collect(a, true); }
PyObject* do_dispatch_backward(PyObject* const* a) { return collect(a, false); }

// collect_backward(dy, o, w, inv, T, k, do, dw, stream): (do, dw)
PyObject* do_collect_backward(PyObject* const* a) {
  const at::Tensor &dy = tensor(a[0], "dy"), &o = tensor(a[1], "o");
  const Call c(o, a[8]);
  const int32_t dt = value_type(o, "o");
  const int32_t T = integer(a[4], "T"), k = integer(a[5], "k");
  const int64_t R = (int64_t)T * k;
  if (o.dim() != 2) refuse("o must be a matrix, got ", o.sizes());
  const int32_t H = extent(o.size(1), "H");
  const Rows gr = c.rows(dy, "dy", T, H, o.scalar_type()), orw = c.rows(o, "o", R, H, o.scalar_type());
  const float* w = (const float*)c.flat(a[2], "w", R, at::kFloat);
  const int32_t* inv = (const int32_t*)c.flat(a[3], "inv", R, at::kInt);
  const at::Tensor d = c.given_or_empty(a[6], "do", {R, H}, o.scalar_type());
  const at::Tensor dw = c.given_or_empty(a[7], "dw", {T, k}, at::kFloat);
  const Rows dr = c.rows(d, "do", R, H, o.scalar_type());
  float* dwp = (float*)c.flat(dw, "dw", R, at::kFloat);
  run("moe_collect_backward", [&] {
    return moe_collect_backward(gr.p, gr.ld, orw.p, orw.ld, dt, w, inv, T, k, H, dr.p, dr.ld, dwp, c.stream);
  });
  return Py_BuildValue("(NN)", answer(a[6], d), answer(a[7], dw));
}

// ---------------------------------------------------------------- 8-bit checkpoints
// act_save(x, handle or None, rows, stream): the handle
PyObject* do_act_save(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const Call c(x, a[3]);
  const int32_t dt = value_type(x, "x");
  if (x.dim() != 2) refuse("x must be a matrix, got ", x.sizes());
  const int32_t R = extent(x.size(0), "R"), F = extent(x.size(1), "F");
  const Rows r = c.rows(x, "x", R, F, x.scalar_type());
  Ckpt k;
  const bool fresh = none(a[1]);
  if (!fresh) k = ckpt(c, a[1], R, F);
  THPObjectPtr handle(fresh ? new_handle(c.empty({ckpt_bytes(R, F)}, at::kByte), 0, R, F, &k) : Py_NewRef(a[1]));
  if (!handle) throw Pending{};
  const int32_t* limit = c.limit(a[2]);
  run("moe_act_save", [&] { return moe_act_save(r.p, r.ld, dt, R, F, k.q, k.e, limit, c.stream); });
  return handle.release();
}

// act_load(checkpoint, dtype, x, rows, stream): x
PyObject* do_act_load(PyObject* const* a) {
  if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 5) refuse("not a checkpoint");
  const at::Tensor& mem = tensor(PyTuple_GET_ITEM(a[0], 0), "codes");
  const Call c(mem, a[4]);
  const int32_t R = integer(PyTuple_GET_ITEM(a[0], 3), "R"), F = integer(PyTuple_GET_ITEM(a[0], 4), "F");
  if (!THPDtype_Check(a[1])) refuse("dtype must be a torch.dtype");
  const at::Tensor x = c.given_or_empty(a[2], "x", {R, F}, reinterpret_cast<THPDtype*>(a[1])->scalar_type);
  const int32_t dt = value_type(x, "x");
  const Rows r = c.rows(x, "x", R, F, x.scalar_type());
  const Ckpt k = ckpt(c, a[0], R, F);
  const int32_t* limit = c.limit(a[3]);
  run("moe_act_load", [&] { return moe_act_load(k.q, k.e, R, F, dt, r.p, r.ld, limit, c.stream); });
  return answer(a[2], x);
}

// swiglu_save(g, u, h, (handle of g, of u) or None, rows, stream): (h, handles)
PyObject* do_swiglu_save(PyObject* const* a) {
  const at::Tensor &g = tensor(a[0], "g"), &u = tensor(a[1], "u");
  const Call c(g, a[5]);
  const int32_t dt = value_type(g, "g");
  if (g.dim() != 2) refuse("g must be a matrix, got ", g.sizes());
  const int32_t R = extent(g.size(0), "R"), F = extent(g.size(1), "F");
  const Rows gr = c.rows(g, "g", R, F, g.scalar_type()), ur = c.rows(u, "u", R, F, g.scalar_type());
  const at::Tensor h = c.given_or_empty(a[2], "h", {R, F}, g.scalar_type());
  const Rows hr = c.rows(h, "h", R, F, g.scalar_type());
  Ckpt kg, ku;
  PyObject* made;
  if (none(a[3])) {
    const int64_t size = ckpt_bytes(R, F);
    const at::Tensor mem = c.empty({2 * size}, at::kByte);
    THPObjectPtr first(new_handle(mem, 0, R, F, &kg)), second(new_handle(mem, size, R, F, &ku));
    made = first && second ? PyTuple_Pack(2, first.get(), second.get()) : nullptr;
  } else {
    kg = ckpt(c, pair(a[3])[0], R, F);
    ku = ckpt(c, pair(a[3])[1], R, F);
    made = Py_NewRef(a[3]);
  }
  if (!made) throw Pending{};
  THPObjectPtr handles(made);
  const int32_t* limit = c.limit(a[4]);
  run("moe_swiglu_save", [&] {
    return moe_swiglu_save(gr.p, gr.ld, ur.p, ur.ld, dt, R, F, hr.p, hr.ld, kg.q, kg.e, ku.q, ku.e, limit, c.stream);
  });
  return Py_BuildValue("(NN)", answer(a[2], h), handles.release());
}

// swiglu_backward(dh, (handle of g, of u), dg, du, h, rebuild_h, rows, stream): (dg, du, h or None)
PyObject* do_swiglu_backward(PyObject* const* a) {
  const at::Tensor& dh = tensor(a[0], "dh");
  const Call c(dh, a[7]);
  const int32_t dt = value_type(dh, "dh");
  if (dh.dim() != 2) refuse("dh must be a matrix, got ", dh.sizes());
  const int32_t R = extent(dh.size(0), "R"), F = extent(dh.size(1), "F");
  const auto type = dh.scalar_type();
  const Rows r = c.rows(dh, "dh", R, F, type);
  const Ckpt kg = ckpt(c, pair(a[1])[0], R, F), ku = ckpt(c, pair(a[1])[1], R, F);
  const int again = none(a[4]) ? PyObject_IsTrue(a[5]) : 1;
  if (again < 0) throw Pending{};
  const at::Tensor dg = c.given_or_empty(a[2], "dg", {R, F}, type), du = c.given_or_empty(a[3], "du", {R, F}, type);
  const at::Tensor h = again ? c.given_or_empty(a[4], "h", {R, F}, type) : at::Tensor();
  const Rows gr = c.rows(dg, "dg", R, F, type), ur = c.rows(du, "du", R, F, type);
  const Rows hr = again ? c.rows(h, "h", R, F, type) : Rows{nullptr, F};
  const int32_t* limit = c.limit(a[6]);
  run("moe_swiglu_backward", [&] {
    return moe_swiglu_backward(r.p, r.ld, dt, kg.q, kg.e, ku.q, ku.e, R, F, gr.p, gr.ld, ur.p, ur.ld, hr.p, hr.ld, limit,
                               c.stream);
  });
  return Py_BuildValue("(NNN)", answer(a[2], dg), answer(a[3], du), again ? answer(a[4], h) : Py_NewRef(Py_None));
}

// ---------------------------------------------------------------- adapters
// adapters(x, y, A, B, scale, perm, inv, offsets, T, k, E, out, status, stream): out
PyObject* do_adapters(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &y = tensor(a[1], "y"), &A = tensor(a[2], "A"), &B = tensor(a[3], "B");
  const Call c(x, a[13]);
  const int32_t dt = value_type(x, "x");
  const auto type = x.scalar_type();
  if (x.dim() != 2) refuse("x must be a matrix, got ", x.sizes());
  const int32_t T = extent(x.size(0), "T"), K = extent(x.size(1), "K");
  if (A.dim() != 3 || B.dim() != 3 || A.size(2) != K || B.size(0) != A.size(0) || B.size(2) != A.size(1))
    refuse("A must be [n, r, ", K, "] and B [n, N, r], got ", A.sizes(), " and ", B.sizes());
  const int32_t n = extent(A.size(0), "n"), r = extent(A.size(1), "r"), N = extent(B.size(1), "N");
  if (integer(a[8], "T") != T || integer(a[9], "k") != 1 || integer(a[10], "E") != n)
    refuse("the routes must be of ", T, " tokens, one entry each, in ", n, " groups");
  const Rows xr = c.rows(x, "x", T, K, type), yr = c.rows(y, "y", T, N, type);
  const void *Ap = c.flat(A, "A", (int64_t)n * r * K, type), *Bp = c.flat(B, "B", (int64_t)n * N * r, type);
  const float* scale = (const float*)c.flat(a[4], "scale", n, at::kFloat);
  const Routes rt = routes(c, a[5], a[6], a[7], T, n);
  const at::Tensor out = c.given_or_empty(a[11], "out", {T, N}, type);
  const Rows outr = c.rows(out, "out", T, N, type);
  int32_t* status = none(a[12]) ? nullptr : (int32_t*)c.flat(a[12], "status", 1, at::kInt);
  run("moe_adapters", [&] {
    return moe_adapters(xr.p, xr.ld, yr.p, yr.ld, dt, T, K, N, r, n, Ap, Bp, scale, rt.perm, rt.offsets, outr.p, outr.ld,
                        status, c.stream);
  });
  return answer(a[11], out);
}

// ---------------------------------------------------------------- module
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, count);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.why.c_str());
    return nullptr;
  } catch (const Pending&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* e) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(e);
  Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<do_##name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"set_error", set_error, METH_O, nullptr},
                         ENTRY(sort, 7),
                         ENTRY(dispatch, 9),
                         ENTRY(dispatch_backward, 7),
                         ENTRY(collect, 7),
                         ENTRY(collect_backward, 9),
                         ENTRY(act_save, 4),
                         ENTRY(act_load, 5),
                         ENTRY(swiglu_save, 6),
                         ENTRY(swiglu_backward, 8),
                         ENTRY(adapters, 14),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_ops() { return PyModule_Create(&module); }
