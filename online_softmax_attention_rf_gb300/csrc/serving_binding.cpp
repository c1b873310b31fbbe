// serving_binding.cpp -- Python entry of the paged serving calls.
//
// Argument marshalling only, like api.py's ctypes calls, for the three calls
// that a decode step makes once a layer or once a token: checked through
// ctypes, one of them costs its caller 20 us of host time, three times what
// the launches take. Each function checks that its torch tensors fit, allocates
// the outputs it was not given, and passes pointers, sizes and the current
// stream of the tensors' device to the C entry point of the same name. It
// returns the outputs, the rf_status of a refused call as an int, or None when
// the tensors do not fit (api.py then names the fault).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "rf.h"

namespace {

using at::Tensor;

struct Misfit {};  // thrown by the checks below, turned into None

void need(bool ok) {
  if (!ok) throw Misfit{};
}

const Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

const Tensor* maybe(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }

template <typename T = void>
T* ptr(const Tensor* t) {
  return t != nullptr ? static_cast<T*>(t->data_ptr()) : nullptr;
}

int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  need(!(v == -1 && PyErr_Occurred()));
  need(v >= INT32_MIN && v <= INT32_MAX);
  return static_cast<int>(v);
}

double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  need(!(v == -1.0 && PyErr_Occurred()));
  return v;
}

// A contiguous tensor of this type and shape on this device.
void fits(const Tensor& t, at::ScalarType dt, at::IntArrayRef shape, at::Device dev) {
  need(t.scalar_type() == dt && t.sizes() == shape && t.is_contiguous() && t.device() == dev);
}
void fits(const Tensor* t, at::ScalarType dt, at::IntArrayRef shape, at::Device dev) {
  if (t != nullptr) fits(*t, dt, shape, dev);
}

rf_dtype dtype_of(const Tensor& t) {
  need(t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16);
  return t.scalar_type() == at::kFloat ? RF_F32 : RF_BF16;
}

// Rows [T, heads, d] with a token's heads back to back: the token stride.
int64_t rows(const Tensor& t, at::ScalarType dt, int64_t T, int64_t d, at::Device dev) {
  need(t.dim() == 3 && t.size(0) == T && t.size(2) == d && t.scalar_type() == dt &&
       t.device() == dev && t.stride(2) == 1 && (t.size(1) == 1 || t.stride(1) == d));
  return T > 1 ? t.stride(0) : t.size(1) * d;
}

// A pool [pages, page, Hkv, d] of any strides with d contiguous.
void pool(const Tensor& t, at::ScalarType dt, int64_t Hkv, int64_t d, at::Device dev) {
  need(t.dim() == 4 && t.size(2) == Hkv && t.size(3) == d && t.stride(3) == 1 &&
       t.scalar_type() == dt && t.device() == dev);
}

int to_int(int64_t v) {
  need(v >= 0 && v <= INT32_MAX);
  return static_cast<int>(v);
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType dt, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(dt).device(dev));
}

rf_stream stream_of(at::Device dev) {
  return reinterpret_cast<rf_stream>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// What a call returns: `a` (and `b`), or the status of a refused call.
PyObject* result(rf_status st, PyObject* a, PyObject* b) {
  if (st != RF_OK) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    return PyLong_FromLong(st);
  }
  PyObject* t = PyTuple_Pack(2, a, b);
  Py_DECREF(a);
  Py_DECREF(b);
  return t;
}

PyObject* wrap_or_none(const Tensor* t) {
  if (t == nullptr) Py_RETURN_NONE;
  return THPVariable_Wrap(*t);
}

PyObject* misfit() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// q, k_cache, v_cache, block_table, plan buffer, B, T, H, Hkv, page, max_pages,
// scale or None, out or None, lse or None, with_lse, workspace
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 16);
    const Tensor &q = tensor(a[0]), &kc = tensor(a[1]), &vc = tensor(a[2]), &table = tensor(a[3]),
                 &plan = tensor(a[4]), &ws = tensor(a[15]);
    const int B = as_int(a[5]), T = as_int(a[6]), H = as_int(a[7]), Hkv = as_int(a[8]),
              page = as_int(a[9]), max_pages = as_int(a[10]);
    const at::Device dev = q.device();
    const at::ScalarType dt = q.scalar_type();
    need(dev.is_cuda() && q.dim() == 3 && q.size(1) == H);
    const int d = to_int(q.size(2));
    const int64_t qs = rows(q, dt, T, d, dev);
    pool(kc, dt, Hkv, d, dev);
    pool(vc, dt, Hkv, d, dev);
    need(kc.size(1) == page && vc.size(1) == page && vc.size(0) == kc.size(0));
    need(table.dim() == 2 && table.size(0) == B && table.size(1) == max_pages &&
         table.scalar_type() == at::kInt && table.device() == dev &&
         (max_pages == 1 || table.stride(1) == 1));
    need(plan.device() == dev && ws.device() == dev && ws.is_contiguous());
    const float scale =
        a[11] == Py_None ? 1.f / std::sqrt(static_cast<float>(d)) : static_cast<float>(as_double(a[11]));
    const Tensor *out = maybe(a[12]), *lse = maybe(a[13]);
    fits(out, dt, {T, H, d}, dev);
    fits(lse, at::kFloat, {T, H}, dev);
    const rf_dtype rdt = dtype_of(q);
    Tensor new_out, new_lse;
    if (out == nullptr) {
      new_out = fresh({T, H, d}, dt, dev);
      out = &new_out;
    }
    const int with_lse = PyObject_IsTrue(a[14]);
    need(with_lse >= 0);
    if (lse == nullptr && with_lse) {
      new_lse = fresh({T, H}, at::kFloat, dev);
      lse = &new_lse;
    }
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_attn_paged(
        q.data_ptr(), qs, kc.data_ptr(), kc.stride(0), kc.stride(1), kc.stride(2), vc.data_ptr(),
        vc.stride(0), vc.stride(1), vc.stride(2), page, to_int(kc.size(0)), ptr<int32_t>(&table),
        B > 1 ? table.stride(0) : max_pages, max_pages, plan.data_ptr(), B, T, H, Hkv, d, scale,
        out->data_ptr(), ptr<float>(lse), ptr<float>(&ws), ws.nbytes(), rdt, stream_of(dev));
    return result(st, wrap_or_none(out), wrap_or_none(lse));
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// q or None, k, v, k_cache, v_cache, slots, pos or None, cos_sin or None,
// q_weight or None, k_weight or None, eps, interleaved, q_out or None
PyObject* kv_append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 13);
    const Tensor *q = maybe(a[0]), *pos = maybe(a[6]), *cs = maybe(a[7]), *qw = maybe(a[8]),
                 *kw = maybe(a[9]), *q_out = maybe(a[12]);
    const Tensor &k = tensor(a[1]), &v = tensor(a[2]), &kc = tensor(a[3]), &vc = tensor(a[4]),
                 &slots = tensor(a[5]);
    const at::Device dev = k.device();
    const at::ScalarType dt = k.scalar_type();
    need(dev.is_cuda() && k.dim() == 3);
    const int T = to_int(k.size(0)), Hkv = to_int(k.size(1)), d = to_int(k.size(2));
    const int64_t ks = rows(k, dt, T, d, dev), vs = rows(v, dt, T, d, dev);
    need(v.size(1) == Hkv);
    pool(kc, dt, Hkv, d, dev);
    pool(vc, dt, Hkv, d, dev);
    need(vc.size(0) == kc.size(0) && vc.size(1) == kc.size(1));
    fits(slots, at::kLong, {T}, dev);
    fits(qw, dt, {d}, dev);
    fits(kw, dt, {d}, dev);
    int rot = 0, max_pos = 0;
    if (cs != nullptr) {
      need(cs->dim() == 2 && cs->scalar_type() == at::kFloat && cs->is_contiguous() &&
           cs->device() == dev && pos != nullptr);
      fits(pos, at::kInt, {T}, dev);
      max_pos = to_int(cs->size(0));
      rot = to_int(cs->size(1));
    }
    int H = 0;
    int64_t qs = 0;
    Tensor fresh_q;
    if (q != nullptr) {
      need(q->dim() == 3);
      H = to_int(q->size(1));
      qs = rows(*q, dt, T, d, dev);
      fits(q_out, dt, {T, H, d}, dev);
    }
    const double eps = as_double(a[10]);
    const int interleaved = PyObject_IsTrue(a[11]);
    need(interleaved >= 0);
    const rf_dtype rdt = dtype_of(k);
    if (q != nullptr && q_out == nullptr) {
      fresh_q = fresh({T, H, d}, dt, dev);
      q_out = &fresh_q;
    }
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_kv_append_paged(
        ptr<>(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, q != nullptr ? q_out->data_ptr() : nullptr,
        kc.data_ptr(), kc.stride(0), kc.stride(1), kc.stride(2), vc.data_ptr(), vc.stride(0),
        vc.stride(1), vc.stride(2), T, H, Hkv, d, to_int(kc.size(1)), to_int(kc.size(0)),
        ptr<int64_t>(&slots), ptr<int32_t>(pos), ptr<float>(cs), max_pos, rot, interleaved, ptr<>(qw),
        ptr<>(kw), static_cast<float>(eps), rdt, stream_of(dev));
    return result(st, wrap_or_none(q != nullptr ? q_out : nullptr), wrap_or_none(nullptr));
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// target, draft or None, tokens, u, expo, n_draft or None, temperature or None,
// workspace or None
PyObject* draft_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 8);
    const Tensor &target = tensor(a[0]), &tokens = tensor(a[2]), &u = tensor(a[3]),
                 &expo = tensor(a[4]);
    const Tensor *draft = maybe(a[1]), *n_draft = maybe(a[5]), *temperature = maybe(a[6]),
                 *ws = maybe(a[7]);
    const at::Device dev = target.device();
    const at::ScalarType dt = target.scalar_type();
    need(dev.is_cuda() && target.dim() == 3 && target.size(1) > 1 && target.is_contiguous());
    const int B = to_int(target.size(0)), S = to_int(target.size(1) - 1), V = to_int(target.size(2));
    fits(draft, dt, {B, S, V}, dev);
    fits(tokens, at::kInt, {B, S}, dev);
    fits(u, at::kFloat, {B, S}, dev);
    fits(expo, at::kFloat, {B, V}, dev);
    fits(n_draft, at::kInt, {B}, dev);
    fits(temperature, at::kFloat, {B}, dev);
    need(ws == nullptr || (ws->device() == dev && ws->is_contiguous()));
    const rf_dtype rdt = dtype_of(target);
    const Tensor out = fresh({B, S + 1}, at::kInt, dev), n_accepted = fresh({B}, at::kInt, dev);
    Tensor new_ws;
    if (ws == nullptr) {
      new_ws = fresh({static_cast<int64_t>(rf_draft_verify_workspace_bytes(B, S))}, at::kByte, dev);
      ws = &new_ws;
    }
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_draft_verify(
        target.data_ptr(), ptr<>(draft), ptr<int32_t>(&tokens), ptr<float>(&u), ptr<float>(&expo),
        ptr<int32_t>(n_draft), ptr<float>(temperature), B, S, V, ptr<int32_t>(&out),
        ptr<int32_t>(&n_accepted), ws->data_ptr(), ws->nbytes(), rdt, stream_of(dev));
    return result(st, THPVariable_Wrap(out), THPVariable_Wrap(n_accepted));
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

#define RF_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RF_METHOD(attn_paged), RF_METHOD(kv_append_paged), RF_METHOD(draft_verify),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rf_serving", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rf_serving() { return PyModule_Create(&module); }
