// serving_binding.cpp -- Python entry of the paged serving calls.
//
// Argument marshalling only, like api.py's ctypes calls, for the calls that a
// decode step makes once a layer or once a token: checked through
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

#include <array>
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

// Several new int32 outputs out of one allocation (one costs more than all the views of
// it), each on a boundary of 16 bytes. Of one type: torch.save refuses tensors of two
// types that share a storage.
template <size_t N>
std::array<Tensor, N> fresh_ints(const int64_t (&outs)[N], at::Device dev) {
  int64_t words = 0;
  for (const int64_t n : outs) words += (n + 3) / 4 * 4;
  const Tensor buf = fresh({words}, at::kInt, dev);
  std::array<Tensor, N> got;
  int64_t at = 0;
  for (size_t i = 0; i < N; ++i) {
    got[i] = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(buf.storage()), buf.key_set(), buf.dtype());
    c10::TensorImpl* t = got[i].unsafeGetTensorImpl();
    t->set_storage_offset(at);
    t->set_sizes_contiguous({outs[i]});
    at += (outs[i] + 3) / 4 * 4;
  }
  return got;
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
// scale or None, out or None, lse or None, with_lse, workspace, tree mask or None
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 17);
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
    const Tensor *out = maybe(a[12]), *lse = maybe(a[13]), *tree = maybe(a[16]);
    if (tree != nullptr) {
      need(tree->dim() == 2);
      fits(tree, at::kLong, {T, tree->size(1)}, dev);
    }
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
    auto call = [&](auto entry, auto... more) {
      return entry(q.data_ptr(), qs, kc.data_ptr(), kc.stride(0), kc.stride(1), kc.stride(2),
                   vc.data_ptr(), vc.stride(0), vc.stride(1), vc.stride(2), page,
                   to_int(kc.size(0)), ptr<int32_t>(&table), B > 1 ? table.stride(0) : max_pages,
                   max_pages, plan.data_ptr(), B, T, H, Hkv, d, scale, out->data_ptr(),
                   ptr<float>(lse), ptr<float>(&ws), ws.nbytes(), more..., rdt, stream_of(dev));
    };
    const rf_status st =
        tree == nullptr ? call(rf_attn_paged)
                        : call(rf_attn_paged_tree, static_cast<const uint64_t*>(tree->data_ptr()),
                               to_int(tree->size(1)));
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

// parent, cu_q, kv_len, words
PyObject* tree_mask(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 4);
    const Tensor &parent = tensor(a[0]), &cu_q = tensor(a[1]), &kv_len = tensor(a[2]);
    const at::Device dev = parent.device();
    need(dev.is_cuda() && parent.dim() == 1 && kv_len.dim() == 1);
    const int T = to_int(parent.size(0)), B = to_int(kv_len.size(0)), words = as_int(a[3]);
    fits(parent, at::kInt, {T}, dev);
    fits(cu_q, at::kInt, {B + 1}, dev);
    fits(kv_len, at::kInt, {B}, dev);
    const Tensor mask = fresh({T, words > 0 ? words : 0}, at::kLong, dev), pos = fresh({T}, at::kInt, dev);
    c10::cuda::CUDAGuard guard(dev);
    if (B == 0) {  // all rows lie outside every sequence, and no kernel runs
      mask.zero_();
      pos.zero_();
    }
    const rf_status st =
        rf_tree_mask(ptr<int32_t>(&parent), ptr<int32_t>(&cu_q), ptr<int32_t>(&kv_len), B, T, words,
                     ptr<uint64_t>(&mask), ptr<int32_t>(&pos), stream_of(dev));
    return result(st, THPVariable_Wrap(mask), THPVariable_Wrap(pos));
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// A tuple of new tensors, or the status of a refused call.
PyObject* results(rf_status st, std::initializer_list<const Tensor*> ts) {
  if (st != RF_OK) return PyLong_FromLong(st);
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (t == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* x : ts) PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(*x));
  return t;
}

// parent, tokens, sampled, cu_q, kv_len
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 5);
    const Tensor &parent = tensor(a[0]), &tokens = tensor(a[1]), &sampled = tensor(a[2]),
                 &cu_q = tensor(a[3]), &kv_len = tensor(a[4]);
    const at::Device dev = parent.device();
    need(dev.is_cuda() && parent.dim() == 1 && kv_len.dim() == 1);
    const int T = to_int(parent.size(0)), B = to_int(kv_len.size(0));
    for (const Tensor* t : {&parent, &tokens, &sampled}) fits(*t, at::kInt, {T}, dev);
    fits(cu_q, at::kInt, {B + 1}, dev);
    fits(kv_len, at::kInt, {B}, dev);
    const auto [path, out, n_path, base, new_len] = fresh_ints({T, T, B, B, B}, dev);
    c10::cuda::CUDAGuard guard(dev);
    if (B == 0) {  // all rows lie outside every sequence, and no kernel runs
      path.fill_(-1);
      out.fill_(-1);
    }
    const rf_status st = rf_tree_accept(
        ptr<int32_t>(&parent), ptr<int32_t>(&tokens), ptr<int32_t>(&sampled), ptr<int32_t>(&cu_q),
        ptr<int32_t>(&kv_len), B, T, ptr<int32_t>(&path), ptr<int32_t>(&out), ptr<int32_t>(&n_path),
        ptr<int32_t>(&base), ptr<int32_t>(&new_len), stream_of(dev));
    return results(st, {&path, &out, &n_path, &base, &new_len});
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// logits, expo, temperature or None, top_k or None, top_p or None, min_p or None
PyObject* sample_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 6);
    const Tensor &logits = tensor(a[0]), &expo = tensor(a[1]);
    const Tensor *temperature = maybe(a[2]), *top_k = maybe(a[3]), *top_p = maybe(a[4]),
                 *min_p = maybe(a[5]);
    const at::Device dev = logits.device();
    need(dev.is_cuda() && logits.dim() == 2);
    const int B = to_int(logits.size(0)), V = to_int(logits.size(1));
    need(V == 1 || logits.stride(1) == 1);
    fits(expo, at::kFloat, {B, V}, dev);
    fits(temperature, at::kFloat, {B}, dev);
    fits(top_k, at::kInt, {B}, dev);
    fits(top_p, at::kFloat, {B}, dev);
    fits(min_p, at::kFloat, {B}, dev);
    const rf_dtype rdt = dtype_of(logits);
    const Tensor token = fresh({B}, at::kInt, dev), logprob = fresh({B}, at::kFloat, dev);
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_sample_rows(
        logits.data_ptr(), logits.stride(0), ptr<float>(&expo), ptr<float>(temperature),
        ptr<int32_t>(top_k), ptr<float>(top_p), ptr<float>(min_p), B, V, ptr<int32_t>(&token),
        ptr<float>(&logprob), rdt, stream_of(dev));
    return results(st, {&token, &logprob});
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// A pool of one layer [pages, page, Hkv, d] or of several [layers, ...].
rf_kv_pool kv_pool(const Tensor& k, const Tensor& v, at::Device dev) {
  const int64_t o = k.dim() == 5;
  need(k.dim() == 4 + o && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() &&
       k.device() == dev && v.device() == dev && dev.is_cuda());
  need(k.size(3 + o) == 1 || (k.stride(3 + o) == 1 && v.stride(3 + o) == 1));
  rf_kv_pool p{};
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  // (a dimension of one has no stride)
  auto stride = [&](const Tensor& t, int64_t i) { return t.size(i) > 1 ? t.stride(i) : 0; };
  p.k_layer_stride = o ? stride(k, 0) : 0;
  p.k_page_stride = stride(k, o);
  p.k_token_stride = stride(k, 1 + o);
  p.k_head_stride = stride(k, 2 + o);
  p.v_layer_stride = o ? stride(v, 0) : 0;
  p.v_page_stride = stride(v, o);
  p.v_token_stride = stride(v, 1 + o);
  p.v_head_stride = stride(v, 2 + o);
  p.layers = o ? to_int(k.size(0)) : 1;
  p.num_pages = to_int(k.size(o));
  p.page = to_int(k.size(1 + o));
  p.Hkv = to_int(k.size(2 + o));
  p.d = to_int(k.size(3 + o));
  p.dt = dtype_of(k);
  return p;
}

// A block table [B, max_pages] with contiguous rows: the rows' distance.
int64_t table_rows(const Tensor& t, int64_t B, at::Device dev) {
  need(t.dim() == 2 && t.size(0) == B && t.scalar_type() == at::kInt && t.device() == dev &&
       (t.size(1) == 1 || t.stride(1) == 1));
  return B > 1 ? t.stride(0) : t.size(1);
}

// k_cache, v_cache, block_table, keep, cu_keep, n_keep or None, base or None
PyObject* kv_compact_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 7);
    const Tensor &k = tensor(a[0]), &v = tensor(a[1]), &table = tensor(a[2]), &keep = tensor(a[3]),
                 &cu_keep = tensor(a[4]);
    const Tensor *n_keep = maybe(a[5]), *base = maybe(a[6]);
    const at::Device dev = k.device();
    const rf_kv_pool pool = kv_pool(k, v, dev);
    need(keep.dim() == 1 && table.dim() == 2);
    const int N = to_int(keep.size(0)), B = to_int(table.size(0));
    const int64_t rows = table_rows(table, B, dev);
    fits(keep, at::kInt, {N}, dev);
    fits(cu_keep, at::kInt, {B + 1}, dev);
    fits(n_keep, at::kInt, {B}, dev);
    fits(base, at::kInt, {B}, dev);
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_kv_compact_paged(
        &pool, ptr<int32_t>(&table), rows, B, to_int(table.size(1)), ptr<int32_t>(&keep), N,
        ptr<int32_t>(&cu_keep), ptr<int32_t>(n_keep), ptr<int32_t>(base), stream_of(dev));
    return results(st, {});
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, src, dst
PyObject* kv_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 4);
    const Tensor &k = tensor(a[0]), &v = tensor(a[1]), &src = tensor(a[2]), &dst = tensor(a[3]);
    const at::Device dev = k.device();
    const rf_kv_pool pool = kv_pool(k, v, dev);
    need(src.dim() == 1);
    const int m = to_int(src.size(0));
    fits(src, at::kInt, {m}, dev);
    fits(dst, at::kInt, {m}, dev);
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st =
        rf_kv_copy_pages(&pool, ptr<int32_t>(&src), ptr<int32_t>(&dst), m, stream_of(dev));
    return results(st, {});
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// block_table, kv_len, src, table_out, refs, page
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 6);
    const Tensor &table = tensor(a[0]), &len = tensor(a[1]), &src = tensor(a[2]), &out = tensor(a[3]),
                 &refs = tensor(a[4]);
    const at::Device dev = table.device();
    need(dev.is_cuda() && len.dim() == 1 && src.dim() == 1 && refs.dim() == 1);
    const int B = to_int(len.size(0)), m = to_int(src.size(0));
    const int64_t rows = table_rows(table, B, dev), out_rows = table_rows(out, m, dev);
    need(out.size(1) == table.size(1));
    fits(len, at::kInt, {B}, dev);
    fits(src, at::kInt, {m}, dev);
    fits(refs, at::kInt, {refs.size(0)}, dev);
    const Tensor len_out = fresh({m}, at::kInt, dev);
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_pages_fork(
        ptr<int32_t>(&table), rows, ptr<int32_t>(&len), B, ptr<int32_t>(&src), m, ptr<int32_t>(&out),
        out_rows, ptr<int32_t>(&len_out), ptr<int32_t>(&refs), to_int(table.size(1)), as_int(a[5]),
        to_int(refs.size(0)), stream_of(dev));
    return results(st, {&len_out});
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// block_table, kv_len, new_len, refs, page
PyObject* pages_grow(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 5);
    const Tensor &table = tensor(a[0]), &len = tensor(a[1]), &new_len = tensor(a[2]),
                 &refs = tensor(a[3]);
    const at::Device dev = table.device();
    need(dev.is_cuda() && len.dim() == 1 && refs.dim() == 1);
    const int m = to_int(len.size(0));
    const int64_t rows = table_rows(table, m, dev);
    fits(len, at::kInt, {m}, dev);
    fits(new_len, at::kInt, {m}, dev);
    fits(refs, at::kInt, {refs.size(0)}, dev);
    const auto [src, dst, left] = fresh_ints({m, m, 1}, dev);
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_pages_grow(
        ptr<int32_t>(&table), rows, ptr<int32_t>(&len), ptr<int32_t>(&new_len), m,
        ptr<int32_t>(&refs), to_int(table.size(1)), as_int(a[4]), to_int(refs.size(0)),
        ptr<int32_t>(&src), ptr<int32_t>(&dst), ptr<int32_t>(&left), stream_of(dev));
    return results(st, {&src, &dst, &left});
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

// block_table, kv_len, refs, page, new_len or None
PyObject* pages_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    need(n == 5);
    const Tensor &table = tensor(a[0]), &len = tensor(a[1]), &refs = tensor(a[2]);
    const Tensor* new_len = maybe(a[4]);
    const at::Device dev = table.device();
    need(dev.is_cuda() && len.dim() == 1 && refs.dim() == 1);
    const int m = to_int(len.size(0));
    const int64_t rows = table_rows(table, m, dev);
    fits(len, at::kInt, {m}, dev);
    fits(new_len, at::kInt, {m}, dev);
    fits(refs, at::kInt, {refs.size(0)}, dev);
    c10::cuda::CUDAGuard guard(dev);
    const rf_status st = rf_pages_release(
        ptr<int32_t>(&table), rows, ptr<int32_t>(&len), ptr<int32_t>(new_len), m,
        ptr<int32_t>(&refs), to_int(table.size(1)), as_int(a[3]), to_int(refs.size(0)),
        stream_of(dev));
    return results(st, {});
  } catch (const Misfit&) {
    return misfit();
  }
  END_HANDLE_TH_ERRORS
}

#define RF_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RF_METHOD(attn_paged), RF_METHOD(kv_append_paged), RF_METHOD(draft_verify),
                         RF_METHOD(tree_mask), RF_METHOD(tree_accept), RF_METHOD(sample_rows),
                         RF_METHOD(kv_compact_paged), RF_METHOD(kv_copy_pages),
                         RF_METHOD(pages_fork), RF_METHOD(pages_grow), RF_METHOD(pages_release),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rf_serving", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rf_serving() { return PyModule_Create(&module); }
