// The common case of the paged-cache calls of the Python binding, without its
// marshalling in Python: checks of tensors that have the right shape, type and
// device, allocation of outputs and workspace, and the library call, in one
// native function each.
//
// A function returns its tensors; or the library's status, an int, where that
// is not MIMO_OK; or None where the arguments are not the plain case (another
// device than the current one, a wrong shape, type or layout): the Python
// wrapper of the same call then takes over and says what is wrong.  The
// library's entry points come in as addresses, so that this module works with
// whichever build of the library the package has loaded.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "../../include/mimo_attn.h"

namespace {

decltype(&mimo_attn_paged_attention) g_attention;
decltype(&mimo_attn_paged_attention_workspace_size) g_attention_ws;
decltype(&mimo_attn_paged_append) g_append;
decltype(&mimo_attn_page_hold) g_hold;
decltype(&mimo_attn_page_hold_workspace_size) g_hold_ws;
decltype(&mimo_attn_page_fork) g_fork;
decltype(&mimo_attn_page_compact) g_compact;
decltype(&mimo_attn_page_compact_workspace_size) g_compact_ws;
decltype(&mimo_attn_page_copy) g_copy;

using Sizes = c10::IntArrayRef;
constexpr auto kBF16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

// The arguments of one call; `plain` falls to false at the first that is not
// of the common case.
struct Args {
  PyObject* const* a;
  bool plain = true;
  c10::Device dev{c10::kCPU};

  // at::empty without its dispatch.
  at::Tensor empty(Sizes sizes, c10::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
  }
  // A tensor that must be there; the first one sets the device.
  const at::Tensor* tensor(int i) {
    if (!plain || !THPVariable_Check(a[i])) {
      plain = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (dev.is_cpu()) {
      dev = t.device();
      if (!dev.is_cuda() || dev.index() != c10::cuda::current_device()) plain = false;
    }
    return &t;
  }
  void* check(const at::Tensor& t, c10::ScalarType type, Sizes sizes) {
    if (t.scalar_type() == type && t.device() == dev && t.sizes() == sizes && t.is_contiguous()) return t.data_ptr();
    plain = false;
    return nullptr;
  }
  void* given(int i, c10::ScalarType type, Sizes sizes) {
    const at::Tensor* t = tensor(i);
    return t ? check(*t, type, sizes) : nullptr;
  }
  // A tensor or None (a null address).
  void* optional(int i, c10::ScalarType type, Sizes sizes) {
    return !plain || a[i] == Py_None ? nullptr : given(i, type, sizes);
  }
  // A tensor or None, which makes a new one.
  void* output(int i, c10::ScalarType type, Sizes sizes, at::Tensor& t) {
    if (!plain) return nullptr;
    if (a[i] != Py_None) {
      const at::Tensor* x = tensor(i);
      if (!x) return nullptr;
      t = *x;
      return check(t, type, sizes);
    }
    t = empty(sizes, type);
    return t.data_ptr();
  }
  // The caller's workspace, or a new one of `need` bytes.
  void* workspace(int i, size_t need, at::Tensor& t, size_t& bytes) {
    bytes = 0;
    if (!plain) return nullptr;
    if (a[i] != Py_None) {
      const at::Tensor* x = tensor(i);
      if (!x || x->device() != dev || !x->is_contiguous()) {
        plain = false;
        return nullptr;
      }
      t = *x;
      bytes = t.nbytes();
      return t.data_ptr();
    }
    if (!need) return nullptr;
    t = empty({(int64_t)need}, at::kByte);
    bytes = need;
    return t.data_ptr();
  }
  int integer(int i) {
    if (!plain) return 0;
    const long v = PyLong_Check(a[i]) ? PyLong_AsLong(a[i]) : LONG_MIN;
    if (v < INT_MIN || v > INT_MAX || PyErr_Occurred()) {
      PyErr_Clear();
      plain = false;
    }
    return (int)v;
  }
  float number(int i) {
    if (!plain) return 0.f;
    const double v = PyFloat_AsDouble(a[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      plain = false;
    }
    return (float)v;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }
};

PyObject* wrapped(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(T));
  int i = 0;
  ((PyTuple_SET_ITEM(r, i++, wrapped(t))), ...);
  return r;
}

mimo_attn_dims_t dims_of(int64_t hq, int64_t hkv, int64_t dqk, int64_t dv) {
  mimo_attn_dims_t d = {};
  d.num_heads_q = (int)hq;
  d.num_heads_kv = (int)hkv;
  d.head_dim_qk = (int)dqk;
  d.head_dim_v = (int)dv;
  d.v_scale = 1.f;
  return d;
}

bool fits(std::initializer_list<int64_t> v) {
  for (int64_t x : v)
    if (x > INT_MAX) return false;
  return true;
}

#define MIMO_NOT_PLAIN() Py_RETURN_NONE
#define MIMO_STATUS(st) \
  if (const int status_ = (st)) return PyLong_FromLong(status_)

// q, k_pages, v_pages, block_table, cu_seqlens_q, seqlens, max_seqlen_q, window, sinks, out, lse, workspace,
// fp32 output, softmax_scale (0: the default), v_scale, with lse
PyObject* paged_attention(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 16) MIMO_NOT_PLAIN();
  Args a{argv};
  const at::Tensor *q = a.tensor(0), *k = a.tensor(1), *v = a.tensor(2), *table = a.tensor(3);
  if (!a.plain || q->dim() != 3 || k->dim() != 4 || v->dim() != 4 || table->dim() != 2) MIMO_NOT_PLAIN();
  const int64_t nt = q->size(0), hq = q->size(1), dqk = q->size(2);
  const int64_t P = k->size(0), ps = k->size(1), hkv = k->size(2), dv = v->size(3), B = table->size(0), M = table->size(1);
  if (!fits({nt, hq, P, ps, hkv, B, M})) MIMO_NOT_PLAIN();
  void *qp = a.check(*q, kBF16, {nt, hq, dqk}), *kp = a.check(*k, kBF16, {P, ps, hkv, dqk}),
       *vp = a.check(*v, kBF16, {P, ps, hkv, dv}), *tp = a.check(*table, kI32, {B, M}), *cp = a.given(4, kI32, {B + 1}),
       *lp = a.given(5, kI32, {B}), *sp = a.optional(8, kF32, {hq});
  const int most = a.integer(6), window = a.integer(7);
  mimo_attn_dims_t d = dims_of(hq, hkv, dqk, dv);
  const bool f32 = argv[12] == Py_True;
  d.out_dtype = f32 ? MIMO_DTYPE_F32 : MIMO_DTYPE_BF16;
  d.softmax_scale = a.number(13);
  d.v_scale = a.number(14);
  if (!a.plain || hkv <= 0) MIMO_NOT_PLAIN();
  at::Tensor out, lse, ws;
  void* op = a.output(9, f32 ? kF32 : kBF16, {nt, hq, dv}, out);
  void* ep = PyObject_IsTrue(argv[15]) == 1 || argv[10] != Py_None ? a.output(10, kF32, {hq, nt}, lse) : nullptr;
  size_t bytes;
  void* wp = a.workspace(11, g_attention_ws(&d, (int)B, (int)nt, most, window), ws, bytes);
  if (!a.plain) MIMO_NOT_PLAIN();
  MIMO_STATUS(g_attention(&d, qp, kp, vp, (const int32_t*)tp, (const int32_t*)cp, (const int32_t*)lp, (int)B, (int)nt,
                          most, (int)P, (int)ps, (int)M, window, (const float*)sp, op, (float*)ep, wp, bytes,
                          a.stream()));
  return tuple(out, lse);
  END_HANDLE_TH_ERRORS
}

// q, k_new, v_new, k_pages, v_pages, block_table, cu_seqlens_q, seqlens, rope_theta, rotary_dim, q_out
PyObject* paged_append(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 11) MIMO_NOT_PLAIN();
  Args a{argv};
  const at::Tensor *q = a.tensor(0), *k = a.tensor(3), *v = a.tensor(4), *table = a.tensor(5);
  if (!a.plain || q->dim() != 3 || k->dim() != 4 || v->dim() != 4 || table->dim() != 2) MIMO_NOT_PLAIN();
  const int64_t nt = q->size(0), hq = q->size(1), dqk = q->size(2);
  const int64_t P = k->size(0), ps = k->size(1), hkv = k->size(2), dv = v->size(3), B = table->size(0), M = table->size(1);
  if (!fits({nt, hq, P, ps, hkv, B, M})) MIMO_NOT_PLAIN();
  void *qp = a.check(*q, kBF16, {nt, hq, dqk}), *knp = a.given(1, kBF16, {nt, hkv, dqk}),
       *vnp = a.given(2, kBF16, {nt, hkv, dv}), *kp = a.check(*k, kBF16, {P, ps, hkv, dqk}),
       *vp = a.check(*v, kBF16, {P, ps, hkv, dv}), *tp = a.check(*table, kI32, {B, M}), *cp = a.given(6, kI32, {B + 1}),
       *lp = a.given(7, kI32, {B});
  const float theta = a.number(8);
  const int rotary = a.integer(9);
  at::Tensor out;
  void* op = a.output(10, kBF16, {nt, hq, dqk}, out);
  if (!a.plain) MIMO_NOT_PLAIN();
  const mimo_attn_dims_t d = dims_of(hq, hkv, dqk, dv);
  MIMO_STATUS(g_append(&d, qp, op, knp, vnp, kp, vp, (const int32_t*)tp, (const int32_t*)cp, (const int32_t*)lp, (int)B,
                       (int)nt, (int)P, (int)ps, (int)M, theta, rotary, a.stream()));
  return argv[10] != Py_None ? Py_NewRef(argv[10]) : wrapped(out);
  END_HANDLE_TH_ERRORS
}

// page_refs, block_table, seqlens, page_size, first, write_from, refs_out, table_out, moves, info, workspace
PyObject* page_hold(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 11) MIMO_NOT_PLAIN();
  Args a{argv};
  const at::Tensor *refs = a.tensor(0), *table = a.tensor(1);
  if (!a.plain || refs->dim() != 1 || table->dim() != 2) MIMO_NOT_PLAIN();
  const int64_t P = refs->size(0), B = table->size(0), M = table->size(1);
  if (!fits({P, B, M})) MIMO_NOT_PLAIN();
  void *rp = a.check(*refs, kI32, {P}), *tp = a.check(*table, kI32, {B, M}), *lp = a.given(2, kI32, {B}),
       *fp = a.optional(4, kI32, {B}), *wp = a.optional(5, kI32, {B});
  const int ps = a.integer(3);
  at::Tensor refs_out, table_out, moves, info, ws;
  void *ro = a.output(6, kI32, {P}, refs_out), *to = a.output(7, kI32, {B, M}, table_out),
       *mo = a.output(8, kI32, {B, 2}, moves), *io = a.output(9, kI32, {2}, info);
  size_t bytes;
  void* sp = a.workspace(10, g_hold_ws((int)P), ws, bytes);
  if (!a.plain) MIMO_NOT_PLAIN();
  MIMO_STATUS(g_hold((const int32_t*)rp, (int)P, (const int32_t*)tp, (int)B, (int)M, ps, (const int32_t*)lp,
                     (const int32_t*)fp, (const int32_t*)wp, (int32_t*)ro, (int32_t*)to, (int32_t*)mo, (int32_t*)io, sp,
                     bytes, a.stream()));
  return tuple(refs_out, table_out, moves, info);
  END_HANDLE_TH_ERRORS
}

// page_refs, block_table, parent, refs_out, table_out
PyObject* page_fork(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 5) MIMO_NOT_PLAIN();
  Args a{argv};
  const at::Tensor *refs = a.tensor(0), *table = a.tensor(1), *parent = a.tensor(2);
  if (!a.plain || refs->dim() != 1 || table->dim() != 2 || parent->dim() != 1) MIMO_NOT_PLAIN();
  const int64_t P = refs->size(0), B = table->size(0), M = table->size(1), n = parent->size(0);
  if (!fits({P, B, M, n})) MIMO_NOT_PLAIN();
  void *rp = a.check(*refs, kI32, {P}), *tp = a.check(*table, kI32, {B, M}), *pp = a.check(*parent, kI32, {n});
  at::Tensor refs_out, table_out;
  void *ro = a.output(3, kI32, {P}, refs_out), *to = a.output(4, kI32, {n, M}, table_out);
  if (!a.plain) MIMO_NOT_PLAIN();
  MIMO_STATUS(g_fork((const int32_t*)rp, (int)P, (const int32_t*)tp, (int)B, (int)M, (const int32_t*)pp, (int)n,
                     (int32_t*)ro, (int32_t*)to, a.stream()));
  return tuple(refs_out, table_out);
  END_HANDLE_TH_ERRORS
}

// page_refs, block_table, max_moves, refs_out, table_out, moves, info, workspace
PyObject* page_compact(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 8) MIMO_NOT_PLAIN();
  Args a{argv};
  const at::Tensor *refs = a.tensor(0), *table = a.tensor(1);
  if (!a.plain || refs->dim() != 1 || table->dim() != 2) MIMO_NOT_PLAIN();
  const int64_t P = refs->size(0), B = table->size(0), M = table->size(1);
  const int most = a.integer(2);
  if (!a.plain || most < 0 || !fits({P, B, M})) MIMO_NOT_PLAIN();
  void *rp = a.check(*refs, kI32, {P}), *tp = a.check(*table, kI32, {B, M});
  at::Tensor refs_out, table_out, moves, info, ws;
  void *ro = a.output(3, kI32, {P}, refs_out), *to = a.output(4, kI32, {B, M}, table_out),
       *mo = a.output(5, kI32, {most, 2}, moves), *io = a.output(6, kI32, {2}, info);
  size_t bytes;
  void* sp = a.workspace(7, g_compact_ws((int)P), ws, bytes);
  if (!a.plain) MIMO_NOT_PLAIN();
  MIMO_STATUS(g_compact((const int32_t*)rp, (int)P, (const int32_t*)tp, (int)B, (int)M, most, (int32_t*)ro, (int32_t*)to,
                        (int32_t*)mo, (int32_t*)io, sp, bytes, a.stream()));
  return tuple(refs_out, table_out, moves, info);
  END_HANDLE_TH_ERRORS
}

// k_pages, v_pages, moves
PyObject* page_copy(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 3) MIMO_NOT_PLAIN();
  Args a{argv};
  const at::Tensor *k = a.tensor(0), *v = a.tensor(1), *moves = a.tensor(2);
  if (!a.plain || (k->dim() != 4 && k->dim() != 5) || v->dim() != k->dim() || moves->dim() != 2) MIMO_NOT_PLAIN();
  const int64_t layers = k->dim() == 5 ? k->size(0) : 1;
  const int64_t P = k->size(-4), ps = k->size(-3), hkv = k->size(-2), dqk = k->size(-1), dv = v->size(-1),
                n = moves->size(0);
  if (!fits({layers, P, ps, hkv, n})) MIMO_NOT_PLAIN();
  auto vs = k->sizes().vec();
  vs.back() = dv;
  void *kp = a.check(*k, kBF16, k->sizes()), *vp = a.check(*v, kBF16, vs), *mp = a.check(*moves, kI32, {n, 2});
  if (!a.plain) MIMO_NOT_PLAIN();
  const mimo_attn_dims_t d = dims_of(hkv, hkv, dqk, dv);
  MIMO_STATUS(g_copy(&d, kp, vp, (int)layers, (int)P, (int)ps, (const int32_t*)mp, (int)n, a.stream()));
  return PyTuple_Pack(2, argv[0], argv[1]);
  END_HANDLE_TH_ERRORS
}

// The addresses of the entry points, in the order of the globals above.
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  void* f[9];
  if (argc != 9) {
    PyErr_SetString(PyExc_TypeError, "bind takes 9 addresses");
    return nullptr;
  }
  for (int i = 0; i < 9; ++i) {
    f[i] = PyLong_AsVoidPtr(argv[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_attention = (decltype(g_attention))f[0];
  g_attention_ws = (decltype(g_attention_ws))f[1];
  g_append = (decltype(g_append))f[2];
  g_hold = (decltype(g_hold))f[3];
  g_hold_ws = (decltype(g_hold_ws))f[4];
  g_fork = (decltype(g_fork))f[5];
  g_compact = (decltype(g_compact))f[6];
  g_compact_ws = (decltype(g_compact_ws))f[7];
  g_copy = (decltype(g_copy))f[8];
  Py_RETURN_NONE;
}

#define MIMO_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MIMO_METHOD(bind),         MIMO_METHOD(paged_attention), MIMO_METHOD(paged_append),
                         MIMO_METHOD(page_hold),    MIMO_METHOD(page_fork),       MIMO_METHOD(page_compact),
                         MIMO_METHOD(page_copy),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_call() { return PyModule_Create(&module); }
