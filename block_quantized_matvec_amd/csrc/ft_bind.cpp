// ft_bind.cpp -- argument marshalling of the operators of a decoder layer's step (ft.rope, ft.kv_store_rope, ft.kv_load,
// ft.norm, ft.lora): torch tensors into pointers, sizes and strides, outputs allocated, a status raised.  Checks and calls
// only, no arithmetic.  In Python the same took 4 to 6 us a call, longer than most of these kernels run at a
// decode step; here it takes 0.4 to 0.6.
#include <torch/csrc/python_headers.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <optional>

#include "ft.h"

namespace {

using at::Tensor;
PyObject* g_error = nullptr;   // ft.FtError

// The library's entry points, as ft.py loaded them (from wherever: this extension does not link to a copy of its own)
struct Library {
  decltype(&ft_rope) rope;
  decltype(&ft_kv_store_rope) kv_store_rope;
  decltype(&ft_kv_load) kv_load;
  decltype(&ft_norm) norm;
  decltype(&ft_lora) lora;
  decltype(&ft_block_elems) block_elems;
  decltype(&ft_block_bytes) block_bytes;
} g_lib = {};

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, not ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

ft_float float_type(at::ScalarType type, const char* name) {
  switch (type) {
    case at::kFloat: return FT_F32;
    case at::kHalf: return FT_F16;
    case at::kBFloat16: return FT_BF16;
    default: TORCH_CHECK_VALUE(false, name, " must be float32, float16 or bfloat16, not ", type);
  }
}
// pointer of a contiguous tensor of this type, shape and device (null: not given)
void* plain(const Tensor* t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device dev) {
  if (!t) return nullptr;
  TORCH_CHECK_VALUE(t->scalar_type() == type && t->sizes() == shape && t->device() == dev && t->is_contiguous(), name,
                    " must be a contiguous ", type, " tensor of shape ", shape, " on ", dev, ", not ", t->dtype(), " ", t->sizes(), " on ",
                    t->device());
  return t->data_ptr();
}
// strides of a (tokens, heads, dim) tensor, and of a (rows, width) one
struct Rows {
  int64_t token, head;
};
Rows rows(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == type && t.device() == dev && t.stride(2) == 1, name, " must be ", shape, " ", type,
                    " on ", dev, " with unit element stride, not ", t.sizes(), " ", t.dtype(), " on ", t.device());
  return {t.stride(0), t.stride(1)};
}
int64_t line(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == type && t.device() == dev && (t.stride(1) == 1 || shape[1] <= 1), name, " must be ",
                    shape, " ", type, " on ", dev, " with unit element stride, not ", t.sizes(), " ", t.dtype(), " on ", t.device());
  return shape[0] > 1 ? t.stride(0) : shape[1];
}
Tensor empty(at::IntArrayRef shape, const Tensor& like) { return at::empty(shape, like.options().requires_grad(false)); }

// The caller's stream (None: the current one of the device), with the device as the library's current one, and the
// stream as torch's current one: tensors made meanwhile are that stream's, as under torch.cuda.stream.  (Memory that the
// current stream gave back may still be in use there; the allocator hands it out to tensors of that stream only.)
struct On {
  c10::OptionalDeviceGuard guard;
  ft_stream_t stream;
  std::optional<c10::hip::HIPStream> before;
  On(const On&) = delete;
  ~On() {
    if (before) c10::hip::setCurrentHIPStream(*before);
  }
  On(at::Device dev, PyObject* o) : guard(dev) {
    if (o == Py_None) {
      stream = c10::hip::getCurrentHIPStream(dev.index()).stream();
      return;
    }
    // any object with the two attributes of a torch stream that name it: its device and its handle
    const auto held = [](PyObject* p) {
      if (!p) throw python_error();
      return THPObjectPtr(p);
    };
    THPObjectPtr at = held(PyObject_GetAttrString(o, "device")), want = held(THPDevice_New(dev));
    const int same = PyObject_RichCompareBool(at.get(), want.get(), Py_EQ);
    if (same < 0) throw python_error();
    TORCH_CHECK_VALUE(same, "the stream is on another device than the tensors, which are on ", dev);
    THPObjectPtr handle = held(PyObject_GetAttrString(o, "cuda_stream"));
    stream = (ft_stream_t)(uintptr_t)PyLong_AsUnsignedLongLongMask(handle.get());
    if (PyErr_Occurred()) throw python_error();
    before = c10::hip::getCurrentHIPStream(dev.index());
    c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal((hipStream_t)stream, dev.index()));
  }
};
template <class Call>
void run(const char* name, Call&& call) {
  ft_status s;
  Py_BEGIN_ALLOW_THREADS
  s = call();
  Py_END_ALLOW_THREADS
  if (s == FT_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, name);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}
PyObject* given(PyObject* o, const Tensor& t) {   // the caller's object, or the new tensor
  if (o == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(o);
  return o;
}

ft_rotation rotation(PyObject* table, PyObject* positions, PyObject* interleaved, int64_t t, at::Device dev) {
  const Tensor& tab = tensor(table, "table");
  const Tensor& pos = tensor(positions, "positions");
  TORCH_CHECK_VALUE(tab.dim() == 2, "table must be (n_pos, rot_dim)");
  ft_rotation r = {};
  r.table = (const float*)plain(&tab, "table", at::kFloat, tab.sizes(), dev);
  r.positions = (const int32_t*)plain(&pos, "positions", at::kInt, {t}, dev);
  r.n_pos = tab.size(0);
  r.rot_dim = tab.size(1);
  r.interleaved = truth(interleaved);
  return r;
}

// x, positions, table, interleaved, weight, eps, out, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Tensor& x = tensor(a[0], "x");
  TORCH_CHECK_VALUE(x.is_cuda() && x.dim() == 3, "x must be a device tensor (t, heads, dim)");
  const ft_float ty = float_type(x.scalar_type(), "x");
  const at::Device dev = x.device();
  const auto type = x.scalar_type();
  const int64_t t = x.size(0), heads = x.size(1), dim = x.size(2);
  const Rows xs = rows(x, "x", x.sizes(), type, dev);
  const ft_rotation r = rotation(a[2], a[1], a[3], t, dev);
  const float* w = (const float*)plain(maybe(a[4], "weight"), "weight", at::kFloat, {dim}, dev);
  const double eps = number(a[5]);
  const On on(dev, a[7]);
  const Tensor out = a[6] == Py_None ? empty(x.sizes(), x) : tensor(a[6], "out");
  const Rows os = rows(out, "out", x.sizes(), type, dev);
  run("ft_rope", [&] {
    return g_lib.rope(&r, ty, x.data_ptr(), xs.token, xs.head, t, heads, dim, w, eps, out.data_ptr(), os.token, os.head, on.stream);
  });
  return given(a[6], out);
  END_HANDLE_TH_ERRORS
}

// address of the cache's structure, its k_pages, q, k, v, slots, positions, table, interleaved, q_weight, k_weight, eps, q_out, stream
PyObject* kv_store_rope(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const auto* cache = (const ft_kv_cache*)(uintptr_t)whole(a[0]);
  const at::Device dev = tensor(a[1], "k_pages").device();
  const Tensor& k = tensor(a[3], "k");
  const Tensor& v = tensor(a[4], "v");
  const Tensor& slots = tensor(a[5], "slots");
  const ft_float ty = float_type(k.scalar_type(), "k");
  const auto type = k.scalar_type();
  TORCH_CHECK_VALUE(k.dim() == 3, "k must be (t, n_kv_head, head_dim)");
  const int64_t t = k.size(0), dim = cache->head_dim;
  const int64_t shape[3] = {t, cache->n_kv_head, dim};
  const Rows ks = rows(k, "k", shape, type, dev), vs = rows(v, "v", shape, type, dev);
  const ft_rotation r = rotation(a[7], a[6], a[8], t, dev);
  ft_qkv_rows o = {};
  o.k = k.data_ptr();
  o.k_token = ks.token;
  o.k_head = ks.head;
  o.v = v.data_ptr();
  o.v_token = vs.token;
  o.v_head = vs.head;
  o.k_weight = (const float*)plain(maybe(a[10], "k_weight"), "k_weight", at::kFloat, {dim}, dev);
  o.eps = number(a[11]);
  const void* at_slots = plain(&slots, "slots", at::kLong, {t}, dev);
  const On on(dev, a[13]);
  Tensor out;
  if (a[2] != Py_None) {
    const Tensor& q = tensor(a[2], "q");
    TORCH_CHECK_VALUE(q.dim() == 3, "q must be (t, heads, head_dim)");
    const int64_t qshape[3] = {t, q.size(1), dim};
    const Rows qs = rows(q, "q", qshape, type, dev);
    out = a[12] == Py_None ? empty(qshape, q) : tensor(a[12], "q_out");
    const Rows os = rows(out, "q_out", qshape, type, dev);
    o.q = q.data_ptr();
    o.q_token = qs.token;
    o.q_head = qs.head;
    o.n_head = q.size(1);
    o.q_weight = (const float*)plain(maybe(a[9], "q_weight"), "q_weight", at::kFloat, {dim}, dev);
    o.q_out = out.data_ptr();
    o.out_token = os.token;
    o.out_head = os.head;
  } else {
    TORCH_CHECK_VALUE(a[9] == Py_None && a[12] == Py_None, "q_out and q_weight are q's");
  }
  run("ft_kv_store_rope", [&] { return g_lib.kv_store_rope(cache, &r, ty, &o, (const int64_t*)at_slots, t, on.stream); });
  if (a[2] == Py_None) Py_RETURN_NONE;
  return given(a[12], out);
  END_HANDLE_TH_ERRORS
}

// address of the cache's structure, its k_pages, slots, dtype of new tensors, k, v, stream
PyObject* kv_load(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const auto* cache = (const ft_kv_cache*)(uintptr_t)whole(a[0]);
  const Tensor& pages = tensor(a[1], "k_pages");
  const at::Device dev = pages.device();
  const Tensor& slots = tensor(a[2], "slots");
  TORCH_CHECK_VALUE(slots.dim() == 1, "slots must be (t,)");
  const Tensor *ko = maybe(a[4], "k"), *vo = maybe(a[5], "v");
  TORCH_CHECK_VALUE(ko || vo || THPDtype_Check(a[3]), "dtype must be float32, float16 or bfloat16");
  const auto type = ko ? ko->scalar_type() : vo ? vo->scalar_type() : reinterpret_cast<THPDtype*>(a[3])->scalar_type;
  const int64_t t = slots.size(0);
  const int64_t shape[3] = {t, cache->n_kv_head, cache->head_dim};
  const ft_float ty = float_type(type, "dtype");
  const auto fresh = pages.options().dtype(type).requires_grad(false);
  const On on(dev, a[6]);
  const Tensor k = ko ? *ko : at::empty(shape, fresh), v = vo ? *vo : at::empty(shape, fresh);
  const Rows ks = rows(k, "k", shape, type, dev), vs = rows(v, "v", shape, type, dev);
  const void* at_slots = plain(&slots, "slots", at::kLong, {t}, dev);
  run("ft_kv_load", [&] {
    return g_lib.kv_load(cache, (const int64_t*)at_slots, t, ty, k.data_ptr(), ks.token, ks.head, v.data_ptr(), vs.token, vs.head, on.stream);
  });
  PyObject* pk = given(a[4], k);
  return Py_BuildValue("(NN)", pk, given(a[5], v));
  END_HANDLE_TH_ERRORS
}

// x, weight, bias, residual, post_weight, post_bias, post (None: by the weights), gate, scale, layer, eps, act (-1: none), rows (None:
// without an act), r, out, xq, stream
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Tensor& x = tensor(a[0], "x");
  TORCH_CHECK_VALUE(x.is_cuda() && x.dim() == 2, "x must be a device tensor (t, width)");
  const ft_float ty = float_type(x.scalar_type(), "x");
  const at::Device dev = x.device();
  const auto type = x.scalar_type();
  const int64_t t = x.size(0), width = x.size(1);
  const at::IntArrayRef shape = x.sizes();
  ft_norm_opts o = {};
  const auto vec = [&](int i, const char* name) { return (const float*)plain(maybe(a[i], name), name, at::kFloat, {width}, dev); };
  o.weight = vec(1, "weight");
  o.bias = vec(2, "bias");
  o.post_weight = vec(4, "post_weight");
  o.post_bias = vec(5, "post_bias");
  o.post = a[6] == Py_None ? o.post_weight || o.post_bias : truth(a[6]);
  o.scale = (float)number(a[8]);
  TORCH_CHECK_VALUE(o.scale != 0.0f, "scale must not be 0");
  o.layer = truth(a[9]);
  o.eps = number(a[10]);
  const int64_t ldx = line(x, "x", shape, type, dev);
  if (const Tensor* p = maybe(a[3], "residual")) {
    o.ld_residual = line(*p, "residual", shape, type, dev);
    o.residual = p->data_ptr();
  }
  if (const Tensor* p = maybe(a[7], "gate")) {
    const bool flat = p->dim() == 1;
    TORCH_CHECK_VALUE((flat || p->dim() == 2) && p->scalar_type() == type && p->device() == dev && p->size(-1) == width &&
                          (flat || p->size(0) == 1 || p->size(0) == t) && (width <= 1 || p->stride(-1) == 1),
                      "gate must be (1 or ", t, ", ", width, ") ", type, " on ", dev, " with unit element stride, not ", p->sizes(), " ",
                      p->dtype(), " on ", p->device());
    if (!flat && p->size(0) > 1) o.ld_gate = p->stride(0);   // 0: one row for all
    o.gate = p->data_ptr();
  }
  const On on(dev, a[16]);
  Tensor r, out, xq;
  bool made_r = false;
  if (a[13] != Py_None) {
    r = tensor(a[13], "r");
    o.ld_r = line(r, "r", shape, type, dev);
  } else if (o.post || o.residual || o.gate || o.scale != 1.0f) {
    r = empty(shape, x);
    o.ld_r = width;
    made_r = true;
  }
  if (r.defined()) o.r = r.data_ptr();
  const int64_t act = whole(a[11]);
  if (a[14] != Py_None) {
    out = tensor(a[14], "out");
    o.ld_out = line(out, "out", shape, type, dev);
  } else if (a[12] == Py_None ? act < 0 : truth(a[12])) {
    out = empty(shape, x);
    o.ld_out = width;
  }
  if (out.defined()) o.out = out.data_ptr();
  if (act >= 0) {
    o.act = (ft_type)act;
    const int64_t size[2] = {t, width / g_lib.block_elems(o.act) * (int64_t)g_lib.block_bytes(o.act)};
    xq = a[15] == Py_None ? at::empty(size, x.options().dtype(at::kByte).requires_grad(false)) : tensor(a[15], "xq");
    o.xq = plain(&xq, "xq", at::kByte, size, dev);
  } else {
    TORCH_CHECK_VALUE(a[15] == Py_None, "xq needs an act");
  }
  run("ft_norm", [&] { return g_lib.norm(ty, x.data_ptr(), ldx, t, width, &o, on.stream); });
  PyObject* pr = made_r ? THPVariable_Wrap(r) : a[13] == Py_None ? a[0] : a[13];
  if (!made_r) Py_INCREF(pr);
  PyObject* po = out.defined() ? given(a[14], out) : Py_NewRef(Py_None);
  PyObject* pq = xq.defined() ? given(a[15], xq) : Py_NewRef(Py_None);
  return Py_BuildValue("(NNN)", pr, po, pq);
  END_HANDLE_TH_ERRORS
}

// x, a, b, ids, y, scales, ranks, out, workspace, stream
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Tensor& x = tensor(a[0], "x");
  const Tensor& wa = tensor(a[1], "a");
  const Tensor& wb = tensor(a[2], "b");
  const Tensor& ids = tensor(a[3], "ids");
  TORCH_CHECK_VALUE(x.is_cuda() && x.dim() == 2 && wa.dim() == 3 && wb.dim() == 3,
                    "x must be a device tensor (t, k), a (n_adapter, rank, k), b (n_adapter, n, rank)");
  const ft_float tx = float_type(x.scalar_type(), "x"), tw = float_type(wa.scalar_type(), "a");
  const at::Device dev = x.device();
  const int64_t t = x.size(0), k = x.size(1), many = wa.size(0), rank = wa.size(1), n = wb.size(1);
  const int64_t oshape[2] = {t, n};
  const int64_t ldx = line(x, "x", x.sizes(), x.scalar_type(), dev);
  const void* pa = plain(&wa, "a", wa.scalar_type(), {many, rank, k}, dev);
  const void* pb = plain(&wb, "b", wa.scalar_type(), {many, n, rank}, dev);
  const void* pi = plain(&ids, "ids", at::kInt, {t}, dev);
  const Tensor* y = maybe(a[4], "y");
  const int64_t ldy = y ? line(*y, "y", oshape, at::kFloat, dev) : 0;
  ft_lora_opts o = {};
  o.scales = (const float*)plain(maybe(a[5], "scales"), "scales", at::kFloat, {many}, dev);
  o.ranks = (const int32_t*)plain(maybe(a[6], "ranks"), "ranks", at::kInt, {many}, dev);
  const On on(dev, a[9]);
  const Tensor out = a[7] == Py_None ? at::empty(oshape, x.options().dtype(at::kFloat).requires_grad(false)) : tensor(a[7], "out");
  const int64_t ldo = line(out, "out", oshape, at::kFloat, dev);
  if (const Tensor* w = maybe(a[8], "workspace")) {
    TORCH_CHECK_VALUE(w->device() == dev && w->is_contiguous(), "workspace must be contiguous on ", dev);
    o.workspace = w->data_ptr();
    o.workspace_bytes = w->nbytes();
  }
  run("ft_lora", [&] {
    return g_lib.lora(tx, x.data_ptr(), ldx, t, k, tw, pa, pb, many, rank, n, (const int32_t*)pi, y ? (const float*)y->data_ptr() : nullptr, ldy,
                   (float*)out.data_ptr(), ldo, &o, on.stream);
  });
  return given(a[7], out);
  END_HANDLE_TH_ERRORS
}

// FtError, the addresses of Library's entry points in their order
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  Library l;
  l.rope = (decltype(l.rope))whole(a[1]);
  l.kv_store_rope = (decltype(l.kv_store_rope))whole(a[2]);
  l.kv_load = (decltype(l.kv_load))whole(a[3]);
  l.norm = (decltype(l.norm))whole(a[4]);
  l.lora = (decltype(l.lora))whole(a[5]);
  l.block_elems = (decltype(l.block_elems))whole(a[6]);
  l.block_bytes = (decltype(l.block_bytes))whole(a[7]);
  g_lib = l;
  Py_INCREF(a[0]);
  Py_XDECREF(g_error);
  g_error = a[0];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* m, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "takes %d arguments, not %zd", N, n);
  return F(m, a, n);
}
PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void*)counted<setup, 8>, METH_FASTCALL, nullptr},
    {"rope", (PyCFunction)(void*)counted<rope, 8>, METH_FASTCALL, nullptr},
    {"kv_store_rope", (PyCFunction)(void*)counted<kv_store_rope, 14>, METH_FASTCALL, nullptr},
    {"kv_load", (PyCFunction)(void*)counted<kv_load, 7>, METH_FASTCALL, nullptr},
    {"norm", (PyCFunction)(void*)counted<norm, 17>, METH_FASTCALL, nullptr},
    {"lora", (PyCFunction)(void*)counted<lora, 10>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ft_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ft_bind(void) { return PyModule_Create(&module); }
