// The 8-bit operators of hyb.py for a call that needs nothing special: plain CUDA
// tensors on the current device and stream and a workspace at hand.  A step of a
// decode loop makes many of these calls, and the kernels of small ones take less
// time than the binding's Python code and ctypes do (matmul_fp8: 18 us, 3.4 through here;
// cache_attention: 26 and 4.6).
//
// A function returns its outputs, an int where the library refused the call (the
// status), or None where the call is not of this kind: hyb.py then goes its own
// way, which also says what is wrong with the arguments.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "hyb.h"

namespace {

const at::Tensor *tensor_of(PyObject *o, int64_t index) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor &t = THPVariable_Unpack(o);
  const at::Device d = t.device();
  return d.is_cuda() && d.index() == index && t.layout() == at::kStrided ? &t : nullptr;
}
bool int_of(PyObject *o, int64_t &v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}
// the device that a weight or a cache, given as its tensors, has to be on: `o`,
// or with None the first tensor's
bool index_of(PyObject *o, PyObject *tensors, int64_t &index) {
  if (o != Py_None) return int_of(o, index);
  if (!PyTuple_CheckExact(tensors) || PyTuple_GET_SIZE(tensors) < 1 ||
      !THPVariable_CheckExact(PyTuple_GET_ITEM(tensors, 0)))
    return false;
  const at::Device d = THPVariable_Unpack(PyTuple_GET_ITEM(tensors, 0)).device();
  index = d.is_cuda() ? d.index() : -1;
  return true;
}
bool current(int64_t index) { return index >= 0 && c10::cuda::current_device() == index; }
hyb_stream_t stream_of(int64_t index) {
  return (hyb_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
}
at::Device cuda(int64_t index) { return at::Device(at::kCUDA, (c10::DeviceIndex)index); }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

template <typename F>
int without_gil(F &&f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}
PyObject *pair(at::Tensor a, at::Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = x ? THPVariable_Wrap(std::move(b)) : nullptr;
  PyObject *r = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// A weight or a cache comes as its tensors and is read anew on every call: a
// tensor keeps its identity when its storage is replaced (Tensor.data, a module
// that is moved).

// (q, scale, n, k) of an Fp8Matrix
bool matrix_of(PyObject *o, int64_t index, hyb_fp8_matrix &A) {
  if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 4) return false;
  const at::Tensor *q = tensor_of(PyTuple_GET_ITEM(o, 0), index);
  const at::Tensor *s = tensor_of(PyTuple_GET_ITEM(o, 1), index);
  if (!q || !s || !int_of(PyTuple_GET_ITEM(o, 2), A.n) || !int_of(PyTuple_GET_ITEM(o, 3), A.k) ||
      A.n < 1 || A.k < 1 || A.n > INT32_MAX || A.k > INT32_MAX)
    return false;
  const int64_t nb = up(A.n, 128) / 128, kb = up(A.k, 128) / 128;
  if ((q->scalar_type() != at::kFloat8_e4m3fn && q->scalar_type() != at::kByte) || q->dim() != 2 ||
      q->size(0) != A.n || q->size(1) != A.k || (A.k > 1 && q->stride(1) != 1) ||
      (A.n > 1 && q->stride(0) < A.k))
    return false;
  if (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != nb || s->size(1) != kb ||
      (kb > 1 && s->stride(1) != 1) || (nb > 1 && s->stride(0) < kb))
    return false;
  A.q = (const uint8_t *)q->const_data_ptr();
  A.ldq = A.n > 1 ? q->stride(0) : up(A.k, 16);
  A.scale = s->const_data_ptr<float>();
  A.lds = std::max(s->stride(0), kb);
  return true;
}

// (k, v, k_scale, v_scale) of a Cache
bool cache_of(PyObject *o, int64_t index, hyb_cache &C) {
  if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 4) return false;
  const at::Tensor *t[4];
  for (int i = 0; i < 4; ++i)
    if (!(t[i] = tensor_of(PyTuple_GET_ITEM(o, i), index))) return false;
  const at::Tensor &k = *t[0], &v = *t[1];
  const bool i8 = k.scalar_type() == at::kChar;
  if ((!i8 && k.scalar_type() != at::kFloat8_e4m3fn) || v.scalar_type() != k.scalar_type() ||
      k.dim() != 4 || v.sizes() != k.sizes() || v.strides() != k.strides() || k.stride(3) != 1)
    return false;
  for (int i = 2; i < 4; ++i)
    if (t[i]->scalar_type() != at::kFloat || t[i]->sizes() != k.sizes().slice(0, 2) ||
        !t[i]->is_contiguous())
      return false;
  for (int64_t n : k.sizes())
    if (n > INT32_MAX) return false;
  C.k = (uint8_t *)k.data_ptr();
  C.v = (uint8_t *)v.data_ptr();
  C.k_scale = t[2]->data_ptr<float>();
  C.v_scale = t[3]->data_ptr<float>();
  C.type = i8 ? HYB_I8 : HYB_E4M3;
  C.num_pages = (int32_t)k.size(0);
  C.kv_heads = (int32_t)k.size(1);
  C.page_size = (int32_t)k.size(2);
  C.head_dim = (int32_t)k.size(3);
  C.stride_page = k.stride(0);
  C.stride_head = k.stride(1);
  C.stride_token = k.stride(2);
  return true;
}

// bf16 [rows][heads][dim] rows with dim contiguous; a single row's or head's
// stride says nothing
struct Rows {
  int64_t rows, heads, ld, hs;
};
bool rows_of(const at::Tensor &t, int64_t dim, Rows &r) {
  if (t.dim() != 3 || t.scalar_type() != at::kBFloat16 || t.size(2) != dim || t.stride(2) != 1)
    return false;
  r.rows = t.size(0);
  r.heads = t.size(1);
  r.ld = r.rows > 1 ? t.stride(0) : std::max(dim, r.heads * dim);
  r.hs = r.heads > 1 ? t.stride(1) : dim;
  return true;
}

bool sequences_of(PyObject *table, PyObject *lens, PyObject *off, PyObject *max_new, int64_t rows,
                  int64_t index, hyb_sequences &s) {
  const at::Tensor *t = tensor_of(table, index), *l = tensor_of(lens, index);
  if (!t || !l || t->scalar_type() != at::kInt || t->dim() != 2 || l->scalar_type() != at::kInt ||
      l->dim() != 1 || !l->is_contiguous())
    return false;
  const int64_t batch = t->size(0), pages = t->size(1);
  if (batch < 1 || pages < 1 || l->size(0) != batch || (pages > 1 && t->stride(1) != 1)) return false;
  if (batch > 1 && t->stride(0) < pages) return false;
  int64_t most = 0;
  if (off == Py_None) {
    if (max_new == Py_None)
      most = rows / batch;
    else if (!int_of(max_new, most))
      return false;
    if (rows != batch * most) return false;
    s.off = nullptr;
  } else {
    const at::Tensor *o = tensor_of(off, index);
    if (!o || o->scalar_type() != at::kInt || o->dim() != 1 || o->size(0) != batch + 1 ||
        !o->is_contiguous() || !int_of(max_new, most))
      return false;
    s.off = o->const_data_ptr<int32_t>();
  }
  if (batch > INT32_MAX || pages > INT32_MAX || most < 1 || most > INT32_MAX) return false;
  s.batch = (int32_t)batch;
  s.max_new = (int32_t)most;
  s.rows = rows;
  s.lens = l->const_data_ptr<int32_t>();
  s.page_table = t->const_data_ptr<int32_t>();
  s.max_pages = (int32_t)pages;
  s.table_stride = batch > 1 ? t->stride(0) : pages;
  return true;
}

// (X, block_rows, ws)
PyObject *quant_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3 || !THPVariable_CheckExact(a[0])) Py_RETURN_NONE;
  const at::Tensor &X = THPVariable_Unpack(a[0]);
  const int64_t index = X.is_cuda() ? X.get_device() : -1;
  if (!current(index) || X.dim() != 2 || X.layout() != at::kStrided) Py_RETURN_NONE;
  const bool f32 = X.scalar_type() == at::kFloat;
  const at::Tensor *ws = tensor_of(a[2], index);
  int64_t br;
  if (!ws || (!f32 && X.scalar_type() != at::kBFloat16) || !int_of(a[1], br) || (br != 1 && br != 128))
    Py_RETURN_NONE;
  const int64_t rows = X.size(0), cols = X.size(1);
  const int64_t ldx = rows > 1 ? X.stride(0) : cols;
  if (rows < 1 || cols < 1 || (cols > 1 && X.stride(1) != 1) || ldx < cols) Py_RETURN_NONE;
  const int64_t ld = up(cols, 16), cb = up(cols, 128) / 128;
  at::Tensor q = at::detail::empty_strided_cuda({rows, cols}, {ld, 1}, at::kFloat8_e4m3fn, cuda(index));
  at::Tensor s = at::detail::empty_cuda({(rows + br - 1) / br, cb}, at::kFloat, cuda(index), std::nullopt);
  const int rc = without_gil([&] {
    return hyb_fp8_quant(rows, cols, X.const_data_ptr(), ldx, f32 ? HYB_F32 : HYB_BF16, (int)br,
                         (uint8_t *)q.data_ptr(), ld, s.data_ptr<float>(), cb, ws->data_ptr(),
                         (size_t)ws->numel(), stream_of(index));
  });
  if (rc != HYB_OK) return PyLong_FromLong(rc);
  return pair(std::move(q), std::move(s));
  END_HANDLE_TH_ERRORS
}

// (an Fp8Matrix's tensors and sizes, device or None, X, xs, Y, ydt, flags, ws)
PyObject *matmul_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t index, ydt, flags;
  hyb_fp8_matrix w;
  if (n != 8 || !index_of(a[1], a[0], index) || !current(index) || !matrix_of(a[0], index, w)) Py_RETURN_NONE;
  const hyb_fp8_matrix *A = &w;
  const at::Tensor *X = tensor_of(a[2], index), *ws = tensor_of(a[7], index);
  if (!X || !ws || X->dim() != 2 || X->size(1) != A->k || X->size(0) < 1 ||
      (A->k > 1 && X->stride(1) != 1) || !int_of(a[5], ydt) || !int_of(a[6], flags) ||
      (ydt != HYB_F32 && ydt != HYB_BF16) || flags < 0 || flags > UINT32_MAX)
    Py_RETURN_NONE;
  const int64_t m = X->size(0), kb = up(A->k, 128) / 128;
  const bool e4m3 = a[3] != Py_None;
  const float *xs = nullptr;
  int64_t ldxs = 0;
  if (X->scalar_type() != (e4m3 ? at::kFloat8_e4m3fn : at::kBFloat16)) Py_RETURN_NONE;
  if (e4m3) {
    const at::Tensor *s = tensor_of(a[3], index);
    if (!s || s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != m || s->size(1) != kb ||
        (kb > 1 && s->stride(1) != 1))
      Py_RETURN_NONE;
    ldxs = m > 1 ? s->stride(0) : kb;
    if (ldxs < kb) Py_RETURN_NONE;
    xs = s->const_data_ptr<float>();
  }
  const at::ScalarType yt = ydt == HYB_F32 ? at::kFloat : at::kBFloat16;
  at::Tensor Y;
  if (a[4] == Py_None) {
    Y = at::detail::empty_cuda({m, A->n}, yt, cuda(index), std::nullopt);
  } else {
    const at::Tensor *y = tensor_of(a[4], index);
    if (!y || y->scalar_type() != yt || y->dim() != 2 || y->size(0) != m || y->size(1) != A->n ||
        (A->n > 1 && y->stride(1) != 1))
      Py_RETURN_NONE;
    Y = *y;
  }
  const int rc = without_gil([&] {
    return hyb_fp8_matmul(A, m, X->const_data_ptr(), m > 1 ? X->stride(0) : up(A->k, 16),
                          e4m3 ? HYB_E4M3 : HYB_BF16, xs, ldxs, Y.data_ptr(),
                          m > 1 ? Y.stride(0) : A->n, (hyb_dtype)ydt, (uint32_t)flags,
                          ws->data_ptr(), (size_t)ws->numel(), stream_of(index));
  });
  if (rc != HYB_OK) return PyLong_FromLong(rc);
  if (a[4] != Py_None) return Py_NewRef(a[4]);
  return THPVariable_Wrap(std::move(Y));
  END_HANDLE_TH_ERRORS
}

// (a Cache's tensors, device or None, K, V, page_table, lens, off, max_new, ws) -> True
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t index;
  hyb_cache cache;
  if (n != 9 || !index_of(a[1], a[0], index) || !current(index) || !cache_of(a[0], index, cache)) Py_RETURN_NONE;
  const hyb_cache *C = &cache;
  const at::Tensor *K = tensor_of(a[2], index), *V = tensor_of(a[3], index), *ws = tensor_of(a[8], index);
  Rows k, v;
  hyb_sequences s;
  if (!K || !V || !ws || !rows_of(*K, C->head_dim, k) || !rows_of(*V, C->head_dim, v) || k.rows < 1 ||
      k.rows != v.rows || k.heads != C->kv_heads || v.heads != C->kv_heads ||
      !sequences_of(a[4], a[5], a[6], a[7], k.rows, index, s))
    Py_RETURN_NONE;
  const int rc = without_gil([&] {
    return hyb_cache_append(C, &s, (const uint16_t *)K->const_data_ptr(), k.ld, k.hs,
                            (const uint16_t *)V->const_data_ptr(), v.ld, v.hs, ws->data_ptr(),
                            (size_t)ws->numel(), stream_of(index));
  });
  if (rc != HYB_OK) return PyLong_FromLong(rc);
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// (a Cache's tensors, device or None, Q, page_table, lens, off, max_new, scale,
// window, sinks, out, return_lse, ws)
PyObject *cache_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t index, window, sinks;
  hyb_cache cache;
  if (n != 13 || !index_of(a[1], a[0], index) || !current(index) || !cache_of(a[0], index, cache)) Py_RETURN_NONE;
  const hyb_cache *C = &cache;
  const at::Tensor *Q = tensor_of(a[2], index), *ws = tensor_of(a[12], index);
  Rows q, o;
  hyb_sequences s;
  if (!Q || !ws || !rows_of(*Q, C->head_dim, q) || q.rows < 1 || q.heads < 1 || q.heads > INT32_MAX ||
      !sequences_of(a[3], a[4], a[5], a[6], q.rows, index, s) || !int_of(a[8], window) ||
      !int_of(a[9], sinks) || window < 0 || window > INT32_MAX || sinks < 0 || sinks > INT32_MAX ||
      !PyBool_Check(a[11]))
    Py_RETURN_NONE;
  double scale;
  if (a[7] == Py_None)
    scale = 1.0 / std::sqrt((double)C->head_dim);
  else if (PyFloat_CheckExact(a[7]))
    scale = PyFloat_AS_DOUBLE(a[7]);
  else
    Py_RETURN_NONE;
  at::Tensor out, lse;
  if (a[10] == Py_None) {
    out = at::detail::empty_cuda({q.rows, q.heads, C->head_dim}, at::kBFloat16, cuda(index), std::nullopt);
  } else {
    const at::Tensor *t = tensor_of(a[10], index);
    if (!t) Py_RETURN_NONE;
    out = *t;
  }
  if (!rows_of(out, C->head_dim, o) || o.rows != q.rows || o.heads != q.heads) Py_RETURN_NONE;
  const bool with_lse = a[11] == Py_True;
  if (with_lse) lse = at::detail::empty_cuda({q.rows, q.heads}, at::kFloat, cuda(index), std::nullopt);
  const int rc = without_gil([&] {
    return hyb_cache_attention(C, &s, (const uint16_t *)Q->const_data_ptr(), q.ld, q.hs,
                               (uint16_t *)out.data_ptr(), o.ld, o.hs,
                               with_lse ? lse.data_ptr<float>() : nullptr, q.heads, (int32_t)q.heads,
                               (float)scale, (int32_t)window, (int32_t)sinks, ws->data_ptr(),
                               (size_t)ws->numel(), stream_of(index));
  });
  if (rc != HYB_OK) return PyLong_FromLong(rc);
  PyObject *first = a[10] != Py_None ? Py_NewRef(a[10]) : THPVariable_Wrap(std::move(out));
  if (!with_lse || !first) return first;
  PyObject *second = THPVariable_Wrap(std::move(lse));
  PyObject *r = second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_DECREF(first);
  Py_XDECREF(second);
  return r;
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"quant_fp8", (PyCFunction)(void (*)(void))quant_fp8, METH_FASTCALL, nullptr},
    {"matmul_fp8", (PyCFunction)(void (*)(void))matmul_fp8, METH_FASTCALL, nullptr},
    {"cache_append", (PyCFunction)(void (*)(void))cache_append, METH_FASTCALL, nullptr},
    {"cache_attention", (PyCFunction)(void (*)(void))cache_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_hyb_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hyb_torch(void) { return PyModule_Create(&kModule); }
