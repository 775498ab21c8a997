// The paged calls from Python tensors. A decoding loop makes two of them per
// layer and token, where the checks of a dozen tensors in Python and ctypes'
// conversions of thirty arguments took 10 us a call, twice what a short call
// takes on the GPU; here they take under one. This module checks types, shapes,
// strides and devices and passes addresses on to the C entry points, whose
// addresses the Python binding hands over. Where an argument does not fit it
// returns None, and the binding finds out which one for its message.
#include <Python.h>

#include <climits>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mla_tree.h"

namespace {

decltype(&mla_paged_append) g_append = nullptr;
decltype(&mla_paged_decode) g_decode = nullptr;

// One tensor argument; `none` where None may stand for it.
struct Arg {
  const at::Tensor* t = nullptr;
  bool ok = true;
  explicit Arg(PyObject* o, bool none = false) {
    if (o == Py_None && none) return;
    ok = THPVariable_Check(o);
    if (ok) t = &THPVariable_Unpack(o);
  }
  // A strided CUDA tensor of that type, rank and device.
  bool is(at::ScalarType type, int64_t dim, int dev) const {
    return t && t->defined() && t->layout() == at::kStrided && t->is_cuda() && t->scalar_type() == type &&
           t->dim() == dim && t->get_device() == dev;
  }
  bool sizes(int64_t a) const { return t->size(0) == a && t->is_contiguous(); }
  bool sizes(int64_t a, int64_t b) const { return t->size(0) == a && t->size(1) == b; }
  bool sizes(int64_t a, int64_t b, int64_t c) const { return sizes(a, b) && t->size(2) == c; }
  bool rows() const { return t->size(t->dim() - 1) < 2 || t->stride(t->dim() - 1) == 1; }
  int64_t stride(int64_t dim) const { return t->stride(dim); }
  template <typename T>
  T* data() const { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
};

// The cache, its table and lengths.
struct Paged {
  Arg cache, table, lens;
  int dev = -1;
  int64_t pages = 0, size = 0, batch = 0, width = 0;
  Paged(PyObject* c, PyObject* t, PyObject* l) : cache(c), table(t), lens(l) {}
  bool ok() {
    if (!cache.ok || !table.ok || !lens.ok || !cache.t->defined() || !cache.t->is_cuda()) return false;
    dev = cache.t->get_device();
    if (!cache.is(at::kBFloat16, 3, dev) || !table.is(at::kInt, 2, dev) || !lens.is(at::kInt, 1, dev)) return false;
    pages = cache.t->size(0);
    size = cache.t->size(1);
    batch = table.t->size(0);
    width = table.t->size(1);
    return cache.t->size(2) == 576 && size > 0 && cache.stride(2) == 1 && (size == 1 || cache.stride(1) == 576) &&
           table.rows() && lens.sizes(batch) && batch <= INT_MAX && width <= INT_MAX && size <= INT_MAX;
  }
  int64_t page_stride() const { return pages > 1 ? cache.stride(0) : size * 576; }
  int64_t table_stride() const { return batch > 1 ? table.stride(0) : width; }
};

bool stream_of(PyObject* o, int dev, mt_stream_t* s) {
  if (o == Py_None) {
    *s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    return true;
  }
  *s = static_cast<mt_stream_t>(PyLong_AsVoidPtr(o));
  return !PyErr_Occurred();
}

// An optional array of int32 of any shape.
bool status_ok(const Arg& a, int dev) {
  return a.ok && (!a.t || (a.t->defined() && a.is(at::kInt, a.t->dim(), dev) && a.t->is_contiguous()));
}

PyObject* does_not_fit() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

template <typename F>
PyObject* guarded(int dev, F call) {
  if (c10::cuda::current_device() == dev) return PyLong_FromLong(call());
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
  return PyLong_FromLong(call());
}

// append(latent, k_rope, qo_indptr, kv_lens, block_table, cache, rope_table,
// q_rope, q_out, positions, norm_weight, norm_eps, rope_style, status, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 15 || !g_append) return does_not_fit();
    Arg latent(a[0]), k_rope(a[1]), indptr(a[2], true), rope(a[6]), q(a[7], true), out(a[8], true), pos(a[9], true),
        weight(a[10], true), status(a[13], true);
    Paged p(a[5], a[4], a[3]);
    if (!p.ok() || !latent.is(at::kBFloat16, 2, p.dev) || !k_rope.is(at::kBFloat16, 2, p.dev) ||
        !indptr.ok || (indptr.t && !indptr.is(at::kInt, 1, p.dev)) || !rope.is(at::kFloat, 2, p.dev) || !q.ok || !out.ok || !pos.ok || !weight.ok ||
        !status_ok(status, p.dev))
      return does_not_fit();
    const int64_t t = latent.t->size(0), angles = rope.t->size(0);
    if (t > INT_MAX || !latent.sizes(t, 512) || !latent.rows() || !k_rope.sizes(t, 64) || !k_rope.rows() ||
        !(indptr.t ? indptr.sizes(p.batch + 1) : t == p.batch) || !rope.sizes(angles, 64) || !rope.t->is_contiguous() || !q.t != !out.t)
      return does_not_fit();
    int64_t heads = 0;
    if (q.t) {
      if (!q.is(at::kBFloat16, 3, p.dev) || !out.is(at::kBFloat16, 3, p.dev)) return does_not_fit();
      heads = q.t->size(1);
      if (heads > INT_MAX || !q.sizes(t, heads, 64) || !out.sizes(t, heads, 64) || !q.rows() || !out.rows())
        return does_not_fit();
    }
    if (pos.t && (!pos.is(at::kInt, 1, p.dev) || !pos.sizes(t))) return does_not_fit();
    if (weight.t && (!weight.is(at::kBFloat16, 1, p.dev) || !weight.sizes(512))) return does_not_fit();
    const double eps = PyFloat_AsDouble(a[11]);
    const long style = PyLong_AsLong(a[12]);
    mt_stream_t stream;
    if (PyErr_Occurred() || style < 0 || style > 1 || !stream_of(a[14], p.dev, &stream)) return does_not_fit();
    const bool some = heads > 0;
    // the stride of a dimension of one element addresses nothing and may be anything
    auto tok = [&](const Arg& x) { return !some ? 0 : t > 1 ? x.stride(0) : 64; };
    auto head = [&](const Arg& x) { return !some ? 0 : heads > 1 ? x.stride(1) : 64; };
    return guarded(p.dev, [&] {
      return g_append(latent.data<mt_bf16>(), t > 1 ? latent.stride(0) : 512, k_rope.data<mt_bf16>(),
                      t > 1 ? k_rope.stride(0) : 64, weight.data<mt_bf16>(), (float)eps,
                      some ? q.data<mt_bf16>() : nullptr, tok(q), head(q),
                      some ? out.data<mt_bf16>() : nullptr, tok(out), head(out),
                      (int)heads, rope.data<float>(), angles, (int)style, pos.data<int32_t>(),
                      indptr.data<int32_t>(), p.lens.data<int32_t>(), (int)p.batch, (int)t, p.table.data<int32_t>(),
                      p.table_stride(), (int)p.width, p.cache.data<mt_bf16>(), p.page_stride(), p.pages, (int)p.size,
                      status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// decode(q, cache, block_table, kv_lens, sm_scale, out, lse, workspace, status, stream)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 10 || !g_decode) return does_not_fit();
    Arg q(a[0]), out(a[5]), lse(a[6]), ws(a[7]), status(a[8], true);
    Paged p(a[1], a[2], a[3]);
    if (!p.ok() || !q.is(at::kBFloat16, 3, p.dev) || !out.is(at::kBFloat16, 3, p.dev) || !lse.is(at::kFloat, 2, p.dev) ||
        !ws.is(at::kByte, 1, p.dev) || !status_ok(status, p.dev))
      return does_not_fit();
    const int64_t heads = q.t->size(1);
    if (heads > INT_MAX || !q.sizes(p.batch, heads, 576) || !q.rows() || !out.sizes(p.batch, heads, 512) ||
        !out.t->is_contiguous() || !lse.sizes(p.batch, heads) || !lse.t->is_contiguous() || !ws.t->is_contiguous())
      return does_not_fit();
    const double scale = PyFloat_AsDouble(a[4]);
    mt_stream_t stream;
    if (PyErr_Occurred() || !stream_of(a[9], p.dev, &stream)) return does_not_fit();
    return guarded(p.dev, [&] {
      return g_decode(q.data<mt_bf16>(), p.batch > 1 ? q.stride(0) : heads * 576, heads > 1 ? q.stride(1) : 576,
                      p.cache.data<mt_bf16>(), p.page_stride(), p.pages, (int)p.size, p.table.data<int32_t>(),
                      p.table_stride(), (int)p.width, p.lens.data<int32_t>(), (int)p.batch, (int)heads, (float)scale,
                      out.data<mt_bf16>(), lse.data<float>(), ws.data<void>(), (size_t)ws.t->numel(),
                      status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// bind(address of mla_paged_append, address of mla_paged_decode)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *x, *y;
  if (!PyArg_ParseTuple(args, "OO", &x, &y)) return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(x));
  g_decode = reinterpret_cast<decltype(g_decode)>(PyLong_AsVoidPtr(y));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
                         {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, nullptr},
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call(void) { return PyModule_Create(&module); }
