// The calls of a decoding loop from Python tensors. The loop makes two of them per
// layer and token, where the checks of a dozen tensors in Python and ctypes'
// conversions of thirty arguments took 10 us a call, twice what a short call
// takes on the GPU; here they take under one. This module checks types, shapes,
// strides and devices and passes addresses on to the C entry points, whose
// addresses the Python binding hands over. Where an argument does not fit it
// returns None, and the binding finds out which one for its message.
#include <Python.h>

#include <climits>
#include <type_traits>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mla_tree.h"

namespace {

decltype(&mla_paged_append) g_append = nullptr;
decltype(&mla_paged_decode) g_decode = nullptr;
decltype(&mla_paged_decode_window) g_window = nullptr;
decltype(&mla_token_logprobs) g_logprobs = nullptr;
decltype(&mla_tree_accept) g_accept = nullptr;
decltype(&mla_paged_compact) g_compact = nullptr;
decltype(&mla_pages_fork) g_fork = nullptr;
decltype(&mla_pages_fit_lens) g_fit = nullptr;
decltype(&mla_paged_copy) g_copy = nullptr;

// One tensor argument; `none` where None may stand for it.
struct Arg {
  const at::Tensor* t = nullptr;
  bool ok = true;
  explicit Arg(PyObject* o, bool none = false) {
    if (o == Py_None && none) return;
    ok = THPVariable_Check(o);
    if (ok) t = &THPVariable_Unpack(o);
  }
  bool here() const { return ok && t && t->defined() && t->is_cuda(); }
  int64_t size(int64_t dim) const { return t->size(dim); }
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

// Shared by the two decode calls: a[0..3] q, cache, block_table, kv_lens and
// a[i..] sm_scale, out, lse, workspace, status, stream; call(...) makes the call.
template <typename F>
PyObject* decode_with(PyObject* const* a, int i, F call) {
  Arg q(a[0]), out(a[i + 1]), lse(a[i + 2]), ws(a[i + 3]), status(a[i + 4], true);
  Paged p(a[1], a[2], a[3]);
  if (!p.ok() || !q.is(at::kBFloat16, 3, p.dev) || !out.is(at::kBFloat16, 3, p.dev) || !lse.is(at::kFloat, 2, p.dev) ||
      !ws.is(at::kByte, 1, p.dev) || !status_ok(status, p.dev))
    return does_not_fit();
  const int64_t heads = q.t->size(1);
  if (heads > INT_MAX || !q.sizes(p.batch, heads, 576) || !q.rows() || !out.sizes(p.batch, heads, 512) ||
      !out.t->is_contiguous() || !lse.sizes(p.batch, heads) || !lse.t->is_contiguous() || !ws.t->is_contiguous())
    return does_not_fit();
  const double scale = PyFloat_AsDouble(a[i]);
  mt_stream_t stream;
  if (PyErr_Occurred() || !stream_of(a[i + 5], p.dev, &stream)) return does_not_fit();
  return guarded(p.dev, [&] { return call(q, p, heads, (float)scale, out, lse, ws, status, stream); });
}

// decode(q, cache, block_table, kv_lens, sm_scale, out, lse, workspace, status, stream)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 10 || !g_decode) return does_not_fit();
    return decode_with(a, 4, [](const Arg& q, const Paged& p, int64_t heads, float scale, const Arg& out, const Arg& lse,
                                const Arg& ws, const Arg& status, mt_stream_t stream) {
      return g_decode(q.data<mt_bf16>(), p.batch > 1 ? q.stride(0) : heads * 576, heads > 1 ? q.stride(1) : 576,
                      p.cache.data<mt_bf16>(), p.page_stride(), p.pages, (int)p.size, p.table.data<int32_t>(),
                      p.table_stride(), (int)p.width, p.lens.data<int32_t>(), (int)p.batch, (int)heads, scale,
                      out.data<mt_bf16>(), lse.data<float>(), ws.data<void>(), (size_t)ws.t->numel(),
                      status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

bool int_of(PyObject* o, int* v) {
  const long x = PyLong_AsLong(o);
  if (PyErr_Occurred() || x < INT_MIN || x > INT_MAX) return false;
  *v = (int)x;
  return true;
}

// decode_window(q, cache, block_table, kv_lens, window, sinks, sm_scale, out, lse, workspace, status, stream)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    int window, sinks;
    if (n != 12 || !g_window || !int_of(a[4], &window) || !int_of(a[5], &sinks)) return does_not_fit();
    return decode_with(a, 6, [&](const Arg& q, const Paged& p, int64_t heads, float scale, const Arg& out, const Arg& lse,
                                 const Arg& ws, const Arg& status, mt_stream_t stream) {
      return g_window(q.data<mt_bf16>(), p.batch > 1 ? q.stride(0) : heads * 576, heads > 1 ? q.stride(1) : 576,
                      p.cache.data<mt_bf16>(), p.page_stride(), p.pages, (int)p.size, p.table.data<int32_t>(),
                      p.table_stride(), (int)p.width, p.lens.data<int32_t>(), window, sinks, (int)p.batch, (int)heads,
                      scale, out.data<mt_bf16>(), lse.data<float>(), ws.data<void>(), (size_t)ws.t->numel(),
                      status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// logprobs(logits, tokens, logprobs, lse, entropy, top_ids, top_logprobs, status, stream)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 9 || !g_logprobs) return does_not_fit();
    Arg x(a[0]), tok(a[1], true), lp(a[2], true), lse(a[3], true), ent(a[4], true), ids(a[5], true), top(a[6], true),
        status(a[7], true);
    if (!x.here() || x.t->dim() != 2) return does_not_fit();
    const int dev = x.t->get_device();
    const at::ScalarType type = x.t->scalar_type();
    const int64_t rows = x.size(0), vocab = x.size(1);
    if (!x.is(type, 2, dev) || (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat) || rows > INT_MAX ||
        vocab < 1 || vocab > INT_MAX || !x.rows() || !status_ok(status, dev) || !tok.ok || !lp.ok || !lse.ok || !ent.ok ||
        !ids.ok || !top.ok || !tok.t != !lp.t)
      return does_not_fit();
    int64_t per_row = 0, k = 0;
    if (tok.t) {
      const int64_t dim = tok.t->dim();
      if ((dim != 1 && dim != 2) || !tok.is(at::kInt, dim, dev) || !lp.is(at::kFloat, dim, dev) || tok.size(0) != rows ||
          lp.t->sizes() != tok.t->sizes() || !lp.t->is_contiguous())
        return does_not_fit();
      per_row = dim == 2 ? tok.size(1) : 1;
      if (per_row > INT_MAX || (dim == 2 && per_row > 1 && tok.stride(1) != 1)) return does_not_fit();
    }
    for (const Arg* v : {&lse, &ent})
      if (v->t && (!v->is(at::kFloat, 1, dev) || !v->sizes(rows))) return does_not_fit();
    if (ids.t) {
      if (!ids.is(at::kInt, 2, dev) || ids.size(0) != rows || !ids.t->is_contiguous()) return does_not_fit();
      k = ids.size(1);
    }
    if (top.t && (!ids.t || !top.is(at::kFloat, 2, dev) || !top.sizes(rows, k) || !top.t->is_contiguous()))
      return does_not_fit();
    mt_stream_t stream;
    if (k > INT_MAX || !stream_of(a[8], dev, &stream)) return does_not_fit();
    const int kind = type == at::kBFloat16 ? MT_LOGITS_BF16 : type == at::kHalf ? MT_LOGITS_FP16 : MT_LOGITS_FP32;
    return guarded(dev, [&] {
      return g_logprobs(x.data<void>(), kind, rows > 1 ? x.stride(0) : vocab, (int)rows, (int)vocab,
                        per_row ? tok.data<int32_t>() : nullptr, per_row && rows > 1 ? tok.stride(0) : per_row, (int)per_row,
                        (int)k, per_row ? lp.data<float>() : nullptr, lse.data<float>(), ent.data<float>(),
                        k ? ids.data<int32_t>() : nullptr, k ? top.data<float>() : nullptr, status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// A contiguous int32 array of that many elements.
bool ints(const Arg& a, int64_t n, int dev) { return a.is(at::kInt, 1, dev) && a.sizes(n); }

// accept(parents, tokens, targets, qo_indptr, kv_lens, path, counts, next_tokens, new_lens, first, status, stream)
PyObject* accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 12 || !g_accept) return does_not_fit();
    Arg parents(a[0]), tokens(a[1]), targets(a[2]), indptr(a[3]), lens(a[4]), path(a[5]), counts(a[6]), next(a[7]),
        new_lens(a[8]), first(a[9], true), status(a[10], true);
    if (!parents.here()) return does_not_fit();
    const int dev = parents.t->get_device();
    if (!parents.is(at::kInt, 1, dev) || !path.ok || !path.is(at::kInt, 2, dev)) return does_not_fit();
    const int64_t t = parents.size(0), batch = path.size(0), most = path.size(1);
    if (t > INT_MAX || batch > INT_MAX - 1 || most > INT_MAX || !parents.sizes(t) || !ints(tokens, t, dev) ||
        !targets.is(at::kInt, 1, dev) || targets.size(0) != t || !ints(indptr, batch + 1, dev) || !ints(lens, batch, dev) ||
        !path.t->is_contiguous() || !ints(counts, batch, dev) || !ints(next, batch, dev) || !ints(new_lens, batch, dev) ||
        !first.ok || (first.t && !ints(first, batch, dev)) || !status_ok(status, dev))
      return does_not_fit();
    mt_stream_t stream;
    if (!stream_of(a[11], dev, &stream)) return does_not_fit();
    return guarded(dev, [&] {
      return g_accept(parents.data<int32_t>(), tokens.data<int32_t>(), targets.data<int32_t>(),
                      t > 1 ? targets.stride(0) : 1, first.data<int32_t>(), indptr.data<int32_t>(), lens.data<int32_t>(),
                      (int)batch, (int)t, (int)most, most ? path.data<int32_t>() : nullptr, counts.data<int32_t>(),
                      next.data<int32_t>(), new_lens.data<int32_t>(), status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// A cache of one layer [pages, page, 576] or of several [layers, pages, page, 576].
struct Layers {
  Arg cache;
  int dev = -1;
  int64_t layers = 1, layer_stride = 0, pages = 0, size = 0, page_stride = 0;
  explicit Layers(PyObject* c) : cache(c) {}
  bool ok() {
    if (!cache.here()) return false;
    dev = cache.t->get_device();
    const int64_t d = cache.t->dim();
    if ((d != 3 && d != 4) || !cache.is(at::kBFloat16, d, dev)) return false;
    if (d == 4) {
      layers = cache.size(0);
      layer_stride = layers > 1 ? cache.stride(0) : 0;
    }
    pages = cache.size(d - 3);
    size = cache.size(d - 2);
    page_stride = pages > 1 ? cache.stride(d - 3) : size * 576;
    return cache.size(d - 1) == 576 && size > 0 && cache.stride(d - 1) == 1 && (size == 1 || cache.stride(d - 2) == 576) &&
           layers <= INT_MAX && size <= INT_MAX;
  }
};

// compact(path, counts, kv_lens, block_table, cache, status, stream)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 7 || !g_compact) return does_not_fit();
    Arg path(a[0]), counts(a[1]), lens(a[2]), table(a[3]), status(a[5], true);
    Layers c(a[4]);
    if (!c.ok() || !path.ok || !table.ok || !path.is(at::kInt, 2, c.dev) || !table.is(at::kInt, 2, c.dev)) return does_not_fit();
    const int64_t batch = table.size(0), width = table.size(1), most = path.size(1);
    if (batch > INT_MAX || width > INT_MAX || most > INT_MAX || path.size(0) != batch || !path.rows() || !table.rows() ||
        !ints(counts, batch, c.dev) || !ints(lens, batch, c.dev) || !status_ok(status, c.dev))
      return does_not_fit();
    mt_stream_t stream;
    if (!stream_of(a[6], c.dev, &stream)) return does_not_fit();
    return guarded(c.dev, [&] {
      return g_compact(path.data<int32_t>(), batch > 1 ? path.stride(0) : most, (int)most, counts.data<int32_t>(),
                       lens.data<int32_t>(), (int)batch, table.data<int32_t>(), batch > 1 ? table.stride(0) : width,
                       (int)width, c.cache.data<mt_bf16>(), c.page_stride, c.pages, (int)c.size, (int)c.layers,
                       c.layer_stride, status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// fork(parents, kv_lens, held, block_table, refs, new_lens, new_held, new_table, status, stream)
PyObject* fork_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 10 || !g_fork) return does_not_fit();
    Arg parents(a[0]), lens(a[1]), held(a[2]), table(a[3]), refs(a[4]), new_lens(a[5]), new_held(a[6]), new_table(a[7]),
        status(a[8], true);
    if (!refs.here()) return does_not_fit();
    const int dev = refs.t->get_device();
    if (!refs.is(at::kInt, 1, dev) || !refs.t->is_contiguous() || !table.is(at::kInt, 2, dev) ||
        !new_table.is(at::kInt, 2, dev))
      return does_not_fit();
    const int64_t old = table.size(0), width = table.size(1), rows = new_table.size(0), pages = refs.size(0);
    if (old > INT_MAX || rows > INT_MAX || width > INT_MAX || new_table.size(1) != width || !table.rows() ||
        !new_table.rows() || !ints(parents, rows, dev) || !ints(lens, old, dev) || !ints(held, old, dev) ||
        !ints(new_lens, rows, dev) || !ints(new_held, rows, dev) || !status_ok(status, dev))
      return does_not_fit();
    mt_stream_t stream;
    if (!stream_of(a[9], dev, &stream)) return does_not_fit();
    return guarded(dev, [&] {
      return g_fork(parents.data<int32_t>(), lens.data<int32_t>(), held.data<int32_t>(), table.data<int32_t>(),
                    old > 1 ? table.stride(0) : width, (int)old, (int)width, refs.data<int32_t>(), pages,
                    new_lens.data<int32_t>(), new_held.data<int32_t>(), new_table.data<int32_t>(),
                    rows > 1 ? new_table.stride(0) : width, (int)rows, status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// fit(kv_lens, want_lens, held, block_table, refs, page_size, copies, workspace, window, sinks, status, stream, step_lens)
PyObject* fit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    int page, window, sinks;
    if (n != 13 || !g_fit || !int_of(a[5], &page) || !int_of(a[8], &window) || !int_of(a[9], &sinks)) return does_not_fit();
    Arg lens(a[0]), want(a[1]), held(a[2]), table(a[3]), refs(a[4]), copies(a[6]), ws(a[7]), status(a[10], true),
        step(a[12], true);
    if (!refs.here()) return does_not_fit();
    const int dev = refs.t->get_device();
    if (!refs.is(at::kInt, 1, dev) || !refs.t->is_contiguous() || !table.is(at::kInt, 2, dev) ||
        !copies.is(at::kInt, 2, dev) || !ws.is(at::kByte, 1, dev))
      return does_not_fit();
    const int64_t batch = table.size(0), width = table.size(1), pages = refs.size(0);
    if (batch > INT_MAX || width > INT_MAX || !table.rows() || !ints(lens, batch, dev) || !ints(want, batch, dev) ||
        !ints(held, batch, dev) || !copies.sizes(batch, 3) || !copies.t->is_contiguous() || !ws.t->is_contiguous() ||
        !step.ok || (step.t && !ints(step, batch, dev)) || !status_ok(status, dev))
      return does_not_fit();
    mt_stream_t stream;
    if (!stream_of(a[11], dev, &stream)) return does_not_fit();
    return guarded(dev, [&] {
      return g_fit(lens.data<int32_t>(), want.data<int32_t>(), held.data<int32_t>(), table.data<int32_t>(),
                   batch > 1 ? table.stride(0) : width, (int)batch, (int)width, refs.data<int32_t>(), pages, page, window,
                   sinks, copies.data<int32_t>(), step.data<int32_t>(), ws.data<void>(), (size_t)ws.t->numel(),
                   status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// copy(copies, cache, status, stream)
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 4 || !g_copy) return does_not_fit();
    Arg copies(a[0]), status(a[2], true);
    Layers c(a[1]);
    if (!c.ok() || !copies.is(at::kInt, 2, c.dev) || copies.size(1) != 3 || !copies.t->is_contiguous() ||
        !status_ok(status, c.dev))
      return does_not_fit();
    mt_stream_t stream;
    if (!stream_of(a[3], c.dev, &stream)) return does_not_fit();
    return guarded(c.dev, [&] {
      return g_copy(copies.data<int32_t>(), copies.size(0), c.cache.data<mt_bf16>(), c.page_stride, c.pages, (int)c.size,
                    (int)c.layers, c.layer_stride, status.data<int32_t>(), stream);
    });
  } catch (...) {
    return does_not_fit();
  }
}

// bind(addresses of mla_paged_append, mla_paged_decode, mla_paged_decode_window, mla_token_logprobs,
// mla_tree_accept, mla_paged_compact, mla_pages_fork, mla_pages_fit_lens, mla_paged_copy)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* x[9];
  if (!PyArg_ParseTuple(args, "OOOOOOOOO", &x[0], &x[1], &x[2], &x[3], &x[4], &x[5], &x[6], &x[7], &x[8])) return nullptr;
  auto set = [](auto& f, PyObject* o) { f = reinterpret_cast<std::decay_t<decltype(f)>>(PyLong_AsVoidPtr(o)); };
  set(g_append, x[0]);
  set(g_decode, x[1]);
  set(g_window, x[2]);
  set(g_logprobs, x[3]);
  set(g_accept, x[4]);
  set(g_compact, x[5]);
  set(g_fork, x[6]);
  set(g_fit, x[7]);
  set(g_copy, x[8]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

#define MT_METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MT_METHOD("append", append),
                         MT_METHOD("decode", decode),
                         MT_METHOD("decode_window", decode_window),
                         MT_METHOD("logprobs", logprobs),
                         MT_METHOD("accept", accept),
                         MT_METHOD("compact", compact),
                         MT_METHOD("fork", fork_rows),
                         MT_METHOD("fit", fit),
                         MT_METHOD("copy", copy_pages),
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_call(void) { return PyModule_Create(&module); }
