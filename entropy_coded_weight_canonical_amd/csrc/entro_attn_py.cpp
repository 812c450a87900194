// Python binding of entro_attn.h: reads torch tensors, checks them against one
// another and hands their pointers and strides to the C ABI.  (Read from Python,
// shapes, strides, types and pointers of a call's tensors took 4 to 6 us and its
// result's memory 1.5 us each, with small calls' kernels at 5 us.)
//
// Functions take their arguments by position, `None` for what is not given.
// The last two are whether memory may be made for the call (it comes from
// torch's current stream) and the stream's handle, `None` for the current one.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <sstream>
#include <stdexcept>

#include "entro_attn.h"

namespace {

// The library's functions, and from Python: the handle of a device's current
// stream, and what raises a status that is not 0.
struct {
  decltype(&entro_attn_prompt) prompt;
  decltype(&entro_attn_prompt_work_bytes) prompt_bytes;
  decltype(&entro_kv_store) store;
  decltype(&entro_kv_load) load;
  decltype(&entro_attn_cache) cache;
  decltype(&entro_attn_cache_work_bytes) cache_bytes;
  decltype(&entro_rope) rope;
  decltype(&entro_kv_append) append;
  decltype(&entro_attn_chunk) chunk;
  decltype(&entro_attn_chunk_work_bytes) chunk_bytes;
  PyObject *raw_stream, *check, *desc;
} g;

struct Raised {};   // a Python exception is set

template <typename... Parts>
[[noreturn]] void refuse(const Parts &...parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw std::invalid_argument(s.str());
}

const at::Tensor &tensor(PyObject *o, const char *what) {
  if (!THPVariable_Check(o)) refuse(what, ": a tensor expected");
  return THPVariable_Unpack(o);
}

// All tensors of a call are on the device of the first one that is named (the
// call's, which the kernels run on), and none is one that a gradient is recorded
// for or that carries a tangent: there is no derivative, backward or forward.  Looked at
// before anything is read or made.
struct Together {
  const at::Device device;
  const Together &operator()(const char *what, const at::Tensor &x) const {
    if (x.device() != device) refuse(what, ": on device ", x.device(), ", the call is on ", device);
    if (x.requires_grad() && c10::GradMode::is_enabled())
      refuse(what, ": requires a gradient, and there is no backward pass; call under torch.no_grad() or detach it");
    if (x._fw_grad(/*level=*/0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
      refuse(what, ": carries a tangent, and there is no forward-mode derivative; unpack it first");
    return *this;
  }
};

int type_of(const at::Tensor &x) {
  if (x.scalar_type() == at::kBFloat16) return ENTRO_BF16;
  if (x.scalar_type() == at::kHalf) return ENTRO_F16;
  refuse("element type ", x.scalar_type(), ": bfloat16 or float16 expected");
}

entro_rows rows(const at::Tensor &x, const char *what, at::ScalarType type, int64_t heads, int64_t dim) {
  if (x.dim() != 3 || x.size(1) != heads || x.size(2) != dim)
    refuse(what, ": shape ", x.sizes(), ", expected [rows, ", heads, ", ", dim, "]");
  if (x.scalar_type() != type || !x.is_cuda())
    refuse(what, ": a ", type, " tensor on the GPU expected, got ", x.scalar_type(), " on ", x.device());
  if (x.stride(2) != 1 && dim > 1) refuse(what, ": the head dimension has to be contiguous");
  return {x.data_ptr(), x.size(0) > 1 ? x.stride(0) : heads * dim, heads > 1 ? x.stride(1) : dim};
}

void *ints(const at::Tensor &x, const char *what, int64_t n) {
  if (x.scalar_type() != at::kInt || x.dim() != 1 || x.size(0) != n || !x.is_cuda() || (n > 1 && !x.is_contiguous()))
    refuse(what, ": ", n, " contiguous int32 values on the GPU expected, got ", x.scalar_type(), " ", x.sizes(), " on ",
           x.device());
  return x.data_ptr();
}

entro_kv_table table_of(const at::Tensor &x, int64_t n) {
  if (x.scalar_type() != at::kInt || x.dim() != 2 || x.size(0) != n || !x.is_cuda())
    refuse("table: int32 [", n, "][pages] on the GPU expected, got ", x.scalar_type(), " ", x.sizes(), " on ", x.device());
  const int64_t pages = x.size(1);
  if (pages > 1 && x.stride(1) != 1) refuse("table: the pages of a sequence have to lie side by side");
  const int64_t stride = n > 1 ? x.stride(0) : pages;
  if (pages > UINT32_MAX || stride > UINT32_MAX) refuse("table: too many pages");
  return {static_cast<int32_t *>(x.data_ptr()), (uint32_t)stride, (uint32_t)pages, (uint32_t)n};
}

uint32_t small(int64_t n, const char *what) {
  if (n < 0 || n > UINT32_MAX) refuse(what, ": ", n, " does not fit 32 bits");
  return (uint32_t)n;
}

// A KVCache's attribute `desc`, made by cache_desc: the C ABI's description and
// the GPU that the tensors are on.
struct CacheDesc {
  entro_kv_cache c;
  int64_t gpu;
  at::Device device() const { return {at::kCUDA, (at::DeviceIndex)gpu}; }
};
// A Rotary's, made by rotary_desc.
struct RotaryDesc {
  entro_rotary r;
  int64_t gpu;
  at::Device device() const { return {at::kCUDA, (at::DeviceIndex)gpu}; }
};
template <typename Desc>
Desc desc_of(PyObject *of, const char *expected) {
  PyObject *desc = PyObject_GetAttr(of, g.desc);
  if (!desc) throw Raised();
  Desc c{};
  const bool ok = PyBytes_Check(desc) && PyBytes_GET_SIZE(desc) == sizeof c;
  if (ok) std::memcpy(&c, PyBytes_AS_STRING(desc), sizeof c);
  Py_DECREF(desc);
  if (!ok) refuse(expected);
  return c;
}
CacheDesc cache_of(PyObject *cache) { return desc_of<CacheDesc>(cache, "cache: a KVCache expected"); }

struct On {
  bool make;          // memory may be made for the call
  PyObject *stream;
  hipStream_t handle(const at::Tensor &x) const {
    PyObject *h = nullptr;
    if (stream == Py_None) {
      PyObject *device = PyLong_FromLong(x.device().index());
      h = device ? PyObject_CallOneArg(g.raw_stream, device) : nullptr;
      Py_XDECREF(device);
    } else {
      Py_INCREF(stream);
      h = stream;
    }
    void *p = h ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    if (PyErr_Occurred()) throw Raised();
    return static_cast<hipStream_t>(p);
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) const {
    if (!make) refuse("on a raw stream handle the caller gives the memory of results and workspace");
    if (!like.is_cuda()) refuse("tensors on the GPU expected, got ", like.device());
    return at::empty(shape, like.options().dtype(type).layout(at::kStrided));
  }
};

std::pair<void *, uint64_t> workspace(const at::Tensor &x) {
  if (!x.is_cuda() || !x.is_contiguous()) refuse("work: a contiguous tensor on the GPU expected");
  return {x.data_ptr(), (uint64_t)x.numel() * x.element_size()};
}

float scale_of(PyObject *o, int64_t dim) {
  if (o == Py_None) return (float)(1.0 / std::sqrt((double)dim));
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)v;
}

void done(entro_status st, const char *name) {
  if (st == ENTRO_OK) return;
  PyObject *r = PyObject_CallFunction(g.check, "is", (int)st, name);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, (int)st);
  throw Raised();
}

using Args = PyObject *const *;

// q, k, v, cu_q, cu_k, status, scale, out, work, make, stream -> out
PyObject *prompt(Args a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const at::Tensor &cu_q = tensor(a[3], "cu_q"), &cu_k = tensor(a[4], "cu_k"), &status = tensor(a[5], "status");
  at::Tensor out, work;
  const Together together{q.device()};
  together("q", q)("k", k)("v", v)("cu_q", cu_q)("cu_k", cu_k)("status", status);
  if (a[7] != Py_None) together("out", out = tensor(a[7], "out"));
  if (a[8] != Py_None) together("work", work = tensor(a[8], "work"));
  const On on{a[9] == Py_True, a[10]};
  const c10::DeviceGuard guard(q.device());
  if (cu_q.dim() != 1 || cu_q.size(0) < 1 || q.dim() != 3 || k.dim() != 3)
    refuse("q, k, v are [rows][heads][dim], cu_q and cu_k hold n + 1 sums");
  const int64_t n = cu_q.size(0) - 1, heads = q.size(1), dim = q.size(2), kv = k.size(1);
  if (v.dim() != 3 || v.size(0) != k.size(0)) refuse("k and v have the same rows");
  const at::ScalarType t = q.scalar_type();
  entro_attn_prompt_args p{};
  p.dtype = (entro_dtype)type_of(q);
  if (!out.defined())
    out = on.empty(q.sizes(), t, q);
  else if (out.dim() == 3 && out.size(0) != q.size(0))
    refuse("out has the rows of q");
  p.out = rows(out, "out", t, heads, dim);
  p.q = rows(q, "q", t, heads, dim);
  p.k = rows(k, "k", t, kv, dim);
  p.v = rows(v, "v", t, kv, dim);
  p.d_cu_q = static_cast<int32_t *>(ints(cu_q, "cu_q", n + 1));
  p.d_cu_k = static_cast<int32_t *>(ints(cu_k, "cu_k", n + 1));
  p.n_seq = small(n, "cu_q");
  p.total_q = small(q.size(0), "q");
  p.total_k = small(k.size(0), "k");
  p.n_heads = small(heads, "q");
  p.n_kv_heads = small(kv, "k");
  p.head_dim = small(dim, "q");
  p.scale = scale_of(a[6], dim);
  if (!work.defined() && on.make) {   // (without workspace the keys are not split)
    const uint64_t bytes = g.prompt_bytes(p.n_seq, p.total_q, p.total_k, p.n_heads, p.n_kv_heads, p.head_dim);
    if (bytes) work = on.empty({(int64_t)bytes}, at::kByte, q);
  }
  if (work.defined()) std::tie(p.d_work, p.work_bytes) = workspace(work);
  done(g.prompt(&p, static_cast<uint32_t *>(ints(status, "status", n)), on.handle(q)), "entro_attn_prompt");
  return THPVariable_Wrap(std::move(out));
}

// The part that the store and the load share.
template <typename Fn, typename A>
void kv_call(Fn fn, A p, const char *name, const entro_kv_cache &c, const at::Tensor &k, const at::Tensor &v,
             const at::Tensor &table, const at::Tensor &status, const On &on) {
  const c10::DeviceGuard guard(k.device());
  const entro_kv_table t = table_of(table, table.dim() ? table.size(0) : 0);
  p.k = rows(k, "k", k.scalar_type(), c.n_kv_heads, c.head_dim);
  p.v = rows(v, "v", k.scalar_type(), c.n_kv_heads, c.head_dim);
  p.dtype = (entro_dtype)type_of(k);
  done(fn(&c, &t, &p, static_cast<uint32_t *>(ints(status, "status", t.n_seq)), on.handle(k)), name);
}

// cache, k, v, table, held, cu_new, status, make, stream
PyObject *store(Args a) {
  const CacheDesc desc = cache_of(a[0]);
  const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &table = tensor(a[3], "table");
  const at::Tensor &held = tensor(a[4], "held"), &cu_new = tensor(a[5], "cu_new"), &status = tensor(a[6], "status");
  if (k.dim() != 3 || v.dim() != 3 || k.size(0) != v.size(0)) refuse("k and v have the same rows");
  if (!k.is_cuda()) refuse("k: a tensor on the GPU expected, got ", k.device());
  Together{desc.device()}("k", k)("v", v)("table", table)("held", held)("cu_new", cu_new)("status", status);
  const int64_t n = table.dim() ? table.size(0) : 0;
  entro_kv_store_args p{};
  p.d_held = static_cast<int32_t *>(ints(held, "held", n));
  p.d_cu_new = static_cast<int32_t *>(ints(cu_new, "cu_new", n + 1));
  p.total_new = small(k.size(0), "k");
  kv_call(g.store, p, "entro_kv_store", desc.c, k, v, table, status, {a[7] == Py_True, a[8]});
  Py_RETURN_NONE;
}

// cache, table, first, cu_out, total, status, type of the results as f16 or not, k, v, make, stream -> (k, v)
PyObject *load(Args a) {
  const CacheDesc desc = cache_of(a[0]);
  const entro_kv_cache &c = desc.c;
  const at::Tensor &table = tensor(a[1], "table"), &first = tensor(a[2], "first"), &cu_out = tensor(a[3], "cu_out");
  const at::Tensor &status = tensor(a[5], "status");
  const Together together{desc.device()};
  together("table", table)("first", first)("cu_out", cu_out)("status", status);
  const On on{a[9] == Py_True, a[10]};
  const int64_t n = table.dim() ? table.size(0) : 0, total = PyLong_AsLongLong(a[4]);
  if (total == -1 && PyErr_Occurred()) throw Raised();
  entro_kv_load_args p{};
  p.total_out = small(total, "total");
  at::Tensor k, v;
  if (a[7] == Py_None) {
    const at::ScalarType t = a[6] == Py_True ? at::kHalf : at::kBFloat16;
    k = on.empty({total, c.n_kv_heads, c.head_dim}, t, table);
    v = on.empty({total, c.n_kv_heads, c.head_dim}, t, table);
  } else {
    together("k", k = tensor(a[7], "k"))("v", v = tensor(a[8], "v"));
    if (k.dim() != 3 || v.dim() != 3 || k.size(0) != total || v.size(0) != total) refuse("the outputs have `total` rows");
  }
  p.d_first = static_cast<int32_t *>(ints(first, "first", n));
  p.d_cu_out = static_cast<int32_t *>(ints(cu_out, "cu_out", n + 1));
  kv_call(g.load, p, "entro_kv_load", c, k, v, table, status, on);
  PyObject *x = THPVariable_Wrap(std::move(k)), *y = THPVariable_Wrap(std::move(v));
  PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// q, cache, table, lens, status, scale, out, work, make, stream -> out
PyObject *cache(Args a) {
  const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[2], "table"), &lens = tensor(a[3], "lens");
  const at::Tensor &status = tensor(a[4], "status");
  const CacheDesc desc = cache_of(a[1]);
  const entro_kv_cache &c = desc.c;
  at::Tensor out, work;
  const Together together{desc.device()};
  together("q", q)("table", table)("lens", lens)("status", status);
  if (a[6] != Py_None) together("out", out = tensor(a[6], "out"));
  if (a[7] != Py_None) together("work", work = tensor(a[7], "work"));
  const On on{a[8] == Py_True, a[9]};
  const c10::DeviceGuard guard(q.device());
  if (q.dim() != 3) refuse("q is [sequences][heads][dim]");
  const int64_t n = q.size(0), heads = q.size(1), dim = q.size(2);
  if (dim != c.head_dim) refuse("q has head dimension ", dim, ", the cache ", c.head_dim);
  const at::ScalarType t = q.scalar_type();
  entro_attn_cache_args p{};
  p.dtype = (entro_dtype)type_of(q);
  if (!out.defined())
    out = on.empty(q.sizes(), t, q);
  else if (out.dim() == 3 && out.size(0) != n)
    refuse("out has the rows of q");
  p.out = rows(out, "out", t, heads, dim);
  p.q = rows(q, "q", t, heads, dim);
  p.n_heads = small(heads, "q");
  if (!work.defined()) {
    const uint64_t bytes = g.cache_bytes(small(n, "q"), p.n_heads, c.n_kv_heads, c.head_dim);
    work = on.empty({(int64_t)std::max<uint64_t>(bytes, 16u)}, at::kByte, q);
  }
  std::tie(p.d_work, p.work_bytes) = workspace(work);
  p.d_lens = static_cast<int32_t *>(ints(lens, "lens", n));
  p.scale = scale_of(a[5], dim);
  const entro_kv_table tb = table_of(table, n);
  done(g.cache(&c, &tb, &p, static_cast<uint32_t *>(ints(status, "status", n)), on.handle(q)), "entro_attn_cache");
  return THPVariable_Wrap(std::move(out));
}

// q, cache, table, lens, cu_q, status, scale, out, work, make, stream -> out
PyObject *chunk(Args a) {
  const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[2], "table"), &lens = tensor(a[3], "lens");
  const at::Tensor &cu_q = tensor(a[4], "cu_q"), &status = tensor(a[5], "status");
  const CacheDesc desc = cache_of(a[1]);
  const entro_kv_cache &c = desc.c;
  at::Tensor out, work;
  const Together together{desc.device()};
  together("q", q)("table", table)("lens", lens)("cu_q", cu_q)("status", status);
  if (a[7] != Py_None) together("out", out = tensor(a[7], "out"));
  if (a[8] != Py_None) together("work", work = tensor(a[8], "work"));
  const On on{a[9] == Py_True, a[10]};
  if (q.dim() != 3) refuse("q is [rows][heads][dim]");
  const int64_t n = table.dim() ? table.size(0) : 0, heads = q.size(1), dim = q.size(2);
  if (dim != c.head_dim) refuse("q has head dimension ", dim, ", the cache ", c.head_dim);
  const at::ScalarType t = q.scalar_type();
  entro_attn_chunk_args p{};
  p.dtype = (entro_dtype)type_of(q);
  if (!out.defined())
    out = on.empty(q.sizes(), t, q);
  else if (out.dim() == 3 && out.size(0) != q.size(0))
    refuse("out has the rows of q");
  p.out = rows(out, "out", t, heads, dim);
  p.q = rows(q, "q", t, heads, dim);
  p.total_q = small(q.size(0), "q");
  p.n_heads = small(heads, "q");
  p.d_lens = static_cast<int32_t *>(ints(lens, "lens", n));
  p.d_cu_q = static_cast<int32_t *>(ints(cu_q, "cu_q", n + 1));
  p.scale = scale_of(a[6], dim);
  if (!work.defined()) {
    const uint64_t bytes = g.chunk_bytes(small(n, "table"), p.total_q, p.n_heads, c.n_kv_heads, c.head_dim);
    if (bytes) work = on.empty({(int64_t)bytes}, at::kByte, q);
  }
  if (work.defined()) std::tie(p.d_work, p.work_bytes) = workspace(work);
  const entro_kv_table tb = table_of(table, n);
  uint32_t *const flags = static_cast<uint32_t *>(ints(status, "status", n));
  const c10::DeviceGuard guard(q.device());
  done(g.chunk(&c, &tb, &p, flags, on.handle(q)), "entro_attn_chunk");
  return THPVariable_Wrap(std::move(out));
}

// Positions of a call's rows on the axes of r; a tensor of one dimension is one axis.
const int32_t *positions_of(const at::Tensor &x, const entro_rotary &r, int64_t rows, int64_t *stride) {
  const bool flat = x.dim() == 1 && r.n_axes == 1;
  if (x.scalar_type() != at::kInt || !x.is_cuda() || !(flat || (x.dim() == 2 && x.size(0) == r.n_axes)) || x.size(-1) != rows)
    refuse("positions: int32 [", r.n_axes, "][", rows, "] on the GPU expected, got ", x.scalar_type(), " ", x.sizes(), " on ",
           x.device());
  if (rows > 1 && x.stride(-1) != 1) refuse("positions: those of an axis have to lie side by side");
  *stride = r.n_axes > 1 ? x.stride(0) : 0;
  return static_cast<const int32_t *>(x.data_ptr());
}

// An operand of 32 or 16 bits, and the type of what it becomes: float16 or bfloat16.
entro_dtype in_type(const at::Tensor &x) {
  if (x.scalar_type() == at::kFloat) return ENTRO_F32;
  if (x.scalar_type() == at::kBFloat16) return ENTRO_BF16;
  if (x.scalar_type() == at::kHalf) return ENTRO_F16;
  refuse("element type ", x.scalar_type(), ": float32, bfloat16 or float16 expected");
}

// rotary, q, k, positions, type of the results as bf16 (False) or f16 (True), q_out, k_out, make, stream -> (q, k)
PyObject *rope(Args a) {
  const RotaryDesc r = desc_of<RotaryDesc>(a[0], "rotary: a Rotary expected");
  const at::Tensor &positions = tensor(a[3], "positions");
  const Together together{r.device()};
  at::Tensor x[2], out[2];
  static const char *const kNames[2] = {"q", "k"}, *const kOuts[2] = {"q_out", "k_out"};
  for (int i = 0; i < 2; ++i) {
    if (a[1 + i] != Py_None) together(kNames[i], x[i] = tensor(a[1 + i], kNames[i]));
    if (a[5 + i] == Py_None) continue;
    if (!x[i].defined()) refuse(kOuts[i], ": there is no ", kNames[i]);
    together(kOuts[i], out[i] = tensor(a[5 + i], kOuts[i]));
  }
  together("positions", positions);
  const On on{a[7] == Py_True, a[8]};
  const at::Tensor &first = x[0].defined() ? x[0] : x[1];
  if (!first.defined()) refuse("q or k expected");
  if (first.dim() != 3) refuse("q and k are [rows][heads][dim]");
  const int64_t n = first.size(0), dim = first.size(2);
  entro_rope_args p{};
  p.in = in_type(first);
  const at::ScalarType t = a[4] == Py_True ? at::kHalf : at::kBFloat16;
  p.out = t == at::kHalf ? ENTRO_F16 : ENTRO_BF16;
  p.rows = small(n, "rows");
  p.head_dim = small(dim, "dim");
  p.d_pos = positions_of(positions, r.r, n, &p.pos_stride);
  for (int i = 0; i < 2; ++i) {
    if (!x[i].defined()) continue;
    if (x[i].dim() != 3 || x[i].size(0) != n) refuse("q and k have the same rows");
    const int64_t heads = x[i].size(1);
    (i ? p.k : p.q) = rows(x[i], kNames[i], first.scalar_type(), heads, dim);
    if (!out[i].defined()) out[i] = on.empty(x[i].sizes(), t, x[i]);
    if (out[i].dim() == 3 && out[i].size(0) != n) refuse(kOuts[i], " has the rows of ", kNames[i]);
    (i ? p.k_out : p.q_out) = rows(out[i], kOuts[i], t, heads, dim);
    (i ? p.n_kv_heads : p.n_heads) = small(heads, kNames[i]);
  }
  const c10::DeviceGuard guard(first.device());
  done(g.rope(&r.r, &p, on.handle(first)), "entro_rope");
  PyObject *y[2];
  for (int i = 0; i < 2; ++i) {
    if (out[i].defined()) {
      y[i] = THPVariable_Wrap(std::move(out[i]));
    } else {
      Py_INCREF(Py_None);
      y[i] = Py_None;
    }
  }
  PyObject *both = y[0] && y[1] ? PyTuple_Pack(2, y[0], y[1]) : nullptr;
  Py_XDECREF(y[0]);
  Py_XDECREF(y[1]);
  return both;
}

// cache, rotary, k, v, table, held, cu_new, status, positions, q, type of its result as in rope, q_out, make, stream -> q_out
PyObject *append(Args a) {
  const CacheDesc desc = cache_of(a[0]);
  const RotaryDesc r = desc_of<RotaryDesc>(a[1], "rotary: a Rotary expected");
  const entro_kv_cache &c = desc.c;
  const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &table = tensor(a[4], "table");
  const at::Tensor &held = tensor(a[5], "held"), &cu_new = tensor(a[6], "cu_new"), &status = tensor(a[7], "status");
  at::Tensor positions, q, out;
  const Together together{desc.device()};
  if (r.device() != desc.device()) refuse("rotary: on device ", r.device(), ", the call is on ", desc.device());
  together("k", k)("v", v)("table", table)("held", held)("cu_new", cu_new)("status", status);
  if (a[8] != Py_None) together("positions", positions = tensor(a[8], "positions"));
  if (a[9] != Py_None) together("q", q = tensor(a[9], "q"));
  if (a[11] != Py_None) {
    if (!q.defined()) refuse("q_out: there is no q");
    together("q_out", out = tensor(a[11], "q_out"));
  }
  const On on{a[12] == Py_True, a[13]};
  if (k.dim() != 3 || v.dim() != 3 || k.size(0) != v.size(0)) refuse("k and v have the same rows");
  const int64_t n = table.dim() ? table.size(0) : 0, total = k.size(0);
  entro_kv_append_args p{};
  p.in = in_type(k);
  const at::ScalarType t = a[10] == Py_True ? at::kHalf : at::kBFloat16;
  p.out = t == at::kHalf ? ENTRO_F16 : ENTRO_BF16;
  p.k = rows(k, "k", k.scalar_type(), c.n_kv_heads, c.head_dim);
  p.v = rows(v, "v", k.scalar_type(), c.n_kv_heads, c.head_dim);
  p.d_held = static_cast<int32_t *>(ints(held, "held", n));
  p.d_cu_new = static_cast<int32_t *>(ints(cu_new, "cu_new", n + 1));
  p.total_new = small(total, "k");
  if (positions.defined()) p.d_pos = positions_of(positions, r.r, total, &p.pos_stride);
  if (q.defined()) {
    if (q.dim() != 3 || q.size(0) != total) refuse("q has the rows of k");
    const int64_t heads = q.size(1);
    p.q = rows(q, "q", k.scalar_type(), heads, c.head_dim);
    if (!out.defined()) out = on.empty(q.sizes(), t, q);
    if (out.dim() == 3 && out.size(0) != total) refuse("q_out has the rows of q");
    p.q_out = rows(out, "q_out", t, heads, c.head_dim);
    p.n_heads = small(heads, "q");
  }
  const entro_kv_table tb = table_of(table, n);
  uint32_t *const flags = static_cast<uint32_t *>(ints(status, "status", n));
  const c10::DeviceGuard guard(k.device());
  done(g.append(&c, &tb, &r.r, &p, flags, on.handle(k)), "entro_kv_append");
  if (!out.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
}

// freqs, axes (a sequence of the pairs' axes, or None), interleaved, gain -> RotaryDesc as bytes
PyObject *rotary_desc(Args a) {
  const at::Tensor &freqs = tensor(a[0], "freqs");
  if (freqs.scalar_type() != at::kFloat || freqs.dim() != 1 || !freqs.is_cuda() || !freqs.is_contiguous())
    refuse("freqs: contiguous float32 [pairs] on the GPU expected, got ", freqs.scalar_type(), " ", freqs.sizes(), " on ",
           freqs.device());
  Together{freqs.device()}("freqs", freqs);
  RotaryDesc d{};
  d.gpu = freqs.device().index();
  d.r.d_freqs = static_cast<const float *>(freqs.data_ptr());
  const int64_t pairs = freqs.size(0);
  if (pairs < 1 || pairs > 64 || pairs % 8) refuse("freqs: 8, 16, .. 64 pairs expected, got ", pairs);
  d.r.pairs = (uint32_t)pairs;
  d.r.n_axes = 1;
  if (a[1] != Py_None) {
    PyObject *axes = PySequence_Fast(a[1], "axes: a sequence expected");
    if (!axes) throw Raised();
    const bool fits = PySequence_Fast_GET_SIZE(axes) == pairs;
    bool fine = true;
    for (int64_t i = 0; fits && i < pairs; ++i) {
      const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(axes, i));
      if (x == -1 && PyErr_Occurred()) {
        Py_DECREF(axes);
        throw Raised();
      }
      if (x < 0 || x > 3) fine = false;
      d.r.axes[i / 16] |= (uint32_t)(x & 3) << (2 * (i % 16));
      d.r.n_axes = std::max<uint32_t>(d.r.n_axes, (uint32_t)(x & 3) + 1);
    }
    Py_DECREF(axes);
    if (!fits || !fine) refuse("axes: the axis, 0 to 3, of each of the ", pairs, " pairs expected");
  }
  d.r.interleaved = PyObject_IsTrue(a[2]) == 1;
  const double gain = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) throw Raised();
  d.r.gain = (float)gain;
  if (!std::isfinite(d.r.gain)) refuse("gain: ", gain, " is not a finite 32-bit number");
  return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&d), sizeof d);
}

// k_codes, v_codes, k_scales, v_scales -> CacheDesc as bytes
PyObject *cache_desc(Args a) {
  const at::Tensor &k = tensor(a[0], "k_codes"), &v = tensor(a[1], "v_codes");
  const at::Tensor &ks = tensor(a[2], "k_scales"), &vs = tensor(a[3], "v_scales");
  if (k.dim() != 4 || v.dim() != 4) refuse("k_codes and v_codes have four dimensions");
  const int64_t pages = k.size(0), kv = k.size(1), page = k.size(2), dim = k.size(3);
  if (v.sizes() != at::IntArrayRef({pages, kv, dim, page}) || ks.sizes() != at::IntArrayRef({pages, kv}) ||
      vs.sizes() != at::IntArrayRef({pages, kv}))
    refuse("the shapes of codes and scales do not belong together");
  for (const at::Tensor *x : {&k, &v, &ks, &vs})
    if (x->scalar_type() != (x->dim() == 4 ? at::kChar : at::kFloat) || !x->is_cuda() || !x->is_contiguous())
      refuse("int8 codes and float32 scales, contiguous and on the GPU, expected");
  Together{k.device()}("k_codes", k)("v_codes", v)("k_scales", ks)("v_scales", vs);
  const CacheDesc c = {{static_cast<int8_t *>(k.data_ptr()), static_cast<int8_t *>(v.data_ptr()),
                        static_cast<float *>(ks.data_ptr()), static_cast<float *>(vs.data_ptr()), small(pages, "pages"),
                        small(page, "page"), small(kv, "heads"), small(dim, "dim")},
                       k.device().index()};
  return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&c), sizeof c);
}

template <PyObject *(*F)(Args), Py_ssize_t N>
PyObject *entry(PyObject *, Args a, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(a);
  } catch (const Raised &) {
    return nullptr;
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &) {   // torch's own, as torch raises them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// The addresses of the library's ten functions, raw_stream, check.
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long f[10];
  PyObject *raw_stream, *check;
  if (!PyArg_ParseTuple(args, "KKKKKKKKKKOO", f, f + 1, f + 2, f + 3, f + 4, f + 5, f + 6, f + 7, f + 8, f + 9, &raw_stream,
                        &check))
    return nullptr;
  g.prompt = reinterpret_cast<decltype(g.prompt)>(f[0]);
  g.prompt_bytes = reinterpret_cast<decltype(g.prompt_bytes)>(f[1]);
  g.store = reinterpret_cast<decltype(g.store)>(f[2]);
  g.load = reinterpret_cast<decltype(g.load)>(f[3]);
  g.cache = reinterpret_cast<decltype(g.cache)>(f[4]);
  g.cache_bytes = reinterpret_cast<decltype(g.cache_bytes)>(f[5]);
  g.rope = reinterpret_cast<decltype(g.rope)>(f[6]);
  g.append = reinterpret_cast<decltype(g.append)>(f[7]);
  g.chunk = reinterpret_cast<decltype(g.chunk)>(f[8]);
  g.chunk_bytes = reinterpret_cast<decltype(g.chunk_bytes)>(f[9]);
  Py_INCREF(raw_stream);
  Py_INCREF(check);
  Py_XSETREF(g.raw_stream, raw_stream);
  Py_XSETREF(g.check, check);
  if (!g.desc && !(g.desc = PyUnicode_InternFromString("desc"))) return nullptr;
  Py_RETURN_NONE;
}

template <PyObject *(*F)(Args), Py_ssize_t N>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<prompt, 11>("attn_prompt"),
    method<store, 9>("kv_store"),
    method<load, 11>("kv_load"),
    method<cache, 10>("attn_cache"),
    method<rope, 9>("rope"),
    method<append, 14>("kv_append"),
    method<chunk, 11>("attn_chunk"),
    method<cache_desc, 4>("cache_desc"),
    method<rotary_desc, 4>("rotary_desc"),
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn() { return PyModule_Create(&module); }
