// Python module _qkbind: the checks and allocations of the calls that stand
// between a decoder layer's linears (norm, cache, attention), in C++.
//
// These kernels run for a few microseconds at decode sizes; the same checks in
// Python took 7 to 10 us a call (about 0.6 us per checked tensor, 1.6 us per
// allocation) and were what bounded the smallest calls.  Here they take about
// 2 us.  Only torch's tensor interface is used: attributes, at::empty, and the
// current stream through torch's Python function.  Errors are the Python
// exceptions that the package's other calls raise (TypeError, ValueError,
// QKError); none of C++'s crosses into Python.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <map>
#include <memory>
#include <string>
#include <utility>

namespace {

// libqk's entry points (include/qk.h), as addresses handed over by the
// package; hipStream_t is a pointer.
struct Lib {
  int (*norm)(int, int, const void*, int64_t, const void*, int64_t, const void*, int, int, double, int, void*,
              int64_t, void*, float*, void*);
  int (*write)(int, int, int, int, const void*, int64_t, const void*, int64_t, int, void*, void*, float*, float*,
               int, int, int, const int*, int64_t, int, const int*, const int*, void*);
  int (*read)(int, int, int, int, void*, int64_t, void*, int64_t, int, const void*, const void*, const float*,
              const float*, int, int, int, const int*, int64_t, int, const int*, const int*, void*);
  size_t (*workspace)(int, int, int, int, int, int, int, int, int);
  int (*attention)(int, int, int, int, int, const void*, int64_t, int, const void*, const void*, const float*,
                   const float*, int, int, int, const int*, int64_t, int, const int*, const int*, int, int, float,
                   int, void*, float*, void*, size_t, void*);
};
Lib lib;
PyObject* py_check = nullptr;          // check(status): raises for a status other than 0
PyObject* py_stream = nullptr;         // current stream of a device index, as a number
PyObject* py_new_workspace = nullptr;  // (bytes, device index) -> a workspace prepared on the current stream
PyObject* py_capturing = nullptr;      // whether the current stream is being captured

// A Python exception on its way out; Raised: it is set already.
struct Raise {
  PyObject* type;
  std::string text;
};
struct Raised {};

[[noreturn]] void value_error(std::string text) { throw Raise{PyExc_ValueError, std::move(text)}; }
[[noreturn]] void type_error(std::string text) { throw Raise{PyExc_TypeError, std::move(text)}; }

std::string dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kChar: return "torch.int8";
    case at::kInt: return "torch.int32";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return std::string("torch.") + c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) value_error(std::string(name) + " must be a GPU tensor");
  return t;
}

void on_device(const at::Tensor& t, const char* name, const c10::Device& dev) {
  if (t.device() != dev) value_error(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
}

void has_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + dtype_name(type) + ", got " + dtype_name(t.scalar_type()));
}

void has_dims(const at::Tensor& t, const char* name, int64_t n) {
  if (t.dim() != n) value_error(std::string(name) + " must have " + std::to_string(n) + " dimensions");
}

// A dense tensor of this type and number of dimensions (0: any).
const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, int64_t dims, const c10::Device& dev) {
  const at::Tensor& t = tensor(o, name);
  has_type(t, name, type);
  on_device(t, name, dev);
  if (dims) has_dims(t, name, dims);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t;
}

// The row stride of a tensor whose rows (the dimensions after the first) are
// dense and do not overlap.
int64_t row_stride(const at::Tensor& t, const char* name, int64_t dims) {
  has_dims(t, name, dims);
  const auto shape = t.sizes(), stride = t.strides();
  int64_t inner = 1;
  for (int64_t i = dims - 1; i > 0; --i) {
    if (stride[i] != inner && shape[i] != 1 && shape[0])
      value_error(std::string("the rows of ") + name + " must be dense");
    inner *= shape[i];
  }
  if (shape[0] <= 1) return inner;
  if (stride[0] < inner) value_error(std::string("the rows of ") + name + " must not overlap");
  return stride[0];
}

// libqk's number of an input type, or -1.
int type_code(at::ScalarType t) {
  return t == at::kFloat ? 0 : t == at::kBFloat16 ? 1 : t == at::kHalf ? 2 : -1;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const c10::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// Sizes go to libqk as ints.
int narrow(int64_t v, const char* what) {
  if (v < 0 || v > 0x7fffffff) value_error(std::string(what) + " does not fit in 31 bits");
  return static_cast<int>(v);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

void* stream_of(const c10::Device& dev) {
  PyObject* index = PyLong_FromLong(dev.index());
  PyObject* got = index ? PyObject_CallOneArg(py_stream, index) : nullptr;
  Py_XDECREF(index);
  if (!got) throw Raised{};
  void* s = PyLong_AsVoidPtr(got);
  Py_DECREF(got);
  if (!s && PyErr_Occurred()) throw Raised{};
  return s;
}

void check(int status) {
  if (status == 0) return;
  PyObject* got = PyObject_CallFunction(py_check, "i", status);
  Py_XDECREF(got);
  throw Raised{};
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("expected " + std::to_string(want) + " arguments");
}

PyObject* wrapped(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw Raised{};
  return o;
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {  // takes the references
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_DECREF(o);
  }
  if (!t) throw Raised{};
  return t;
}

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// ---- norm ----

// (x, weight, eps, residual, fp8, residual_out, q, scale)
PyObject* rms_norm_quant(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 8);
  const at::Tensor& x = tensor(a[0], "x");
  const at::ScalarType dt = x.scalar_type();
  const int code = type_code(dt);
  if (code < 0) type_error("x dtype " + dtype_name(dt) + " not supported");
  const c10::Device dev = x.device();
  const int64_t ldx = row_stride(x, "x", 2);
  const int64_t m = x.size(0), k = x.size(1);
  const at::Tensor& w = tensor(a[1], "weight");
  if (w.scalar_type() != dt && w.scalar_type() != at::kFloat)
    type_error("weight must be " + dtype_name(dt) + " or fp32, got " + dtype_name(w.scalar_type()));
  on_device(w, "weight", dev);
  has_dims(w, "weight", 1);
  if (!w.is_contiguous()) value_error("weight must be contiguous");
  if (w.size(0) != k) value_error("weight must be [k]");
  const bool fp8 = truth(a[4]);

  const void* res = nullptr;
  at::Tensor r_out;
  int64_t ldr = 0, ldo = 0;
  const bool residual = a[3] != Py_None;
  if (residual) {
    const at::Tensor& r = tensor(a[3], "residual");
    has_type(r, "residual", dt);
    on_device(r, "residual", dev);
    ldr = row_stride(r, "residual", 2);
    if (r.sizes() != x.sizes()) value_error("residual and residual_out must be [m, k]");
    res = r.data_ptr();
    if (a[5] != Py_None) {
      r_out = tensor(a[5], "residual_out");
      has_type(r_out, "residual_out", dt);
      on_device(r_out, "residual_out", dev);
      if (r_out.sizes() != x.sizes()) value_error("residual and residual_out must be [m, k]");
    } else {
      r_out = make(x.sizes(), dt, dev);
    }
    ldo = row_stride(r_out, "residual_out", 2);
  } else if (a[5] != Py_None) {
    value_error("residual_out needs a residual");
  }
  at::Tensor q, scale;
  if (a[6] != Py_None) {
    q = tensor(a[6], "q");
    if (!(fp8 && q.scalar_type() == at::kByte)) has_type(q, "q", fp8 ? at::kFloat8_e4m3fn : at::kChar);
    on_device(q, "q", dev);
    if (!q.is_contiguous()) value_error("q must be contiguous");
    if (q.sizes() != x.sizes()) value_error("q must be [m, k] and scale [m]");
  } else {
    q = make(x.sizes(), fp8 ? at::kFloat8_e4m3fn : at::kChar, dev);
  }
  if (a[7] != Py_None) {
    scale = dense(a[7], "scale", at::kFloat, 1, dev);
    if (scale.size(0) != m) value_error("q must be [m, k] and scale [m]");
  } else {
    scale = make({m}, at::kFloat, dev);
  }
  const c10::DeviceGuard guard(dev);
  check(lib.norm(narrow(m, "rows"), narrow(k, "columns"), x.data_ptr(), ldx, res, ldr, w.data_ptr(), code,
                 type_code(w.scalar_type()), number(a[2]), fp8, residual ? r_out.data_ptr() : nullptr, ldo,
                 q.data_ptr(), static_cast<float*>(scale.data_ptr()), stream_of(dev)));
  PyObject* const qo = a[6] != Py_None ? same(a[6]) : wrapped(q);
  PyObject* const so = a[7] != Py_None ? same(a[7]) : wrapped(scale);
  if (!residual) return tuple_of({qo, so});
  return tuple_of({qo, so, a[5] != Py_None ? same(a[5]) : wrapped(r_out)});
}

// ---- cache ----

struct Cache {
  at::Tensor k, v, ks, vs;
  int blocks, heads, block, dim, code;
  const int* table;
  int64_t ldt;
  int width;
};

// The four tensors of a KVCache and its block table.
Cache cache_of(PyObject* o, PyObject* table, int64_t seqs, const c10::Device& dev) {
  PyObject* const parts = PySequence_Fast(o, "cache must be a KVCache");
  if (!parts) throw Raised{};
  struct Hold {
    PyObject* p;
    ~Hold() { Py_DECREF(p); }
  } hold{parts};
  if (PySequence_Fast_GET_SIZE(parts) != 4) value_error("cache must be a KVCache of four tensors");
  PyObject** p = PySequence_Fast_ITEMS(parts);
  Cache c{tensor(p[0], "cache.k"), tensor(p[1], "cache.v"), tensor(p[2], "cache.k_scale"), tensor(p[3], "cache.v_scale"),
          0, 0, 0, 0, 0, nullptr, 0, 0};
  if (c.k.dim() != 4) value_error("cache.k must be [blocks, kv_heads, block, dim]");
  const int64_t blocks = c.k.size(0), heads = c.k.size(1), block = c.k.size(2), dim = c.k.size(3);
  const int64_t want_v[4] = {blocks, heads, dim, block}, want_s[2] = {blocks, heads};
  if (c.v.sizes() != at::IntArrayRef(want_v, 4) || c.ks.sizes() != at::IntArrayRef(want_s, 2) ||
      c.vs.sizes() != at::IntArrayRef(want_s, 2))
    value_error("cache.v must be [blocks, kv_heads, dim, block], the scales [blocks, kv_heads]");
  if (block != 16 && block != 32 && block != 64 && block != 128) value_error("block must be one of (16, 32, 64, 128)");
  if (dim % 16 || dim < 16 || dim > 256) value_error("dim must be a multiple of 16 from 16 to 256");
  const at::ScalarType dt = c.k.scalar_type();
  if ((dt != at::kChar && dt != at::kFloat8_e4m3fn) || c.v.scalar_type() != dt)
    type_error("cache codes must be int8 or float8_e4m3fn");
  if (c.ks.scalar_type() != at::kFloat || c.vs.scalar_type() != at::kFloat) type_error("cache scales must be fp32");
  const std::pair<const at::Tensor*, const char*> all[] = {
      {&c.k, "cache.k"}, {&c.v, "cache.v"}, {&c.ks, "cache.k_scale"}, {&c.vs, "cache.v_scale"}};
  for (const auto& t : all) {
    on_device(*t.first, t.second, dev);
    if (!t.first->is_contiguous()) value_error(std::string(t.second) + " must be contiguous");
  }
  const at::Tensor& tb = tensor(table, "table");
  has_type(tb, "table", at::kInt);
  on_device(tb, "table", dev);
  c.ldt = row_stride(tb, "table", 2);
  if (tb.size(0) != seqs) value_error("table must have one row for each of the " + std::to_string(seqs) + " sequences");
  c.blocks = narrow(blocks, "blocks");
  c.heads = narrow(heads, "kv_heads");
  c.block = static_cast<int>(block);
  c.dim = static_cast<int>(dim);
  c.code = dt == at::kChar ? 0 : 1;
  c.table = static_cast<const int*>(tb.data_ptr());
  c.width = narrow(tb.size(1), "the table's width");
  return c;
}

// The call that write and read share: k and v are read or written.
void cache_rows(bool write, PyObject* cache, PyObject* ko, PyObject* vo, PyObject* table, PyObject* start_o, PyObject* cu_o) {
  const at::Tensor& k = tensor(ko, "k");
  const at::ScalarType dt = k.scalar_type();
  const int code = type_code(dt);
  if (code < 0) type_error("k dtype " + dtype_name(dt) + " not supported");
  const c10::Device dev = k.device();
  const int64_t ldk = row_stride(k, "k", 3);
  const at::Tensor& v = tensor(vo, "v");
  has_type(v, "v", dt);
  on_device(v, "v", dev);
  const int64_t ldv = row_stride(v, "v", 3);
  const at::Tensor& start = dense(start_o, "start", at::kInt, 1, dev);
  const at::Tensor& cu = dense(cu_o, "cu", at::kInt, 1, dev);
  const int64_t seqs = start.size(0);
  const Cache c = cache_of(cache, table, seqs, dev);
  if (cu.size(0) != seqs + 1) value_error("cu must have one entry more than start");
  if (v.sizes() != k.sizes() || k.size(1) != c.heads || k.size(2) != c.dim)
    value_error("k and v must be [tokens, kv_heads, dim] of the cache's heads and dim");
  const c10::DeviceGuard guard(dev);
  const int ns = narrow(seqs, "sequences"), nt = narrow(k.size(0), "tokens");
  float* const ks = static_cast<float*>(c.ks.data_ptr());
  float* const vs = static_cast<float*>(c.vs.data_ptr());
  const int* const st = static_cast<const int*>(start.data_ptr());
  const int* const cp = static_cast<const int*>(cu.data_ptr());
  check(write ? lib.write(ns, nt, c.heads, c.dim, k.data_ptr(), ldk, v.data_ptr(), ldv, code, c.k.data_ptr(),
                          c.v.data_ptr(), ks, vs, c.blocks, c.block, c.code, c.table, c.ldt, c.width, st, cp, stream_of(dev))
              : lib.read(ns, nt, c.heads, c.dim, k.data_ptr(), ldk, v.data_ptr(), ldv, code, c.k.data_ptr(),
                         c.v.data_ptr(), ks, vs, c.blocks, c.block, c.code, c.table, c.ldt, c.width, st, cp, stream_of(dev)));
}

// (cache, k, v, table, start, cu)
PyObject* kv_cache_write(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 6);
  cache_rows(true, a[0], a[1], a[2], a[3], a[4], a[5]);
  return same(a[0]);
}

// (cache, table, start, cu, tokens, dtype number, k, v)
PyObject* kv_cache_read(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 8);
  const int64_t tokens = integer(a[4]), want = integer(a[5]);
  if (tokens < 0) value_error("tokens must not be negative");
  struct Ref {
    PyObject* p = nullptr;
    ~Ref() { Py_XDECREF(p); }
  } first, made_k, made_v;
  PyObject *ko = a[6], *vo = a[7];
  if (ko == Py_None || vo == Py_None) {
    first.p = PySequence_GetItem(a[0], 0);
    if (!first.p) throw Raised{};
    const at::Tensor& kc = tensor(first.p, "cache.k");
    if (kc.dim() != 4) value_error("cache.k must be [blocks, kv_heads, block, dim]");
    const int64_t shape[3] = {tokens, kc.size(1), kc.size(3)};
    const at::ScalarType dt = ko != Py_None ? tensor(ko, "k").scalar_type()
                              : want == 0   ? at::kFloat
                              : want == 1   ? at::kBFloat16
                                            : at::kHalf;
    if (ko == Py_None) ko = made_k.p = wrapped(make(at::IntArrayRef(shape, 3), dt, kc.device()));
    if (vo == Py_None) vo = made_v.p = wrapped(make(at::IntArrayRef(shape, 3), dt, kc.device()));
  }
  const at::Tensor& k = tensor(ko, "k");
  if (k.dim() > 0 && k.size(0) != tokens) value_error("k must have `tokens` rows");
  cache_rows(false, a[0], ko, vo, a[1], a[2], a[3]);
  return tuple_of({same(ko), same(vo)});
}

// ---- attention ----

// One prepared workspace per device and stream, for calls that are not being
// captured: a graph may be replayed on any stream, beside calls on the one it
// was captured on.  None is freed, since calls on its stream may still be
// running.  Each is at least twice the one before, so together they are at most
// twice the last.
std::map<std::pair<int, void*>, PyObject*>& workspaces() {
  static auto* all = new std::map<std::pair<int, void*>, PyObject*>;
  return *all;
}

// (q, cache, table, lens, cu, scale, window, max_q, max_kv, out, return_lse, workspace)
PyObject* kv_attention(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 12);
  const at::Tensor& q = tensor(a[0], "q");
  const at::ScalarType dt = q.scalar_type();
  if (dt != at::kBFloat16 && dt != at::kHalf) type_error("q dtype " + dtype_name(dt) + " not supported");
  const c10::Device dev = q.device();
  const int64_t ldq = row_stride(q, "q", 3);
  const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2);
  const at::Tensor& lens = dense(a[3], "lens", at::kInt, 1, dev);
  const int64_t seqs = lens.size(0);
  const Cache c = cache_of(a[1], a[2], seqs, dev);
  if (dim != c.dim || c.heads == 0 || heads % c.heads)
    value_error("q must be [tokens, heads, dim] with heads a multiple of the cache's and its dim");
  const int* cu = nullptr;
  const bool ragged = a[4] != Py_None;
  if (ragged) {
    const at::Tensor& t = dense(a[4], "cu", at::kInt, 1, dev);
    if (t.size(0) != seqs + 1) value_error("cu must have one entry more than lens");
    cu = static_cast<const int*>(t.data_ptr());
  } else if (tokens != seqs) {
    value_error("without cu every sequence has one row");
  }
  at::Tensor out, lse;
  if (a[9] != Py_None) {
    out = dense(a[9], "out", dt, 3, dev);
    if (out.sizes() != q.sizes()) value_error("out must be [tokens, heads, dim]");
  } else {
    out = make(q.sizes(), dt, dev);
  }
  const bool want_lse = truth(a[10]);
  if (want_lse) lse = make({tokens, heads}, at::kFloat, dev);
  const float scale = a[5] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim)))
                                      : static_cast<float>(number(a[5]));
  const int64_t window = integer(a[6]);
  const int64_t reach = static_cast<int64_t>(c.width) * c.block;
  int64_t max_q = a[7] != Py_None ? integer(a[7]) : ragged ? std::max<int64_t>(tokens, 1) : 1;
  int64_t max_kv = a[8] != Py_None ? std::min(integer(a[8]), reach) : reach;
  const int64_t top = 0x7fffffff;
  max_q = std::min(std::max<int64_t>(max_q, -1), top);
  max_kv = std::min(std::max<int64_t>(max_kv, -1), top);
  const int w = static_cast<int>(std::min(std::max<int64_t>(window, -1), top));
  const int ns = narrow(seqs, "sequences"), nt = narrow(tokens, "tokens"), nh = narrow(heads, "heads");

  const c10::DeviceGuard guard(dev);
  void* const stream = stream_of(dev);
  void* ws = nullptr;
  size_t bytes = 0;
  struct Release {
    void operator()(PyObject* o) const { Py_DECREF(o); }
  };
  std::unique_ptr<PyObject, Release> own;  // a workspace made for this call, until it is enqueued
  const std::pair<int, void*> key(dev.index(), stream);
  if (a[11] != Py_None) {
    const at::Tensor& t = tensor(a[11], "workspace");
    on_device(t, "workspace", dev);
    if (!t.is_contiguous()) value_error("workspace must be contiguous");
    ws = t.data_ptr();
    bytes = t.nbytes();
  } else {
    const size_t need = lib.workspace(ns, nt, nh, c.heads, c.dim, ragged, static_cast<int>(max_q), static_cast<int>(max_kv), w);
    if (need > 0) {
      PyObject* use = nullptr;
      size_t had = 0;
      const std::unique_ptr<PyObject, Release> capturing(PyObject_CallNoArgs(py_capturing));
      if (!capturing) throw Raised{};
      const bool keep = !truth(capturing.get());
      const auto at = workspaces().find(key);
      if (keep && at != workspaces().end()) {
        use = at->second;
        had = THPVariable_Unpack(use).nbytes();
      }
      if (had < need) {
        use = PyObject_CallFunction(py_new_workspace, "ni", static_cast<Py_ssize_t>(std::max(need, 2 * had)),
                                    static_cast<int>(dev.index()));
        if (!use) throw Raised{};
        own.reset(use);
        if (keep) workspaces()[key] = own.release();
      }
      ws = THPVariable_Unpack(use).data_ptr();
      bytes = THPVariable_Unpack(use).nbytes();
    }
  }
  const int status = lib.attention(
      ns, nt, nh, c.heads, c.dim, q.data_ptr(), ldq, type_code(dt), c.k.data_ptr(), c.v.data_ptr(),
      static_cast<const float*>(c.ks.data_ptr()), static_cast<const float*>(c.vs.data_ptr()), c.blocks, c.block, c.code,
      c.table, c.ldt, c.width, static_cast<const int*>(lens.data_ptr()), cu, static_cast<int>(max_q),
      static_cast<int>(max_kv), scale, w, out.data_ptr(), want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws,
      bytes, stream);
  if (status != 0 && status < 1000) workspaces().erase(key);  // part of the call may have run: a fresh one next time
  check(status);
  PyObject* const oo = a[9] != Py_None ? same(a[9]) : wrapped(out);
  return want_lse ? tuple_of({oo, wrapped(lse)}) : oo;
}

// ---- module ----

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (const Raise& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const Raised&) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "libqk call failed");
  } catch (...) {  // torch's errors, out of memory among them, as torch raises them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// (addresses of the five entry points, check, stream, new_workspace, capturing)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  need_args(n, 9);
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (PyErr_Occurred()) throw Raised{};
      value_error("an entry point has no address");
    }
  }
  lib.norm = reinterpret_cast<decltype(lib.norm)>(p[0]);
  lib.write = reinterpret_cast<decltype(lib.write)>(p[1]);
  lib.read = reinterpret_cast<decltype(lib.read)>(p[2]);
  lib.workspace = reinterpret_cast<decltype(lib.workspace)>(p[3]);
  lib.attention = reinterpret_cast<decltype(lib.attention)>(p[4]);
  PyObject** const hold[] = {&py_check, &py_stream, &py_new_workspace, &py_capturing};
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(a[5 + i]);
    Py_XDECREF(*hold[i]);
    *hold[i] = a[5 + i];
  }
  Py_RETURN_NONE;
}

#define QK_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {QK_METHOD(bind),          QK_METHOD(rms_norm_quant), QK_METHOD(kv_cache_write),
                         QK_METHOD(kv_cache_read), QK_METHOD(kv_attention),   {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qkbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qkbind() { return PyModule_Create(&module); }
