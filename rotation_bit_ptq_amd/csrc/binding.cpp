// The binding of the operators that are called once per layer and decode
// step (block_norm, adapter_add, kv_append, kv_read, paged_attention): checks
// of the tensors, allocation of the outputs, and the call of the C ABI, in a
// few microseconds less than the same in Python.  The functions here take
// their arguments by position; names, defaults and documentation are those of
// rotation_bit_ptq_amd/__init__.py.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/orbit.h"

namespace {

PyObject* g_error = nullptr;       // rotation_bit_ptq_amd.OrbitError
PyObject* g_raw_stream = nullptr;  // the current stream of a GPU, as an integer

// A refusal: Python's error is set, by refuse() an OrbitError.
struct Refused {};

template <class... A>
[[noreturn]] void refuse(const char* format, A... args) {
  PyErr_Format(g_error, format, args...);
  throw Refused();
}

typedef std::initializer_list<int64_t> Shape;

std::string text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

// A tensor on a GPU, of `dims` dimensions (any number if negative).
const at::Tensor& tensor(PyObject* o, const char* name, int64_t dims) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse("%s must be a torch tensor on a GPU", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (dims >= 0 && t.dim() != dims) refuse("%s must have %lld dimension(s), got %lld", name, (long long)dims, (long long)t.dim());
  return t;
}

// `t` lies on GPU `dev`, has this shape and type, and its innermost dimension
// is contiguous.
void check(const at::Tensor& t, const char* name, int dev, Shape shape, at::ScalarType type) {
  if (t.get_device() != dev) refuse("%s must be on GPU %d, where the first argument is", name, dev);
  if (t.sizes() != at::IntArrayRef(shape)) refuse("%s must be %s, got %s", name, text(shape).c_str(), text(t.sizes()).c_str());
  if (t.scalar_type() != type) refuse("%s must be %s, got %s", name, at::toString(type), at::toString(t.scalar_type()));
  if (t.dim() && t.stride(-1) != 1 && t.size(-1) > 1 && t.numel()) refuse("%s's innermost dimension must be contiguous", name);
}
const at::Tensor& checked(PyObject* o, const char* name, int dev, Shape shape, at::ScalarType type) {
  const at::Tensor& t = tensor(o, name, (int64_t)shape.size());
  check(t, name, dev, shape, type);
  return t;
}
void dense(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
}

// A floating type's orbit_dtype.
int32_t dtype(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kFloat: return ORBIT_F32;
    case at::kBFloat16: return ORBIT_BF16;
    case at::kHalf: return ORBIT_F16;
    default: refuse("%s must be float32, bfloat16 or float16", name);
  }
}
at::ScalarType type_of(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) refuse("a dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();  // the object's own error
  return v != 0;
}

at::Tensor fresh(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type));
}

// The call itself, on the current stream of `dev` and with that GPU current.
template <class F>
void launch(const char* what, int dev, F call) {
  PyObject* const s = PyObject_CallFunction(g_raw_stream, "i", dev);
  if (!s) throw Refused();
  const hipStream_t stream = (hipStream_t)PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (PyErr_Occurred()) throw Refused();
  int before = dev;
  (void)hipGetDevice(&before);
  if (before != dev) (void)hipSetDevice(dev);
  const orbit_status st = call(stream);
  if (before != dev) (void)hipSetDevice(before);
  if (st == ORBIT_OK) return;
  int hip = 0;
  if (st == ORBIT_E_HIP) orbit_last_hip_error(&hip);
  refuse("%s: %s (status %d, hip %d)", what, orbit_status_string(st), (int)st, hip);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* const p = PyTuple_New(2);
  if (!p) throw Refused();
  PyTuple_SET_ITEM(p, 0, wrap(a));
  PyTuple_SET_ITEM(p, 1, wrap(b));
  return p;
}

// x, branch, weight, norm, post, post_weight, gate, scale, shift, groups,
// residual_scale, eps, out_dtype, r_out, out
PyObject* block_norm(PyObject* const* v) {
  const at::Tensor& x = tensor(v[0], "x", 2);
  const int dev = x.get_device();
  const int64_t M = x.size(0), D = x.size(1);
  const at::ScalarType xt = x.scalar_type();
  orbit_block_norm_args a = {};
  a.x_dtype = dtype(xt, "x");
  check(x, "x", dev, {M, D}, xt);
  a.x = x.data_ptr();
  a.x_stride = x.stride(0);
  a.rows = M;
  a.dim = D;
  a.groups = 1;
  a.norm = (int32_t)integer(v[3]);
  a.post = (int32_t)integer(v[4]);
  a.residual_scale = (float)number(v[10]);
  a.eps = (float)number(v[11]);
  const bool branch = v[1] != Py_None, norm = a.norm != ORBIT_NORM_NONE;
  at::Tensor r, y;
  if (branch) {
    const at::Tensor& b = tensor(v[1], "branch", 2);
    a.branch_dtype = dtype(b.scalar_type(), "branch");
    check(b, "branch", dev, {M, D}, b.scalar_type());
    a.branch = b.data_ptr();
    a.branch_stride = b.stride(0);
    r = v[13] == Py_None ? fresh(x, x.sizes(), xt) : checked(v[13], "r_out", dev, {M, D}, xt);
    a.r_out = r.data_ptr();
    a.r_stride = r.stride(0);
  } else if (!norm) {
    refuse("block_norm needs a branch, a norm, or both");
  } else if (a.post != ORBIT_NORM_NONE || v[5] != Py_None || v[6] != Py_None || v[13] != Py_None) {
    refuse("post, post_weight, gate and r_out need a branch");
  }
  if (norm) {
    if (v[14] == Py_None) {
      y = fresh(x, x.sizes(), type_of(v[12], xt));
    } else {
      const at::Tensor& out = tensor(v[14], "out", 2);
      check(out, "out", dev, {M, D}, type_of(v[12], out.scalar_type()));
      y = out;
    }
    a.y_dtype = dtype(y.scalar_type(), "out");
    a.y_out = y.data_ptr();
    a.y_stride = y.stride(0);
  } else if (v[2] != Py_None || v[7] != Py_None || v[8] != Py_None || v[14] != Py_None) {
    refuse("weight, scale, shift and out need a norm");
  }
  const char* first = nullptr;  // the parameters share one type
  at::ScalarType pt = at::kFloat;
  auto typed = [&](PyObject* o, const char* name, int64_t dims) -> const at::Tensor& {
    const at::Tensor& t = tensor(o, name, dims);
    if (!first) {
      pt = t.scalar_type();
      a.p_dtype = dtype(pt, name);
      first = name;
    }
    return t;
  };
  auto vector = [&](PyObject* o, const char* name, const void*& to) {
    if (o == Py_None) return;
    const at::Tensor& t = typed(o, name, 1);
    check(t, name, dev, {D}, pt);
    to = t.data_ptr();
  };
  vector(v[2], "weight", a.weight);
  vector(v[5], "post_weight", a.post_weight);
  bool modulated = false;
  auto rows = [&](PyObject* o, const char* name, const void*& to, int64_t& stride) {
    if (o == Py_None) return;
    const at::Tensor& t = typed(o, name, 2);
    if (!modulated) {
      if (t.size(0) < 1) refuse("%s must have a row", name);
      a.groups = t.size(0);
      modulated = true;
    }
    check(t, name, dev, {a.groups, D}, pt);
    to = t.data_ptr();
    stride = t.stride(0);
  };
  rows(v[6], "gate", a.gate, a.gate_stride);
  rows(v[7], "scale", a.scale, a.scale_stride);
  rows(v[8], "shift", a.shift, a.shift_stride);
  if (v[9] != Py_None) a.group_ids = (const int32_t*)checked(v[9], "groups", dev, {M}, at::kInt).data_ptr();
  // an empty branch has no address to tell it from none
  if (M) launch("orbit_block_norm", dev, [&](hipStream_t s) { return orbit_block_norm(&a, s); });
  return !branch ? wrap(y) : !norm ? wrap(r) : pair(r, y);
}

// y, x, A, B, ids, scale, ranks, out
PyObject* adapter_add(PyObject* const* v) {
  const at::Tensor& x = tensor(v[1], "x", 2);
  const int dev = x.get_device();
  const at::Tensor &y = tensor(v[0], "y", 2), &A = tensor(v[2], "A", 3), &B = tensor(v[3], "B", 3);
  const at::ScalarType xt = x.scalar_type(), yt = y.scalar_type();
  if (xt != at::kBFloat16 && xt != at::kHalf) refuse("x must be bfloat16 or float16");
  orbit_adapter_args a = {};
  a.M = x.size(0);
  a.K = x.size(1);
  a.N = y.size(1);
  a.adapters = A.size(0);
  a.rank = A.size(1);
  a.x_dtype = dtype(xt, "x");
  a.y_dtype = dtype(yt, "y");
  check(x, "x", dev, {a.M, a.K}, xt);
  check(y, "y", dev, {a.M, a.N}, yt);
  check(A, "A", dev, {a.adapters, a.rank, a.K}, xt);
  check(B, "B", dev, {a.adapters, a.N, a.rank}, xt);
  dense(A, "A");
  dense(B, "B");
  a.x = x.data_ptr();
  a.y = y.data_ptr();
  a.A = A.data_ptr();
  a.B = B.data_ptr();
  a.x_stride = x.stride(0);
  a.y_stride = y.stride(0);
  a.ids = (const int32_t*)checked(v[4], "ids", dev, {a.M}, at::kInt).data_ptr();
  if (v[5] != Py_None) a.scale = (const float*)checked(v[5], "scale", dev, {a.adapters}, at::kFloat).data_ptr();
  if (v[6] != Py_None) a.ranks = (const int32_t*)checked(v[6], "ranks", dev, {a.adapters}, at::kInt).data_ptr();
  const at::Tensor out = v[7] == Py_None ? fresh(y, {a.M, a.N}, yt) : checked(v[7], "out", dev, {a.M, a.N}, yt);
  a.out = out.data_ptr();
  a.out_stride = out.stride(0);
  a.workspace_bytes = orbit_adapter_workspace(a.M, a.K, a.rank);
  if (a.workspace_bytes < 0)
    refuse("orbit_adapter_add: invalid shape (M %lld, K %lld, rank %lld)", (long long)a.M, (long long)a.K, (long long)a.rank);
  const at::Tensor work = fresh(x, {a.workspace_bytes}, at::kByte);
  a.workspace = work.data_ptr();
  launch("orbit_adapter_add", dev, [&](hipStream_t s) { return orbit_adapter_add(&a, s); });
  return wrap(out);
}

// The cache [pages, heads, page size, head dim] of four arguments.
orbit_kv_cache cache_of(PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso, int dev) {
  const at::Tensor &k = tensor(ko, "k_cache", 4), &v = tensor(vo, "v_cache", 4);
  orbit_kv_cache c = {};
  switch (k.scalar_type()) {
    case at::kBFloat16: c.format = ORBIT_KV_BF16; break;
    case at::kHalf: c.format = ORBIT_KV_F16; break;
    case at::kChar: c.format = ORBIT_KV_INT8; break;
    default: refuse("k_cache and v_cache must be bfloat16, float16 or int8");
  }
  const int64_t pages = k.size(0), heads = k.size(1), page = k.size(2), dim = k.size(3);
  check(k, "k_cache", dev, {pages, heads, page, dim}, k.scalar_type());
  check(v, "v_cache", dev, {pages, heads, page, dim}, k.scalar_type());
  dense(k, "k_cache");
  dense(v, "v_cache");
  if (heads > 1024 || page > 1024 || dim > 256) refuse("k_cache: heads, page size or head dimension too large: %s", text(k.sizes()).c_str());
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.pages = pages;
  c.kv_heads = (int32_t)heads;
  c.page_size = (int32_t)page;
  c.head_dim = (int32_t)dim;
  if (c.format == ORBIT_KV_INT8) {
    const at::Tensor &ks = checked(kso, "k_scale", dev, {pages, heads, page}, at::kHalf),
                     &vs = checked(vso, "v_scale", dev, {pages, heads, page}, at::kHalf);
    dense(ks, "k_scale");
    dense(vs, "v_scale");
    c.k_scale = ks.data_ptr();
    c.v_scale = vs.data_ptr();
  } else if (kso != Py_None || vso != Py_None) {
    refuse("k_scale and v_scale belong to an int8 cache");
  }
  return c;
}

// k, v, k_cache, v_cache, slots, positions, cos_sin, interleaved, q, q_out,
// k_scale, v_scale, hadamard
PyObject* kv_append(PyObject* const* v) {
  const at::Tensor& k = tensor(v[0], "k", 3);
  const int dev = k.get_device();
  const at::ScalarType kt = k.scalar_type();
  orbit_kv_append_args a = {};
  a.in_dtype = dtype(kt, "k");
  a.cache = cache_of(v[2], v[3], v[10], v[11], dev);
  const int64_t T = k.size(0), heads = a.cache.kv_heads, dim = a.cache.head_dim;
  check(k, "k", dev, {T, heads, dim}, kt);
  const at::Tensor& val = checked(v[1], "v", dev, {T, heads, dim}, kt);
  a.tokens = T;
  a.k = k.data_ptr();
  a.v = val.data_ptr();
  a.k_token_stride = k.stride(0);
  a.k_head_stride = k.stride(1);
  a.v_token_stride = val.stride(0);
  a.v_head_stride = val.stride(1);
  a.slots = (const int64_t*)checked(v[4], "slots", dev, {T}, at::kLong).data_ptr();
  if (v[6] != Py_None) {
    const at::Tensor& table = tensor(v[6], "cos_sin", 2);
    if (table.size(0) < 1) refuse("cos_sin must have a row");
    check(table, "cos_sin", dev, {table.size(0), table.size(1)}, at::kFloat);
    dense(table, "cos_sin");
    if (v[5] == Py_None) refuse("cos_sin needs positions");
    if (table.size(1) > dim) refuse("cos_sin turns %lld coordinates, the heads have %lld", (long long)table.size(1), (long long)dim);
    a.positions = (const int64_t*)checked(v[5], "positions", dev, {T}, at::kLong).data_ptr();
    a.cos_sin = (const float*)table.data_ptr();
    a.table_len = table.size(0);
    a.rot_dim = (int32_t)table.size(1);
  }
  a.interleaved = truth(v[7]);
  a.hadamard = truth(v[12]);
  at::Tensor q_out;
  if (v[8] != Py_None) {
    const at::Tensor& q = tensor(v[8], "q", 3);
    a.q_heads = q.size(1);
    check(q, "q", dev, {T, a.q_heads, dim}, kt);
    if (v[9] == Py_None) {
      q_out = fresh(q, {T, a.q_heads, dim}, kt);
    } else {
      q_out = checked(v[9], "q_out", dev, {T, a.q_heads, dim}, kt);
      dense(q_out, "q_out");
    }
    a.q = q.data_ptr();
    a.q_out = q_out.data_ptr();
    a.q_token_stride = q.stride(0);
    a.q_head_stride = q.stride(1);
  } else if (v[9] != Py_None) {
    refuse("q_out needs q");
  }
  launch("orbit_kv_append", dev, [&](hipStream_t s) { return orbit_kv_append(&a, s); });
  if (!q_out.defined()) Py_RETURN_NONE;
  return wrap(q_out);
}

// k_cache, v_cache, slots, k_scale, v_scale, dtype
PyObject* kv_read(PyObject* const* v) {
  const at::Tensor& cache = tensor(v[0], "k_cache", 4);
  const int dev = cache.get_device();
  const orbit_kv_cache c = cache_of(v[0], v[1], v[3], v[4], dev);
  const at::Tensor& slots = tensor(v[2], "slots", 1);
  const int64_t T = slots.size(0);
  check(slots, "slots", dev, {T}, at::kLong);
  const at::ScalarType type = type_of(v[5], c.format == ORBIT_KV_INT8 ? at::kHalf : cache.scalar_type());
  const int32_t out_type = dtype(type, "dtype");
  const at::Tensor k = fresh(cache, {T, c.kv_heads, c.head_dim}, type), val = fresh(cache, {T, c.kv_heads, c.head_dim}, type);
  launch("orbit_kv_read", dev, [&](hipStream_t s) {
    return orbit_kv_read(&c, (const int64_t*)slots.data_ptr(), T, k.data_ptr(), val.data_ptr(), (orbit_dtype)out_type, s);
  });
  return pair(k, val);
}

// q, k_cache, v_cache, block_table, lengths, scale, window, k_scale, v_scale,
// out, return_lse
PyObject* paged_attention(PyObject* const* v) {
  const at::Tensor& q = tensor(v[0], "q", 3);
  const int dev = q.get_device();
  const at::ScalarType qt = q.scalar_type();
  orbit_paged_attention_args a = {};
  a.q_dtype = dtype(qt, "q");
  a.cache = cache_of(v[1], v[2], v[7], v[8], dev);
  const int64_t B = q.size(0), H = q.size(1), D = a.cache.head_dim;
  check(q, "q", dev, {B, H, D}, qt);
  const at::Tensor& table = tensor(v[3], "block_table", 2);
  check(table, "block_table", dev, {B, table.size(1)}, at::kInt);
  a.q = q.data_ptr();
  a.q_batch_stride = q.stride(0);
  a.q_head_stride = q.stride(1);
  a.block_table = (const int32_t*)table.data_ptr();
  a.table_stride = table.stride(0);
  a.table_width = table.size(1);
  a.lengths = (const int32_t*)checked(v[4], "lengths", dev, {B}, at::kInt).data_ptr();
  a.batch = B;
  a.q_heads = H;
  a.window = integer(v[6]);
  a.sm_scale = v[5] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)number(v[5]);
  at::Tensor out, lse, work;
  if (v[9] == Py_None) {
    out = fresh(q, {B, H, D}, qt);
  } else {
    out = checked(v[9], "out", dev, {B, H, D}, qt);
    dense(out, "out");
  }
  a.out = out.data_ptr();
  const bool with_lse = truth(v[10]);
  if (with_lse) {
    lse = fresh(q, {B, H}, at::kFloat);
    a.lse = (float*)lse.data_ptr();
  }
  a.workspace_bytes = orbit_paged_attention_workspace(B, H, a.cache.kv_heads, D, a.cache.page_size, a.table_width, a.window, a.cache.format);
  if (a.workspace_bytes < 0)
    refuse("orbit_paged_attention: invalid shape (batch %lld, %lld query heads on %d, dim %lld, window %lld)", (long long)B,
           (long long)H, (int)a.cache.kv_heads, (long long)D, (long long)a.window);
  if (a.workspace_bytes) {
    work = fresh(q, {a.workspace_bytes}, at::kByte);
    a.workspace = work.data_ptr();
  }
  launch("orbit_paged_attention", dev, [&](hipStream_t s) { return orbit_paged_attention(&a, s); });
  return with_lse ? pair(out, lse) : wrap(out);
}

// One entry: the number of arguments is checked, refusals and torch's own
// exceptions (out of memory) become Python's.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(v);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* start(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "two arguments: the error class and the current stream's function");
    return nullptr;
  }
  Py_INCREF(v[0]);
  Py_INCREF(v[1]);
  g_error = v[0];
  g_raw_stream = v[1];
  Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    {"start", (PyCFunction)(void (*)(void))start, METH_FASTCALL, nullptr},
    ENTRY(block_norm, 15),
    ENTRY(adapter_add, 8),
    ENTRY(kv_append, 13),
    ENTRY(kv_read, 6),
    ENTRY(paged_attention, 11),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
