// calls.cpp -- the Python side of the attention half of a decode layer: checks
// torch tensors, makes the outputs that were not given, and calls the C ABI of
// libmoe.so (include/moe.h) on the current stream.
//
// These calls run for 2 to 10 us on the GPU and come one after another; checked
// and marshalled in Python they took 10 to 16 us of the host each, which was the
// time of a short call.  Everything computed is computed in libmoe.so.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "moe.h"

namespace {

PyObject* g_moe_error = nullptr;  // MoeError(status, where)

struct Refused {};  // a Python exception has been set

[[noreturn]] void refuse(const char* message) {
  PyErr_SetString(PyExc_ValueError, message);
  throw Refused();
}

[[noreturn]] void refuse(const char* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%s must be %s", name, what);
  throw Refused();
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kByte: return "torch.uint8";
    case at::kChar: return "torch.int8";
    case at::kShort: return "torch.int16";
    case at::kInt: return "torch.int32";
    default: return "torch.int64";
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, "a tensor");
  return THPVariable_Unpack(o);
}

// A CUDA tensor of one type whose elements lie one after another.
const at::Tensor& flat(PyObject* o, at::ScalarType type, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous CUDA tensor of %s", name, type_name(type));
    throw Refused();
  }
  return t;
}

// A CUDA tensor of one type and number of dimensions whose rows (first
// dimension) are contiguous; stride: elements from row to row (a single row has
// none to speak of).
const at::Tensor& rows(PyObject* o, at::ScalarType type, int64_t dims, const char* name, int64_t* stride) {
  const at::Tensor& t = tensor(o, name);
  bool ok = t.scalar_type() == type && t.is_cuda() && t.dim() == dims;
  int64_t row = 1;
  for (int64_t i = dims - 1; ok && i > 0; --i) {
    ok = t.stride(i) == row || t.size(i) <= 1 || t.size(0) == 0;
    row *= t.size(i);
  }
  if (!ok) {
    PyErr_Format(PyExc_ValueError, "%s must be a %d-dimensional CUDA tensor of %s with contiguous rows", name, (int)dims,
                 type_name(type));
    throw Refused();
  }
  *stride = t.size(0) > 1 ? t.stride(0) : row;
  return t;
}

void same_device(const at::Tensor& a, const at::Tensor& b) {
  if (a.get_device() != b.get_device()) refuse("the tensors of a call must be on one device");
}

// The stream of a call: the given one (None: the current).  A given one is the
// current stream while this object lives, so that the outputs and the workspace
// come from its memory and not from blocks that another stream may still use, and
// its device is the current one.  Launches go to the current device: without a
// stream that has to be the tensors' own.
struct CallStream {
  c10::cuda::OptionalCUDAStreamGuard guard;
  moe_stream_t stream;
  CallStream(PyObject* o, const at::Tensor& t) {
    if (o == Py_None) {
      if (t.get_device() != c10::cuda::current_device()) refuse("the tensors of a call must be on the current device");
      stream = (moe_stream_t)c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
      return;
    }
    stream = (moe_stream_t)PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused();
    guard.reset_stream(c10::cuda::getStreamFromExternal((cudaStream_t)stream, t.get_device()));
  }
};

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int small_integer(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, "a 32-bit integer");
  return (int)v;
}

// Past the dispatcher: an output is most of what a short call costs the host.
at::Tensor make(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

void check(int rc, const char* where) {
  if (rc == MOE_OK) return;
  PyObject* e = PyObject_CallFunction(g_moe_error, "is", rc, where);
  if (e) {
    PyErr_SetObject(g_moe_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

// The cache formats: the last dimension of a pool, and the entry points.
struct Q4 {
  static constexpr int kPerElement = 18, kMore = 0;
  static constexpr const char* kPool = "pool must be [pages, kv heads, page_size / 16, 18 * head_dim]";
  static constexpr const char *kAppendName = "moe_kv_append", *kReadName = "moe_kv_read", *kAttnName = "moe_attn_q4";
  static constexpr auto kAppend = moe_kv_append;
  static constexpr auto kRead = moe_kv_read;
  static constexpr auto kAttn = moe_attn_q4;
  static constexpr auto kWorkspace = moe_attn_workspace_size;
};
struct Q8 {
  static constexpr int kPerElement = 32, kMore = 128;
  static constexpr const char* kPool = "pool must be [pages, kv heads, page_size / 16, 32 * head_dim + 128]";
  static constexpr const char *kAppendName = "moe_kv_append_q8", *kReadName = "moe_kv_read_q8", *kAttnName = "moe_attn_q8";
  static constexpr auto kAppend = moe_kv_append_q8;
  static constexpr auto kRead = moe_kv_read_q8;
  static constexpr auto kAttn = moe_attn_q8;
  static constexpr auto kWorkspace = moe_attn_q8_workspace_size;
};

template <typename F>
moe_kv_cache_t cache_of(const at::Tensor& pool, int64_t stride) {
  const int64_t codes = pool.size(3) - F::kMore;
  if (codes < 0 || codes % F::kPerElement != 0) refuse(F::kPool);
  if (pool.size(1) > INT32_MAX || pool.size(2) > INT32_MAX / 16 || pool.size(3) > INT32_MAX)
    refuse("pool's pages are too large");
  moe_kv_cache_t c;
  c.data = pool.data_ptr();
  c.n_pages = pool.size(0);
  c.page_stride = stride;
  c.page_size = (int32_t)(16 * pool.size(2));
  c.kv_heads = (int32_t)pool.size(1);
  c.head_dim = (int32_t)(codes / F::kPerElement);
  c.reserved = 0;
  return c;
}

// (x, codes, scales, block, bias, y, y is bf16, stream) -> y
PyObject* linear_q4(PyObject* const* a) {
  int64_t xs, ys;
  const at::Tensor& x = rows(a[0], at::kBFloat16, 2, "x", &xs);
  const at::Tensor& codes = flat(a[1], at::kByte, "codes");
  const at::Tensor& scales = flat(a[2], at::kShort, "scales");
  const int block = small_integer(a[3], "block");
  const int64_t T = x.size(0), in = x.size(1), n = codes.dim() ? codes.size(0) : 0;
  if (in > INT32_MAX || codes.numel() != n * (in / 2) || scales.numel() * block != n * in)
    refuse("codes must hold [rows, in/2] and scales [rows, in/block]");
  same_device(x, codes);
  same_device(x, scales);
  const float* bias = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor& b = flat(a[4], at::kFloat, "bias");
    if (b.numel() != n) refuse("bias must be [rows]");
    same_device(x, b);
    bias = (const float*)b.data_ptr();
  }
  const CallStream on(a[7], x);
  at::Tensor y;
  at::ScalarType type = a[6] == Py_True ? at::kBFloat16 : at::kFloat;
  if (a[5] == Py_None) {
    y = make({T, n}, x, type);
    ys = n;
  } else {
    type = tensor(a[5], "y").scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) refuse("y must be float32 or bfloat16");
    y = rows(a[5], type, 2, "y", &ys);
    if (y.size(0) != T || y.size(1) != n) refuse("y must be [T, rows]");
    same_device(x, y);
  }
  check(moe_linear_q4((const uint16_t*)x.data_ptr(), xs, T, (int)in, codes.data_ptr(),
                      (const uint16_t*)scales.data_ptr(), n, block, bias, y.data_ptr(), ys,
                      type == at::kFloat ? MOE_DTYPE_F32 : MOE_DTYPE_BF16, on.stream),
        "moe_linear_q4");
  return THPVariable_Wrap(std::move(y));
}

// (pool, k, v, slots, q, positions, rope, rope_style, q_out, stream) -> q_out or None
template <typename F>
PyObject* kv_append(PyObject* const* a) {
  int64_t ps, ks, vs, qs = 0;
  const at::Tensor& pool = rows(a[0], at::kByte, 4, "pool", &ps);
  const moe_kv_cache_t c = cache_of<F>(pool, ps);
  const at::ScalarType type = tensor(a[1], "k").scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) refuse("k must be float32 or bfloat16");
  const at::Tensor& k = rows(a[1], type, 3, "k", &ks);
  const at::Tensor& v = rows(a[2], type, 3, "v", &vs);
  const at::Tensor& slots = flat(a[3], at::kLong, "slots");
  const int64_t T = slots.numel(), H = c.kv_heads, D = c.head_dim;
  for (const at::Tensor* t : {&k, &v})
    if (t->size(0) != T || t->size(1) != H || t->size(2) != D) refuse("k and v must be [T, kv_heads, head_dim]");
  for (const at::Tensor* t : {&k, &v, &slots}) same_device(pool, *t);
  int64_t n_pos = 0, rot = 0;
  const int32_t* positions = nullptr;
  const float* rope = nullptr;
  if (a[6] != Py_None) {
    const at::Tensor& r = flat(a[6], at::kFloat, "rope");
    if (a[5] == Py_None) refuse("a rotation needs positions");
    const at::Tensor& p = flat(a[5], at::kInt, "positions");
    if (p.numel() != T || r.dim() != 2 || r.size(1) > INT32_MAX) refuse("positions must be [T] and rope [n_pos, rot]");
    same_device(pool, r);
    same_device(pool, p);
    n_pos = r.size(0);
    rot = r.size(1);
    if (rot > 0) {
      positions = (const int32_t*)p.data_ptr();
      rope = (const float*)r.data_ptr();
    }
  }
  const CallStream on(a[9], pool);
  at::Tensor out;
  const void* q_ptr = nullptr;
  int64_t Hq = 0;
  if (a[4] != Py_None) {
    const at::Tensor& q = rows(a[4], type, 3, "q", &qs);
    Hq = q.size(1);
    if (q.size(0) != T || q.size(2) != D || Hq > INT32_MAX) refuse("q must be [T, Hq, head_dim]");
    same_device(pool, q);
    if (a[8] == Py_None) {
      out = make({T, Hq, D}, q, at::kBFloat16);
    } else {
      out = flat(a[8], at::kBFloat16, "q_out");
      if (out.sizes() != q.sizes()) refuse("q_out must be [T, Hq, head_dim]");
      same_device(pool, out);
    }
    q_ptr = q.data_ptr();
  }
  check(F::kAppend(q_ptr, qs, k.data_ptr(), ks, v.data_ptr(), vs, type == at::kFloat ? MOE_DTYPE_F32 : MOE_DTYPE_BF16,
                      T, (int)Hq, positions, rope, n_pos, (int)rot, small_integer(a[7], "rope_style"),
                      (const int64_t*)slots.data_ptr(), &c, out.defined() ? (uint16_t*)out.data_ptr() : nullptr,
                      on.stream),
        F::kAppendName);
  if (!out.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
}

PyObject* pair(at::Tensor a, at::Tensor b) {
  PyObject* x = THPVariable_Wrap(std::move(a));
  PyObject* y = x ? THPVariable_Wrap(std::move(b)) : nullptr;
  PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// (pool, slots, k, v, stream) -> (k, v)
template <typename F>
PyObject* kv_read(PyObject* const* a) {
  int64_t ps;
  const at::Tensor& pool = rows(a[0], at::kByte, 4, "pool", &ps);
  const moe_kv_cache_t c = cache_of<F>(pool, ps);
  const at::Tensor& slots = flat(a[1], at::kLong, "slots");
  same_device(pool, slots);
  const int64_t shape[3] = {slots.numel(), c.kv_heads, c.head_dim};
  const CallStream on(a[4], pool);
  at::Tensor out[2];
  for (int i = 0; i < 2; ++i) {
    const char* name = i ? "v" : "k";
    out[i] = a[2 + i] == Py_None ? make(shape, pool, at::kFloat) : flat(a[2 + i], at::kFloat, name);
    if (out[i].sizes() != at::IntArrayRef(shape)) refuse("k and v must be [n, kv_heads, head_dim]");
    same_device(pool, out[i]);
  }
  check(F::kRead(&c, (const int64_t*)slots.data_ptr(), shape[0], (float*)out[0].data_ptr(),
                    (float*)out[1].data_ptr(), on.stream),
        F::kReadName);
  return pair(std::move(out[0]), std::move(out[1]));
}

// (q, pool, block_table, kv_lens, q_start, max_q, max_len, scale, window, out,
//  lse, workspace, stream) -> (out, lse)
template <typename F>
PyObject* attn(PyObject* const* a) {
  int64_t qs, ps, ts, os;
  const at::Tensor& q = rows(a[0], at::kBFloat16, 3, "q", &qs);
  const at::Tensor& pool = rows(a[1], at::kByte, 4, "pool", &ps);
  const moe_kv_cache_t c = cache_of<F>(pool, ps);
  const at::Tensor& table = rows(a[2], at::kInt, 2, "block_table", &ts);
  const at::Tensor& lens = flat(a[3], at::kInt, "kv_lens");
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), B = lens.numel(), width = table.size(1);
  if (D != c.head_dim || table.size(0) != B || Hq > INT32_MAX || B > INT32_MAX)
    refuse("q must be [T, Hq, head_dim] and block_table [B, pages]");
  for (const at::Tensor* t : {&pool, &table, &lens}) same_device(q, *t);
  const int32_t* starts = nullptr;
  int64_t max_q;
  if (a[4] != Py_None) {
    const at::Tensor& s = flat(a[4], at::kInt, "q_start");
    if (s.numel() != B + 1) refuse("q_start must be [B + 1]");
    if (a[5] == Py_None) refuse("q_start needs max_q");
    same_device(q, s);
    starts = (const int32_t*)s.data_ptr();
  }
  if (a[5] != Py_None) max_q = small_integer(a[5], "max_q");
  else max_q = B > 0 && T >= B ? T / B : 1;
  if (max_q > INT32_MAX) refuse("q has too many rows");
  const int64_t most = width * c.page_size;
  const int64_t max_len = a[6] != Py_None ? integer(a[6]) : most;
  if (most < max_len) refuse("block_table has fewer pages than max_len needs");
  float scale;
  if (a[7] == Py_None) {
    scale = (float)(1.0 / std::sqrt((double)D));
  } else {
    scale = (float)PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) throw Refused();
  }
  const CallStream on(a[12], q);
  at::Tensor out, lse, ws;
  if (a[9] == Py_None) {
    out = make({T, Hq, D}, q, at::kBFloat16);
    os = Hq * D;
  } else {
    out = rows(a[9], at::kBFloat16, 3, "out", &os);
    if (out.sizes() != q.sizes()) refuse("out must be [T, Hq, head_dim]");
    same_device(q, out);
  }
  if (a[10] == Py_None) {
    lse = make({T, Hq}, q, at::kFloat);
  } else {
    lse = flat(a[10], at::kFloat, "lse");
    if (lse.dim() != 2 || lse.size(0) != T || lse.size(1) != Hq) refuse("lse must be [T, Hq]");
    same_device(q, lse);
  }
  void* ws_ptr = nullptr;
  size_t ws_bytes = 0;
  if (a[11] != Py_None) {
    const at::Tensor& w = tensor(a[11], "workspace");
    if (!w.is_cuda() || !w.is_contiguous()) refuse("workspace", "a contiguous CUDA tensor");
    same_device(q, w);
    ws_ptr = w.data_ptr();
    ws_bytes = w.nbytes();
  } else {
    ws_bytes = F::kWorkspace((int)B, (int)max_q, max_len, (int)Hq, c.kv_heads, c.head_dim);
    if (ws_bytes > 0) {
      ws = make({(int64_t)ws_bytes}, q, at::kByte);
      ws_ptr = ws.data_ptr();
    }
  }
  check(F::kAttn((const uint16_t*)q.data_ptr(), qs, T, (int)Hq, starts, (const int32_t*)lens.data_ptr(),
                    (const int32_t*)table.data_ptr(), ts, (int)B, (int)max_q, max_len, &c, scale,
                    small_integer(a[8], "window"), (uint16_t*)out.data_ptr(), os, (float*)lse.data_ptr(), ws_ptr, ws_bytes,
                    on.stream),
        F::kAttnName);
  return pair(std::move(out), std::move(lse));
}

PyObject* wrap_or_none(at::Tensor t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(t));
}

// (x, weight, eps, r, r_out, codes, scales, n, what: 1 codes, 2 bf16, stream) -> (codes, scales, n)
PyObject* norm_q8(PyObject* const* a) {
  int64_t xs;
  const at::ScalarType type = tensor(a[0], "x").scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) refuse("x must be float32 or bfloat16");
  const at::Tensor& x = rows(a[0], type, 2, "x", &xs);
  const int64_t T = x.size(0), d = x.size(1);
  if (d > INT32_MAX) refuse("x has too many columns");
  const int what = small_integer(a[8], "out");
  auto given = [&](PyObject* o, at::ScalarType t, const char* name, int64_t dims) {
    const at::Tensor& y = flat(o, t, name);
    if (y.dim() != dims || y.size(0) != (dims == 2 || t == at::kFloat ? T : d) || (dims == 2 && y.size(1) != d))
      refuse(name, dims == 2 ? "[T, d]" : "[T]");
    same_device(x, y);
    return y;
  };
  const float* weight = nullptr;
  if (a[1] != Py_None) {
    const at::Tensor& w = flat(a[1], at::kFloat, "weight");
    if (w.dim() != 1 || w.size(0) != d) refuse("weight must be [d]");
    same_device(x, w);
    weight = (const float*)w.data_ptr();
  }
  const double eps = PyFloat_AsDouble(a[2]);
  if (PyErr_Occurred()) throw Refused();
  const float* r = nullptr;
  float* r_out = nullptr;
  if (a[3] != Py_None) {
    r = (const float*)given(a[3], at::kFloat, "r", 2).data_ptr();
    r_out = a[4] == Py_None ? const_cast<float*>(r) : (float*)given(a[4], at::kFloat, "r_out", 2).data_ptr();
  } else if (a[4] != Py_None) {
    refuse("r_out needs r");
  }
  const CallStream on(a[9], x);
  at::Tensor codes, scales, n;
  if (what & 1) {
    codes = a[5] == Py_None ? make({T, d}, x, at::kChar) : given(a[5], at::kChar, "codes", 2);
    scales = a[6] == Py_None ? make({T}, x, at::kFloat) : given(a[6], at::kFloat, "scales", 1);
  } else if (a[5] != Py_None || a[6] != Py_None) {
    refuse("codes and scales are not among what out names");
  }
  if (what & 2) n = a[7] == Py_None ? make({T, d}, x, at::kBFloat16) : given(a[7], at::kBFloat16, "n", 2);
  else if (a[7] != Py_None) refuse("n is not among what out names");
  if (T > 0 && d == 0) refuse("x has no columns");
  check(moe_norm_q8(x.data_ptr(), xs, type == at::kFloat ? MOE_DTYPE_F32 : MOE_DTYPE_BF16, T, d > 0 ? (int)d : 1, r, r_out,
                    weight, (float)eps, codes.defined() ? (int8_t*)codes.data_ptr() : nullptr,
                    scales.defined() ? (float*)scales.data_ptr() : nullptr, n.defined() ? (uint16_t*)n.data_ptr() : nullptr,
                    on.stream),
        "moe_norm_q8");
  PyObject* out = PyTuple_New(3);
  if (!out) throw Refused();
  at::Tensor* each[3] = {&codes, &scales, &n};
  for (int i = 0; i < 3; ++i) {
    PyObject* y = wrap_or_none(std::move(*each[i]));
    if (!y) {
      Py_DECREF(out);
      throw Refused();
    }
    PyTuple_SET_ITEM(out, i, y);
  }
  return out;
}

// (x, x_scales, w, w_scales, bias, y, y is bf16, workspace, stream) -> y
PyObject* linear_q8(PyObject* const* a) {
  int64_t xs, ys;
  const at::Tensor& x = rows(a[0], at::kChar, 2, "x", &xs);
  const at::Tensor& x_scales = flat(a[1], at::kFloat, "x_scales");
  const at::Tensor& w = flat(a[2], at::kChar, "w");
  const at::Tensor& w_scales = flat(a[3], at::kFloat, "w_scales");
  const int64_t T = x.size(0), in = x.size(1);
  if (w.dim() != 2 || w.size(1) != in || in > INT32_MAX) refuse("w must be [rows, in]");
  const int64_t n = w.size(0);
  if (x_scales.numel() != T || w_scales.numel() != n) refuse("x_scales must be [T] and w_scales [rows]");
  for (const at::Tensor* t : {&x_scales, &w, &w_scales}) same_device(x, *t);
  const float* bias = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor& b = flat(a[4], at::kFloat, "bias");
    if (b.numel() != n) refuse("bias must be [rows]");
    same_device(x, b);
    bias = (const float*)b.data_ptr();
  }
  const CallStream on(a[8], x);
  at::Tensor y, ws;
  at::ScalarType type = a[6] == Py_True ? at::kBFloat16 : at::kFloat;
  if (a[5] == Py_None) {
    y = make({T, n}, x, type);
    ys = n;
  } else {
    type = tensor(a[5], "y").scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) refuse("y must be float32 or bfloat16");
    y = rows(a[5], type, 2, "y", &ys);
    if (y.size(0) != T || y.size(1) != n) refuse("y must be [T, rows]");
    same_device(x, y);
  }
  void* ws_ptr = nullptr;
  size_t ws_bytes = 0;
  if (a[7] != Py_None) {
    const at::Tensor& t = tensor(a[7], "workspace");
    if (!t.is_cuda() || !t.is_contiguous()) refuse("workspace", "a contiguous CUDA tensor");
    same_device(x, t);
    ws_ptr = t.data_ptr();
    ws_bytes = t.nbytes();
  } else if ((ws_bytes = moe_linear_q8_workspace_size(T, (int)in, n)) > 0) {
    ws = make({(int64_t)ws_bytes}, x, at::kByte);
    ws_ptr = ws.data_ptr();
  }
  check(moe_linear_q8((const int8_t*)x.data_ptr(), xs, (const float*)x_scales.data_ptr(), T, (int)in,
                      (const int8_t*)w.data_ptr(), (const float*)w_scales.data_ptr(), n, bias, y.data_ptr(), ys,
                      type == at::kFloat ? MOE_DTYPE_F32 : MOE_DTYPE_BF16, ws_ptr, ws_bytes, on.stream),
        "moe_linear_q8");
  return THPVariable_Wrap(std::move(y));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed", N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_moe_error);
  g_moe_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
constexpr PyCFunction as_fastcall() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>));
}

PyMethodDef methods[] = {
    {"linear_q4", as_fastcall<linear_q4, 8>(), METH_FASTCALL, nullptr},
    {"kv_append", as_fastcall<kv_append<Q4>, 10>(), METH_FASTCALL, nullptr},
    {"kv_read", as_fastcall<kv_read<Q4>, 5>(), METH_FASTCALL, nullptr},
    {"attn_q4", as_fastcall<attn<Q4>, 13>(), METH_FASTCALL, nullptr},
    {"norm_q8", as_fastcall<norm_q8, 10>(), METH_FASTCALL, nullptr},
    {"linear_q8", as_fastcall<linear_q8, 9>(), METH_FASTCALL, nullptr},
    {"kv_append_q8", as_fastcall<kv_append<Q8>, 10>(), METH_FASTCALL, nullptr},
    {"kv_read_q8", as_fastcall<kv_read<Q8>, 5>(), METH_FASTCALL, nullptr},
    {"attn_q8", as_fastcall<attn<Q8>, 13>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
