// Python entry of the calls that a serving loop makes once per layer and step
// on a few tokens, where the host's time is what counts: arguments checked,
// outputs allocated and the C ABI called from one compiled function (the same
// checks made attribute by attribute in Python took 10 of a call's 15 us).
// Tensors are checked here for what the ABI cannot see (type, device, shape,
// layout); everything else is the ABI's to check.  A call returns its tensor,
// or the ABI's status as an int where that is not PKV_OK.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/CUDAContext.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <utility>

#include "pkv.h"
#include "pkv_blocks.h"

namespace {

using at::Tensor;

// Entry points of the loaded library, handed over by bind().
decltype(&pkv_chunk_plan) g_chunk_plan = nullptr;
decltype(&pkv_chunk_attention) g_chunk_attention = nullptr;
decltype(&pkv_rotary_append_axes) g_rotary_append = nullptr;
decltype(&pkv_compact_tokens) g_compact_tokens = nullptr;
decltype(&pkv_append) g_append = nullptr;
decltype(&pkv_read_tokens) g_read_tokens = nullptr;
decltype(&pkv_extend_tables) g_extend_tables = nullptr;
decltype(&pkv_truncate_tables) g_truncate_tables = nullptr;

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  PyErr_SetString(type, buf);
  throw Raised{};
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) { return c10::toString(t); }

// A contiguous tensor of a type on the caches' device.
const Tensor& dense(PyObject* o, at::ScalarType type, const char* name, at::Device dev) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
  if (t.device() != dev) raise(PyExc_ValueError, "%s must be on %s", name, dev.str().c_str());
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}

int64_t integer(PyObject* o, const char* name) {
  PyObject* i = PyNumber_Index(o);  // whole numbers of any kind, no floats
  if (i == nullptr) throw Raised{};
  const int64_t v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  (void)name;
  return v;
}

int32_t int32(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, "%s %lld is out of range", name, static_cast<long long>(v));
  return static_cast<int32_t>(v);
}

int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) raise(PyExc_ValueError, "%s is too large (%lld)", name, static_cast<long long>(v));
  return static_cast<int32_t>(v);
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

struct Caches {
  const Tensor& k;
  const Tensor& v;
  pkv_cache_desc desc;
  at::Device dev;
};

Caches caches(PyObject* ko, PyObject* vo) {
  const Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  if (k.dim() != 4) raise(PyExc_ValueError, "cache must be [num_blocks, num_kv_heads, block_size, head_dim]");
  if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
    raise(PyExc_ValueError, "k_cache and v_cache must have the same shape and dtype");
  if (!k.is_contiguous() || !v.is_contiguous()) raise(PyExc_ValueError, "caches must be contiguous");
  if (k.device() != v.device() || !k.is_cuda()) raise(PyExc_ValueError, "caches must be CUDA tensors on one device");
  int32_t dtype;
  int64_t d_row = k.size(3);
  if (k.scalar_type() == at::kBFloat16) {
    dtype = PKV_BF16;
  } else if (k.scalar_type() == at::kByte && (d_row == 36 || d_row == 72)) {
    dtype = PKV_E2M1;  // rows of head_dim / 2 + head_dim / 16 bytes
    d_row = d_row / 9 * 16;
  } else if (k.scalar_type() == at::kByte || k.scalar_type() == at::kFloat8_e4m3fn) {
    dtype = PKV_E4M3;
  } else {
    raise(PyExc_TypeError, "cache dtype %s: expected bfloat16 or uint8/float8_e4m3fn", type_name(k.scalar_type()));
  }
  pkv_cache_desc d = {k.size(0), size32(k.size(2), "block_size"), size32(k.size(1), "num_kv_heads"),
                      size32(d_row, "head_dim"), dtype};
  return Caches{k, v, d, k.device()};
}

// Scales of an E4M3 or E2M1 cache, [rows, H_kv] or [H_kv] each (an E2M1 cache
// may have none); their row stride.
struct Scales {
  const float* k = nullptr;
  const float* v = nullptr;
  int64_t stride = 0;
};

Scales scales(PyObject* ko, PyObject* vo, PyObject* so, const Caches& c, int64_t rows) {
  Scales s;
  if (c.desc.dtype == PKV_E2M1 && ko == Py_None && vo == Py_None) return s;
  if (c.desc.dtype == PKV_BF16) {
    if (ko != Py_None || vo != Py_None) raise(PyExc_ValueError, "scales given for a bf16 cache");
    return s;
  }
  if (ko == Py_None || vo == Py_None) raise(PyExc_ValueError, "k_scale and v_scale are both needed");
  const Tensor &k = dense(ko, at::kFloat, "k_scale", c.dev), &v = dense(vo, at::kFloat, "v_scale", c.dev);
  if (k.sizes() != v.sizes()) raise(PyExc_ValueError, "k_scale and v_scale differ in shape");
  const int64_t heads = c.desc.num_kv_heads;
  s.k = k.const_data_ptr<float>();
  s.v = v.const_data_ptr<float>();
  if (so == Py_None) {
    const bool per_row = k.dim() == 2 && k.size(0) == rows && k.size(1) == heads;
    if (!per_row && !(k.dim() == 1 && k.size(0) == heads))
      raise(PyExc_ValueError, "k_scale and v_scale must be [%lld, %lld] or [%lld]", static_cast<long long>(rows),
            static_cast<long long>(heads), static_cast<long long>(heads));
    s.stride = per_row ? heads : 0;
  } else {
    s.stride = integer(so, "scale_row_stride");
    if (s.stride < 0 || (rows > 0 && (s.stride > k.numel() || k.numel() < s.stride * (rows - 1) + heads)))
      raise(PyExc_ValueError, "scale_row_stride reaches past the scales");
  }
  return s;
}

// The interpreter's lock, given up while this lives and taken back on every way out.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs the ABI call on the device's current stream without the interpreter's
// lock: `call` neither touches Python objects nor refuses arguments.
template <class F>
pkv_status on_stream(at::Device dev, F&& call) {
  const c10::cuda::CUDAGuard guard(dev);
  pkv_stream_t stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  const Unlocked unlocked;
  return call(stream);
}

// A Python tuple of the tensors.
PyObject* tuple(std::initializer_list<Tensor> tensors) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (t == nullptr) throw Raised{};
  Py_ssize_t i = 0;
  for (const Tensor& x : tensors) {
    PyObject* o = THPVariable_Wrap(x);
    if (o == nullptr) {
      Py_DECREF(t);
      throw Raised{};
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
}

PyObject* chunk_attention(PyObject* const* a, Py_ssize_t n) {
  expect(n, 19);
  const Caches c = caches(a[1], a[2]);
  const Tensor& q = dense(a[0], at::kBFloat16, "q", c.dev);
  if (q.dim() != 3 || q.size(2) != c.desc.head_dim) raise(PyExc_ValueError, "q must be [T, H_q, head_dim]");
  const Tensor& tables = dense(a[3], at::kInt, "block_tables", c.dev);
  const Tensor& ctx = dense(a[4], at::kInt, "context_lens", c.dev);
  const Tensor& starts = dense(a[5], at::kInt, "q_starts", c.dev);
  if (starts.dim() != 1 || starts.size(0) < 1) raise(PyExc_ValueError, "q_starts must be [B + 1]");
  const int64_t b = starts.size(0) - 1;
  if (tables.dim() != 2 || tables.size(0) != b || ctx.dim() != 1 || ctx.size(0) != b)
    raise(PyExc_ValueError, "block_tables must be [B, MB] and context_lens [B]");
  const int32_t t = size32(q.size(0), "T"), hq = size32(q.size(1), "H_q"), batch = size32(b, "B");
  const int32_t mb = size32(tables.size(1), "MB");
  const float scale = real(a[6]);
  const int32_t max_q = a[7] == Py_None ? (t > 1 ? t : 1) : int32(a[7], "max_q_len");
  const int32_t max_ctx = a[8] == Py_None ? size32(static_cast<int64_t>(mb) * c.desc.block_size, "the tables' capacity")
                                          : int32(a[8], "max_context_len");
  const Scales sc = scales(a[9], a[10], a[18], c, b);
  pkv_score_mods mods = {real(a[11]), int32(a[12], "window"), nullptr, nullptr};
  if (a[13] != Py_None) {
    const Tensor& s = dense(a[13], at::kFloat, "slopes", c.dev);
    if (s.dim() != 1 || s.size(0) != hq) raise(PyExc_ValueError, "slopes must be [H_q]");
    mods.slopes = s.const_data_ptr<float>();
  }
  if (a[14] != Py_None) {
    const Tensor& p = dense(a[14], at::kInt, "prefix_lens", c.dev);
    if (p.dim() != 1 || p.size(0) != b) raise(PyExc_ValueError, "prefix_lens must be [B]");
    mods.prefix_lens = p.const_data_ptr<int32_t>();
  }
  const int32_t split = int32(a[17], "split_tokens");
  if (a[15] != Py_None && dense(a[15], at::kBFloat16, "out", c.dev).sizes() != q.sizes())
    raise(PyExc_ValueError, "out must be [T, H_q, D]");
  // planned for this device's SMs, as the library plans the call itself
  pkv_decode_plan_t plan;
  const int sms = at::cuda::getDeviceProperties(c.dev.index())->multiProcessorCount;
  pkv_status st = g_chunk_plan(t, batch, max_q, hq, &c.desc, max_ctx, mods.window, mods.prefix_lens != nullptr, split,
                               sms, &plan);
  if (st != PKV_OK) return PyLong_FromLong(st);
  Tensor scratch;  // freed in stream order when the call returns
  void* ws = nullptr;
  size_t ws_bytes = 0;
  if (plan.workspace_bytes > 0) {
    if (a[16] == Py_None)
      scratch = at::empty({plan.workspace_bytes}, c.k.options().dtype(at::kByte));
    else
      scratch = dense(a[16], at::kByte, "workspace", c.dev);
    ws = scratch.data_ptr();
    ws_bytes = static_cast<size_t>(scratch.numel());
  }
  Tensor out = a[15] == Py_None ? at::empty(q.sizes(), q.options()) : THPVariable_Unpack(a[15]);
  st = on_stream(c.dev, [&](pkv_stream_t stream) {
    return g_chunk_attention(q.data_ptr(), t, starts.const_data_ptr<int32_t>(), batch, max_q, hq, c.k.data_ptr(),
                             c.v.data_ptr(), &c.desc, tables.const_data_ptr<int32_t>(), mb,
                             ctx.const_data_ptr<int32_t>(), max_ctx, scale, &mods, out.data_ptr(), sc.k, sc.v,
                             sc.stride, ws, ws_bytes, split, stream);
  });
  if (st != PKV_OK) return PyLong_FromLong(st);
  if (a[15] != Py_None) {
    Py_INCREF(a[15]);
    return a[15];
  }
  return THPVariable_Wrap(std::move(out));
}

// [N, heads, D] whose tokens may lie further apart than their rows (a slice of
// a fused projection): the elements between tokens.
int64_t token_rows(const Tensor& t, const char* name, at::ScalarType type, at::Device dev, int64_t n, int64_t heads,
                   int64_t d) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
  if (t.device() != dev) raise(PyExc_ValueError, "%s must be on %s", name, dev.str().c_str());
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != d)
    raise(PyExc_ValueError, "%s must be [%lld, %lld, %lld]", name, static_cast<long long>(n),
          static_cast<long long>(heads), static_cast<long long>(d));
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
    raise(PyExc_ValueError, "%s: the heads of a token must be contiguous", name);
  return n > 1 ? t.stride(0) : heads * d;
}

PyObject* rotary_append(PyObject* const* a, Py_ssize_t n_args) {
  expect(n_args, 15);
  const Caches c = caches(a[6], a[7]);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  if (q.dim() != 3) raise(PyExc_ValueError, "q must be [N, H_q, D]");
  const int64_t n = q.size(0), hq = q.size(1), d = c.desc.head_dim, hkv = c.desc.num_kv_heads;
  if (q.size(2) != d) raise(PyExc_ValueError, "q's head_dim does not match the cache");
  const at::ScalarType type = q.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat)
    raise(PyExc_TypeError, "q dtype %s: expected bfloat16 or float32", type_name(type));
  const int64_t q_st = token_rows(q, "q", type, c.dev, n, hq, d), k_st = token_rows(k, "k", type, c.dev, n, hkv, d),
                v_st = token_rows(v, "v", type, c.dev, n, hkv, d);
  const Tensor& pos = tensor(a[3], "positions");
  const Tensor& freq = dense(a[4], at::kDouble, "inv_freq", c.dev);
  const Tensor& slots = dense(a[5], at::kLong, "slot_mapping", c.dev);
  if (pos.scalar_type() != at::kLong)
    raise(PyExc_TypeError, "positions must be %s, got %s", type_name(at::kLong), type_name(pos.scalar_type()));
  if (pos.device() != c.dev) raise(PyExc_ValueError, "positions must be on %s", c.dev.str().c_str());
  const bool many = a[14] != Py_None;  // [axes, N], an axis' positions contiguous
  const int64_t along = many ? 1 : 0;
  if (pos.dim() != 1 + along || pos.size(along) != n || slots.dim() != 1 || slots.size(0) != n)
    raise(PyExc_ValueError, many ? "positions must be [num_axes, N] and slot_mapping [N]"
                                 : "positions and slot_mapping must have one entry per token");
  if (n > 1 && pos.stride(along) != 1) raise(PyExc_ValueError, "positions must be contiguous");
  const int32_t* axes = nullptr;
  int32_t num_axes = 1;
  if (many) {
    const Tensor& t = dense(a[14], at::kInt, "axes", c.dev);
    if (t.dim() != 1 || t.size(0) != freq.numel()) raise(PyExc_ValueError, "axes must be [rotary_dim / 2]");
    axes = t.const_data_ptr<int32_t>();
    num_axes = size32(pos.size(0), "num_axes");
  }
  if (freq.dim() != 1) raise(PyExc_ValueError, "inv_freq must be [rotary_dim / 2]");
  const int32_t heads = size32(hq, "H_q"), rotary_dim = size32(2 * freq.size(0), "rotary_dim");
  const Scales sc = scales(a[8], a[9], a[13], c, n);
  const float magnitude = real(a[10]);
  const int interleaved = PyObject_IsTrue(a[11]);
  if (interleaved < 0) throw Raised{};
  Tensor out;
  int64_t o_st = hq * d;
  if (a[12] == Py_None) {
    out = at::empty({n, hq, d}, c.k.options().dtype(at::kBFloat16));
  } else {
    out = tensor(a[12], "out");
    o_st = token_rows(out, "out", at::kBFloat16, c.dev, n, hq, d);
  }
  const pkv_status st = on_stream(c.dev, [&](pkv_stream_t stream) {
    return g_rotary_append(q.data_ptr(), q_st, k.data_ptr(), k_st, v.data_ptr(), v_st,
                           type == at::kBFloat16 ? PKV_BF16 : PKV_F32, n, heads, pos.const_data_ptr<int64_t>(),
                           many ? pos.stride(0) : 0, num_axes, axes, freq.const_data_ptr<double>(), rotary_dim, interleaved, magnitude,
                           slots.const_data_ptr<int64_t>(), c.k.data_ptr(), c.v.data_ptr(), &c.desc, sc.k, sc.v,
                           sc.stride, out.data_ptr(), o_st, stream);
  });
  if (st != PKV_OK) return PyLong_FromLong(st);
  if (a[12] != Py_None) {
    Py_INCREF(a[12]);
    return a[12];
  }
  return THPVariable_Wrap(std::move(out));
}

PyObject* compact_tokens(PyObject* const* a, Py_ssize_t n_args) {
  expect(n_args, 7);
  const Caches c = caches(a[0], a[1]);
  const Tensor& tables = dense(a[2], at::kInt, "block_tables", c.dev);
  const Tensor& keep = dense(a[3], at::kInt, "keep", c.dev);
  const Tensor& starts = dense(a[4], at::kInt, "keep_starts", c.dev);
  if (tables.dim() != 2 || keep.dim() != 1) raise(PyExc_ValueError, "block_tables must be [B, MB] and keep 1-D");
  const int64_t b = tables.size(0);
  if (starts.dim() != 1 || starts.size(0) != b + 1) raise(PyExc_ValueError, "keep_starts must be [B + 1]");
  const int32_t* first = nullptr;
  if (a[5] != Py_None) {
    const Tensor& t = dense(a[5], at::kInt, "dst_start", c.dev);
    if (t.dim() != 1 || t.size(0) != b) raise(PyExc_ValueError, "dst_start must be [B]");
    first = t.const_data_ptr<int32_t>();
  }
  const int32_t n = size32(keep.size(0), "keep"), batch = size32(b, "B"), mb = size32(tables.size(1), "MB");
  const int32_t most = a[6] == Py_None ? n : int32(a[6], "max_keep");
  const pkv_status st = on_stream(c.dev, [&](pkv_stream_t stream) {
    return g_compact_tokens(c.k.data_ptr(), c.v.data_ptr(), &c.desc, tables.const_data_ptr<int32_t>(),
                            mb > 1 ? mb : 1, batch, keep.const_data_ptr<int32_t>(), n,
                            starts.const_data_ptr<int32_t>(), first, most, stream);
  });
  return PyLong_FromLong(st);
}

// Appends to an E2M1 cache (the other types' appends are checked in Python).
PyObject* append(PyObject* const* a, Py_ssize_t n_args) {
  expect(n_args, 8);
  const Caches c = caches(a[3], a[4]);
  const Tensor &k = tensor(a[0], "k_new"), &v = tensor(a[1], "v_new");
  if (k.dim() != 3 || k.sizes() != v.sizes()) raise(PyExc_ValueError, "k_new / v_new must both be [N, H_kv, D]");
  const int64_t n = k.size(0);
  if (k.size(1) != c.desc.num_kv_heads || k.size(2) != c.desc.head_dim)
    raise(PyExc_ValueError, "k_new heads / head_dim do not match the cache");
  const at::ScalarType type = k.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat)
    raise(PyExc_TypeError, "k_new dtype %s: expected bfloat16 or float32", type_name(type));
  dense(a[0], type, "k_new", c.dev);
  dense(a[1], type, "v_new", c.dev);
  const Tensor& slots = dense(a[2], at::kLong, "slot_mapping", c.dev);
  if (slots.numel() != n) raise(PyExc_ValueError, "slot_mapping must have one entry per row");
  const Scales sc = scales(a[5], a[6], a[7], c, n);
  const pkv_status st = on_stream(c.dev, [&](pkv_stream_t stream) {
    return g_append(k.data_ptr(), v.data_ptr(), type == at::kBFloat16 ? PKV_BF16 : PKV_F32, n,
                    slots.const_data_ptr<int64_t>(), c.k.data_ptr(), c.v.data_ptr(), &c.desc, sc.k, sc.v, sc.stride,
                    stream);
  });
  return PyLong_FromLong(st);
}

PyObject* read_tokens(PyObject* const* a, Py_ssize_t n_args) {
  expect(n_args, 7);
  const Caches c = caches(a[1], a[2]);
  const Tensor& slots = dense(a[0], at::kLong, "slot_mapping", c.dev);
  if (slots.dim() != 1) raise(PyExc_ValueError, "slot_mapping must be [N]");
  const int64_t n = slots.size(0);
  const Scales sc = scales(a[3], a[4], a[5], c, n);
  const int f32 = PyObject_IsTrue(a[6]);
  if (f32 < 0) throw Raised{};
  const auto options = c.k.options().dtype(f32 ? at::kFloat : at::kBFloat16);
  const int64_t shape[3] = {n, c.desc.num_kv_heads, c.desc.head_dim};
  Tensor k = at::empty(shape, options), v = at::empty(shape, options);
  const pkv_status st = on_stream(c.dev, [&](pkv_stream_t stream) {
    return g_read_tokens(slots.const_data_ptr<int64_t>(), n, c.k.data_ptr(), c.v.data_ptr(), &c.desc, sc.k, sc.v,
                         sc.stride, k.data_ptr(), v.data_ptr(), f32 ? PKV_F32 : PKV_BF16, stream);
  });
  if (st != PKV_OK) return PyLong_FromLong(st);
  return tuple({std::move(k), std::move(v)});
}

// `n` elements of `type` from byte `at` of a tensor's storage on, as a tensor of
// their own.
Tensor part(const Tensor& base, at::ScalarType type, int64_t at, int64_t n) {
  const auto meta = c10::scalarTypeToTypeMeta(type);
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), meta);
  t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(meta.itemsize()));
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// The geometry that tables are made for: one cache tensor.
Caches one_cache(PyObject* ko) { return caches(ko, ko); }

const Tensor& ints(PyObject* o, const char* name, at::Device dev, int64_t n) {
  const Tensor& t = dense(o, at::kInt, name, dev);
  if (t.dim() != 1 || t.size(0) != n) raise(PyExc_ValueError, "%s must be [%lld]", name, static_cast<long long>(n));
  return t;
}

// The stack of free blocks and its count.
struct Stack {
  const Tensor& blocks;
  const Tensor& count;
  int32_t capacity;
};
Stack stack(PyObject* blocks, PyObject* count, at::Device dev) {
  const Tensor& t = dense(blocks, at::kInt, "free_blocks", dev);
  if (t.dim() != 1) raise(PyExc_ValueError, "free_blocks must be 1-D");
  return Stack{t, ints(count, "free_count", dev, 1), size32(t.size(0), "free_blocks")};
}

PyObject* extend_tables(PyObject* const* a, Py_ssize_t n_args) {
  expect(n_args, 8);
  const Caches c = one_cache(a[5]);
  const Tensor& tables = dense(a[0], at::kInt, "block_tables", c.dev);
  if (tables.dim() != 2) raise(PyExc_ValueError, "block_tables must be [B, MB]");
  const int64_t b = tables.size(0);
  const int32_t batch = size32(b, "B"), mb = size32(tables.size(1), "MB");
  const Tensor &past = ints(a[1], "past_lens", c.dev, b), &news = ints(a[2], "new_lens", c.dev, b);
  const Stack st = stack(a[3], a[4], c.dev);
  const int64_t most = integer(a[6], "max_tokens");
  if (most < 0 || most > 0x7FFFFFFF) raise(PyExc_ValueError, "max_tokens %lld", static_cast<long long>(most));
  Tensor r[7];  // context_lens, q_starts, slot_mapping, positions, block_starts, free_count, lacking
  const int64_t sizes[7] = {b, b + 1, most, most, b + 1, 1, 1};
  static const char* const names[7] = {"out.context_lens", "out.q_starts",   "out.slot_mapping", "out.positions",
                                       "out.block_starts", "out.free_count", "out.lacking"};
  if (a[7] == Py_None) {
    // one allocation: the 64-bit arrays first
    const Tensor all = at::empty({16 * most + 4 * (3 * b + 4)}, tables.options().dtype(at::kByte));
    int64_t at64 = 0, at32 = 16 * most;
    for (int i = 0; i < 7; ++i) {
      const bool wide = i == 2 || i == 3;
      r[i] = part(all, wide ? at::kLong : at::kInt, wide ? at64 : at32, sizes[i]);
      (wide ? at64 : at32) += (wide ? 8 : 4) * sizes[i];
    }
  } else {
    if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 7) raise(PyExc_TypeError, "out must be seven tensors");
    for (int i = 0; i < 7; ++i) {
      const Tensor& t = dense(PyTuple_GET_ITEM(a[7], i), i == 2 || i == 3 ? at::kLong : at::kInt, names[i], c.dev);
      if (t.dim() != 1 || t.size(0) != sizes[i])
        raise(PyExc_ValueError, "%s must be [%lld]", names[i], static_cast<long long>(sizes[i]));
      r[i] = t;
    }
  }
  const pkv_table_step out = {r[0].data_ptr<int32_t>(), r[1].data_ptr<int32_t>(), r[4].data_ptr<int32_t>(),
                              r[2].data_ptr<int64_t>(), r[3].data_ptr<int64_t>(), r[5].data_ptr<int32_t>(),
                              r[6].data_ptr<int32_t>()};
  const pkv_status s = on_stream(c.dev, [&](pkv_stream_t stream) {
    return g_extend_tables(tables.data_ptr<int32_t>(), mb, batch, past.const_data_ptr<int32_t>(),
                           news.const_data_ptr<int32_t>(), st.blocks.const_data_ptr<int32_t>(), st.capacity,
                           st.count.const_data_ptr<int32_t>(), &c.desc, most, &out, stream);
  });
  if (s != PKV_OK) return PyLong_FromLong(s);
  if (a[7] != Py_None) {
    Py_INCREF(a[7]);
    return a[7];
  }
  return tuple({r[0], r[1], r[2], r[3], r[4], r[5], r[6]});
}

PyObject* truncate_tables(PyObject* const* a, Py_ssize_t n_args) {
  expect(n_args, 7);
  const Caches c = one_cache(a[5]);
  const Tensor& tables = dense(a[0], at::kInt, "block_tables", c.dev);
  if (tables.dim() != 2) raise(PyExc_ValueError, "block_tables must be [B, MB]");
  const int64_t b = tables.size(0);
  const int32_t batch = size32(b, "B"), mb = size32(tables.size(1), "MB");
  const Tensor &ctx = ints(a[1], "context_lens", c.dev, b), &keep = ints(a[2], "keep_lens", c.dev, b);
  const Stack st = stack(a[3], a[4], c.dev);
  const Tensor mine = at::empty({b + 2}, tables.options());
  const Tensor count = a[6] == Py_None ? part(mine, at::kInt, 4 * (b + 1), 1) : ints(a[6], "out", c.dev, 1);
  const pkv_status s = on_stream(c.dev, [&](pkv_stream_t stream) {
    return g_truncate_tables(tables.const_data_ptr<int32_t>(), mb, batch, ctx.const_data_ptr<int32_t>(),
                             keep.const_data_ptr<int32_t>(), st.blocks.data_ptr<int32_t>(), st.capacity,
                             st.count.const_data_ptr<int32_t>(), &c.desc, mine.data_ptr<int32_t>(),
                             count.data_ptr<int32_t>(), stream);
  });
  if (s != PKV_OK) return PyLong_FromLong(s);
  if (a[6] != Py_None) {
    Py_INCREF(a[6]);
    return a[6];
  }
  return THPVariable_Wrap(count);
}

PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  constexpr int kCalls = 8;
  expect(n, kCalls);
  void* p[kCalls];
  for (int i = 0; i < kCalls; ++i) p[i] = reinterpret_cast<void*>(static_cast<uintptr_t>(integer(a[i], "address")));
  g_chunk_plan = reinterpret_cast<decltype(g_chunk_plan)>(p[0]);
  g_chunk_attention = reinterpret_cast<decltype(g_chunk_attention)>(p[1]);
  g_rotary_append = reinterpret_cast<decltype(g_rotary_append)>(p[2]);
  g_compact_tokens = reinterpret_cast<decltype(g_compact_tokens)>(p[3]);
  g_append = reinterpret_cast<decltype(g_append)>(p[4]);
  g_read_tokens = reinterpret_cast<decltype(g_read_tokens)>(p[5]);
  g_extend_tables = reinterpret_cast<decltype(g_extend_tables)>(p[6]);
  g_truncate_tables = reinterpret_cast<decltype(g_truncate_tables)>(p[7]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define PKV_ENTRY(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name>)), METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {PKV_ENTRY(bind), PKV_ENTRY(chunk_attention), PKV_ENTRY(rotary_append),
                           PKV_ENTRY(compact_tokens), PKV_ENTRY(append), PKV_ENTRY(read_tokens),
                           PKV_ENTRY(extend_tables), PKV_ENTRY(truncate_tables), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", "Compiled calls of the paged-KV library.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
