// CPython module `_binding`: argument marshalling of the calls that run once
// per layer of a decoding step (norm + rotation, the paged caches' calls),
// where the host's time counts.  It does for them what the ctypes binding in
// cpattn.py does for the others -- checks each tensor's type, device, shape and
// layout, allocates what was not given, and hands the addresses and PyTorch's
// current stream to libcpattn.so -- without interpreting Python for each
// argument: a norm of 32 tokens takes the host 5.8 us this way and took it
// 18-20 us through ctypes, an attention call of one token 11 and 27 us.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>
#include <string>
#include <vector>

#include "cpattn.h"

namespace {

PyObject* g_error = nullptr;  // cpattn.CpattnError

// A Python exception that is set already.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised();
}

std::string shape_text(c10::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

std::string type_text(c10::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name, c10::ScalarType dtype) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != dtype)
    raise(PyExc_TypeError, std::string(name) + " must be " + type_text(dtype) + ", got " +
                               type_text(t.scalar_type()));
  return t;
}

void on_device(const at::Tensor& t, const char* name, c10::Device dev) {
  if (t.device() != dev)
    raise(PyExc_ValueError,
          std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
}

void of_shape(const at::Tensor& t, const char* name, c10::IntArrayRef shape) {
  if (!t.sizes().equals(shape))
    raise(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) +
                                ", got " + shape_text(t.sizes()));
}

// A contiguous tensor of that type, device and shape; its address.
void* flat(PyObject* o, const char* name, c10::ScalarType dtype, c10::Device dev,
           c10::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name, dtype);
  on_device(t, name, dev);
  of_shape(t, name, shape);
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

// The first tensor of a call, bf16 [T, heads, D] on a CUDA device.
const at::Tensor& leading(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name, at::kBFloat16);
  if (t.dim() != 3) raise(PyExc_ValueError, std::string(name) + " must be [T, heads, D]");
  if (!t.is_cuda())
    raise(PyExc_ValueError,
          std::string(name) + " must be on a CUDA device, got " + t.device().str());
  return t;
}

struct Rows {
  void* at = nullptr;
  int64_t stride = 0;  // elements from token to token
};

// A bf16 [T, heads, D] tensor whose tokens' heads are contiguous.
Rows rows(PyObject* o, const char* name, c10::Device dev, int64_t T, int64_t heads, int64_t D) {
  const at::Tensor& t = tensor(o, name, at::kBFloat16);
  on_device(t, name, dev);
  of_shape(t, name, {T, heads, D});
  Rows r;
  r.at = t.data_ptr();
  r.stride = T > 1 ? t.stride(0) : heads * D;
  if (t.numel() > 0 && ((D > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != D)))
    raise(PyExc_ValueError, std::string(name) + ": the heads of a token must be contiguous");
  if (t.numel() == 0) r.stride = heads * D;
  return r;
}

int64_t heads_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name, at::kBFloat16);
  if (t.dim() != 3) raise(PyExc_ValueError, std::string(name) + " must be [T, heads, D]");
  return t.size(1);
}

int as_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX)
    raise(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

int64_t number(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  (void)name;
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

// The tensors a call allocates and the stream it runs on.
class Call {
 public:
  Call(c10::Device dev, PyObject* stream) : dev_(dev), guard_(dev) {
    const auto current = c10::cuda::getCurrentCUDAStream(dev.index());
    current_ = stream_ = current.unwrap();
    if (stream != Py_None) {
      const int64_t id = attr(stream, "stream_id"), index = attr(stream, "device_index");
      if (index != dev.index())
        raise(PyExc_ValueError, "stream must be on " + dev.str() + ", got cuda:" +
                                    std::to_string(index));
      stream_ = c10::Stream::unpack3(id, dev.index(), c10::DeviceType::CUDA);
      other_ = stream_ != current_;
    }
  }
  // Memory of the call's stream: a block of the current one's may still have work
  // pending there.  The caller reads the tensor on the current stream, which the
  // allocator has to be told.
  at::Tensor make(c10::IntArrayRef shape, c10::ScalarType dtype) {
    if (!other_) return at::detail::empty_cuda(shape, dtype, dev_, std::nullopt);
    const c10::cuda::CUDAStreamGuard on(stream_);
    at::Tensor t = at::detail::empty_cuda(shape, dtype, dev_, std::nullopt);
    t.record_stream(current_);
    return t;
  }
  void* stream() const { return c10::cuda::CUDAStream(stream_).stream(); }
  static void check(int status, const char* what) {
    if (status == CPATTN_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", status, what);
    if (e != nullptr) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw Raised();
  }

 private:
  static int64_t attr(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    if (v == nullptr) throw Raised();
    const int64_t n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) throw Raised();
    return n;
  }
  c10::Device dev_;
  c10::cuda::CUDAGuard guard_;
  c10::Stream stream_{c10::Stream::DEFAULT, c10::Device(c10::DeviceType::CPU)};
  c10::Stream current_{c10::Stream::DEFAULT, c10::Device(c10::DeviceType::CPU)};
  bool other_ = false;
};

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* keep(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// A new tuple of references that the callee owns.
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t != nullptr && o != nullptr) PyTuple_SET_ITEM(t, i, o);
    ++i;
  }
  for (PyObject* o : items)
    if (o == nullptr) {
      Py_XDECREF(t);
      throw Raised();
    }
  if (t == nullptr) throw Raised();
  return t;
}

// An output: the caller's tensor, or a new one.
struct Output {
  PyObject* given = nullptr;
  at::Tensor made;
  Rows r;
  PyObject* object() const { return given ? keep(given) : wrap(made); }
};

Output rows_out(Call& call, PyObject* o, const char* name, c10::Device dev, int64_t T,
                int64_t heads, int64_t D) {
  Output out;
  if (o == Py_None) {
    out.made = call.make({T, heads, D}, at::kBFloat16);
    out.r.at = out.made.data_ptr();
    out.r.stride = heads * D;
  } else {
    out.given = o;
    out.r = rows(o, name, dev, T, heads, D);
  }
  return out;
}

Output flat_out(Call& call, PyObject* o, const char* name, c10::ScalarType dtype, c10::Device dev,
                c10::IntArrayRef shape) {
  Output out;
  if (o == Py_None) {
    out.made = call.make(shape, dtype);
    out.r.at = out.made.data_ptr();
  } else {
    out.given = o;
    out.r.at = flat(o, name, dtype, dev, shape);
  }
  return out;
}

// What the norm + rotation calls share.
struct TurnArgs {
  const int32_t* positions = nullptr;
  const float* table = nullptr;
  int rot = 0, max_pos = 0;
  const void *wq = nullptr, *wk = nullptr;
  int32_t* status = nullptr;
};

TurnArgs turn_args(PyObject* positions, PyObject* table, PyObject* wq, PyObject* wk,
                   PyObject* status, int64_t T, int64_t D, c10::Device dev) {
  TurnArgs a;
  if (table != Py_None) {
    const at::Tensor& t = tensor(table, "rope_table", at::kFloat);
    if (t.dim() != 2)
      raise(PyExc_ValueError, "rope_table must be [max_position, rotary_dim]");
    // Its address would be null, which means that there is no rotation.
    if (t.numel() == 0) raise(PyExc_ValueError, "rope_table must not be empty");
    a.max_pos = as_int(t.size(0), "max_position");
    a.rot = as_int(t.size(1), "rotary_dim");
    a.table = static_cast<const float*>(flat(table, "rope_table", at::kFloat, dev, t.sizes()));
    if (positions != nullptr)
      a.positions = static_cast<const int32_t*>(flat(positions, "positions", at::kInt, dev, {T}));
  }
  if (wq != Py_None) a.wq = flat(wq, "q_weight", at::kBFloat16, dev, {D});
  if (wk != Py_None) a.wk = flat(wk, "k_weight", at::kBFloat16, dev, {D});
  if (status != Py_None)
    a.status = static_cast<int32_t*>(flat(status, "status", at::kInt, dev, {1}));
  return a;
}

// q, k, positions, rope_table, q_weight, k_weight, eps, interleaved, q_out,
// k_out, status, stream -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject* const* a) {
  const at::Tensor& q = leading(a[0], "q");
  const c10::Device dev = q.device();
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2), Hk = heads_of(a[1], "k");
  const Rows qr = rows(a[0], "q", dev, T, H, D), kr = rows(a[1], "k", dev, T, Hk, D);
  const TurnArgs t = turn_args(a[2], a[3], a[4], a[5], a[10], T, D, dev);
  const float eps = static_cast<float>(real(a[6]));
  const bool interleaved = truth(a[7]);
  Call call(dev, a[11]);
  const Output qo = rows_out(call, a[8], "q_out", dev, T, H, D);
  const Output ko = rows_out(call, a[9], "k_out", dev, T, Hk, D);
  Call::check(cpattn_qk_norm_rope(qr.at, qr.stride, kr.at, kr.stride, t.positions, t.table, t.rot,
                                  t.max_pos, t.wq, t.wk, eps, interleaved, T, as_int(H, "heads"),
                                  as_int(Hk, "heads"), as_int(D, "head_dim"), qo.r.at,
                                  qo.r.stride, ko.r.at, ko.r.stride, t.status, call.stream()),
              "cpattn_qk_norm_rope");
  return tuple({qo.object(), ko.object()});
}

// dq_out, dk_out, q, k, positions, rope_table, q_weight, k_weight, eps,
// interleaved, dq, dk, dq_weight, dk_weight, workspace, status, stream
// -> (dq, dk, dq_weight, dk_weight)
PyObject* qk_norm_rope_bwd(PyObject* const* a) {
  const at::Tensor& gq = leading(a[0], "dq_out");
  const c10::Device dev = gq.device();
  const int64_t T = gq.size(0), H = gq.size(1), D = gq.size(2), Hk = heads_of(a[1], "dk_out");
  const Rows gqr = rows(a[0], "dq_out", dev, T, H, D), gkr = rows(a[1], "dk_out", dev, T, Hk, D);
  const TurnArgs t = turn_args(a[4], a[5], a[6], a[7], a[15], T, D, dev);
  const float eps = static_cast<float>(real(a[8]));
  const bool interleaved = truth(a[9]);
  const bool normed = t.wq != nullptr || t.wk != nullptr;
  Rows qr, kr;
  if (normed) {
    qr = rows(a[2], "q", dev, T, H, D);
    kr = rows(a[3], "k", dev, T, Hk, D);
  } else if (a[12] != Py_None || a[13] != Py_None) {
    raise(PyExc_ValueError, "dq_weight and dk_weight need q_weight and k_weight");
  }
  Call call(dev, a[16]);
  const Output dq = rows_out(call, a[10], "dq", dev, T, H, D);
  const Output dk = rows_out(call, a[11], "dk", dev, T, Hk, D);
  Output dwq, dwk, ws;
  size_t ws_bytes = 0;
  if (normed) {
    dwq = flat_out(call, a[12], "dq_weight", at::kFloat, dev, {D});
    dwk = flat_out(call, a[13], "dk_weight", at::kFloat, dev, {D});
    int64_t bytes =
        static_cast<int64_t>(cpattn_qk_norm_rope_bwd_workspace_size(as_int(D, "head_dim")));
    if (a[14] != Py_None) bytes = tensor(a[14], "workspace", at::kByte).numel();
    ws = flat_out(call, a[14], "workspace", at::kByte, dev, {bytes});
    ws_bytes = static_cast<size_t>(bytes);
  }
  Call::check(
      cpattn_qk_norm_rope_bwd(gqr.at, gqr.stride, gkr.at, gkr.stride, qr.at, qr.stride, kr.at,
                              kr.stride, t.positions, t.table, t.rot, t.max_pos, t.wq, t.wk, eps,
                              interleaved, T, as_int(H, "heads"), as_int(Hk, "heads"),
                              as_int(D, "head_dim"), dq.r.at, dq.r.stride, dk.r.at, dk.r.stride,
                              static_cast<float*>(dwq.r.at), static_cast<float*>(dwk.r.at),
                              ws.r.at, ws_bytes, t.status, call.stream()),
      "cpattn_qk_norm_rope_bwd");
  return tuple({dq.object(), dk.object(), normed ? dwq.object() : keep(Py_None),
                normed ? dwk.object() : keep(Py_None)});
}

struct Cache {
  void *k = nullptr, *v = nullptr;
  int64_t pages = 0, page_stride = 0;
  int size = 0, heads = 0, seqs = 0, row = 0, dim = 0;
  const int32_t *table = nullptr, *cu = nullptr, *kv = nullptr;
};

// One cache of that shape, its pages contiguous; its address, and the elements from
// page to page.
void* page_args(PyObject* o, const char* name, c10::ScalarType dtype, c10::Device dev,
                c10::IntArrayRef shape, int64_t* stride) {
  const at::Tensor& t = tensor(o, name, dtype);
  on_device(t, name, dev);
  of_shape(t, name, shape);
  *stride = shape[1] * shape[2] * shape[3];
  if (!t.is_contiguous()) {
    int64_t want = 1;
    for (int d = 3; d > 0; --d) {
      if (t.size(d) > 1 && t.stride(d) != want)
        raise(PyExc_ValueError, std::string(name) + ": a page must be contiguous");
      want *= t.size(d);
    }
    if (shape[0] > 1) *stride = t.stride(0);
  }
  return t.data_ptr();
}

// k_cache and v_cache (a[0], a[1]) of that shape, page_table, cu_seqlens, kv_lens.
void cache_tensors(Cache& c, PyObject* const* a, c10::ScalarType dtype, c10::Device dev,
                   c10::IntArrayRef shape) {
  int64_t strides[2];
  c.k = page_args(a[0], "k_cache", dtype, dev, shape, strides);
  c.v = page_args(a[1], "v_cache", dtype, dev, shape, strides + 1);
  if (strides[0] != strides[1])
    raise(PyExc_ValueError, "k_cache and v_cache must have the same page stride");
  c.page_stride = strides[0];
  const at::Tensor& kv = tensor(a[4], "kv_lens", at::kInt);
  if (kv.dim() != 1) raise(PyExc_ValueError, "kv_lens must be [num_seqs]");
  const at::Tensor& table = tensor(a[2], "page_table", at::kInt);
  if (table.dim() != 2) raise(PyExc_ValueError, "page_table must be [num_seqs, max_pages]");
  c.seqs = as_int(kv.size(0), "num_seqs");
  c.row = as_int(table.size(1), "max_pages");
  c.table = static_cast<int32_t*>(
      flat(a[2], "page_table", at::kInt, dev, {kv.size(0), table.size(1)}));
  c.cu = static_cast<int32_t*>(flat(a[3], "cu_seqlens", at::kInt, dev, {kv.size(0) + 1}));
  c.kv = static_cast<int32_t*>(flat(a[4], "kv_lens", at::kInt, dev, {kv.size(0)}));
}

// k_cache, v_cache, page_table, cu_seqlens, kv_lens; heads < 0: the cache's.
Cache cache_args(PyObject* const* a, c10::Device dev, int64_t heads, int64_t D) {
  Cache c;
  const at::Tensor& k = tensor(a[0], "k_cache", at::kBFloat16);
  if (k.dim() != 4)
    raise(PyExc_ValueError, "k_cache must be [num_pages, page_size, heads, D]");
  if (heads < 0) heads = k.size(2);
  c.pages = k.size(0);
  c.size = as_int(k.size(1), "page_size");
  c.heads = as_int(heads, "heads");
  cache_tensors(c, a, at::kBFloat16, dev, {c.pages, c.size, heads, D});
  return c;
}

// The same with 4-bit caches (strides in bytes); D < 0: the cache's.
Cache fp4_args(PyObject* const* a, c10::Device dev, int64_t heads, int64_t D) {
  Cache c;
  const at::Tensor& k = tensor(a[0], "k_cache", at::kByte);
  if (k.dim() != 4)
    raise(PyExc_ValueError, "k_cache must be [num_pages, heads, page_size, 9 * D / 16]");
  if (heads < 0) heads = k.size(1);
  if (D < 0) D = k.size(3) / 9 * 16;
  c.pages = k.size(0);
  c.size = as_int(k.size(2), "page_size");
  c.heads = as_int(heads, "heads");
  c.dim = as_int(D, "head_dim");
  cache_tensors(c, a, at::kByte, dev, {c.pages, heads, c.size, D / 16 * 9});
  return c;
}

// k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, rope_table,
// interleaved, k_weight, eps, q, q_weight, q_out, status, stream -> q_out
PyObject* paged_append(PyObject* const* a) {
  const at::Tensor& k = leading(a[0], "k");
  const c10::Device dev = k.device();
  const int64_t T = k.size(0), Hk = k.size(1), D = k.size(2);
  const Rows kr = rows(a[0], "k", dev, T, Hk, D), vr = rows(a[1], "v", dev, T, Hk, D);
  const Cache c = cache_args(a + 2, dev, Hk, D);
  const TurnArgs t = turn_args(nullptr, a[7], a[12], a[9], a[14], T, D, dev);
  const bool interleaved = truth(a[8]);
  const float eps = static_cast<float>(real(a[10]));
  const bool with_q = a[11] != Py_None;
  if (!with_q && (a[12] != Py_None || a[13] != Py_None))
    raise(PyExc_ValueError, "q_out and q_weight need q");
  const int64_t H = with_q ? heads_of(a[11], "q") : 0;
  Rows qr;
  if (with_q) qr = rows(a[11], "q", dev, T, H, D);
  Call call(dev, a[15]);
  Output qo;
  if (with_q) qo = rows_out(call, a[13], "q_out", dev, T, H, D);
  Call::check(cpattn_paged_append(kr.at, kr.stride, vr.at, vr.stride, c.k, c.v, c.pages, c.size,
                                  c.page_stride, c.table, c.row, c.cu, c.kv, c.seqs, T,
                                  as_int(Hk, "heads"), as_int(D, "head_dim"), t.table, t.rot,
                                  t.max_pos, interleaved, t.wq, t.wk, eps,
                                  with_q ? qr.at : nullptr, qr.stride, as_int(H, "heads"),
                                  qo.r.at, qo.r.stride, t.status, call.stream()),
              "cpattn_paged_append");
  return with_q ? qo.object() : keep(Py_None);
}

// q, k_cache, v_cache, page_table, cu_seqlens, kv_lens, max_seqlen, max_kv_len,
// softmax_scale, causal, out, lse, workspace, stream -> (out, lse)
PyObject* paged_attn(PyObject* const* a) {
  const at::Tensor& q = leading(a[0], "q");
  const c10::Device dev = q.device();
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
  if (!q.is_contiguous()) raise(PyExc_ValueError, "q must be contiguous");
  const Cache c = cache_args(a + 1, dev, -1, D);
  const int max_q = as_int(number(a[6], "max_seqlen"), "max_seqlen");
  const int max_kv = as_int(number(a[7], "max_kv_len"), "max_kv_len");
  const float scale =
      a[8] == Py_None ? 1.f / std::sqrt(static_cast<float>(D)) : static_cast<float>(real(a[8]));
  const bool causal = truth(a[9]);
  Call call(dev, a[13]);
  const Output out = flat_out(call, a[10], "out", at::kBFloat16, dev, {T, H, D});
  const Output lse = flat_out(call, a[11], "lse", at::kFloat, dev, {T, H});
  int64_t bytes;
  if (a[12] != Py_None) {
    bytes = tensor(a[12], "workspace", at::kByte).numel();
  } else {
    bytes = static_cast<int64_t>(cpattn_paged_attn_workspace_size(
        T, c.seqs, as_int(H, "heads"), c.heads, as_int(D, "head_dim"), max_q));
    // Sizes the call itself will refuse, with its status.
    if (bytes == 0) bytes = 256;
  }
  const Output ws = flat_out(call, a[12], "workspace", at::kByte, dev, {bytes});
  Call::check(cpattn_paged_attn(q.data_ptr(), c.k, c.v, c.pages, c.size, c.page_stride, c.table,
                                c.row, c.cu, c.kv, c.seqs, T, max_q, max_kv, as_int(H, "heads"),
                                c.heads, as_int(D, "head_dim"), scale, causal, out.r.at,
                                static_cast<float*>(lse.r.at), ws.r.at,
                                static_cast<size_t>(bytes), call.stream()),
              "cpattn_paged_attn");
  return tuple({out.object(), lse.object()});
}

// k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, k_scale, v_scale, status,
// stream -> None
PyObject* paged_append_fp4(PyObject* const* a) {
  const at::Tensor& k = leading(a[0], "k");
  const c10::Device dev = k.device();
  const int64_t T = k.size(0), Hk = k.size(1), D = k.size(2);
  const Rows kr = rows(a[0], "k", dev, T, Hk, D), vr = rows(a[1], "v", dev, T, Hk, D);
  const Cache c = fp4_args(a + 2, dev, Hk, D);
  const float ks = static_cast<float>(real(a[7])), vs = static_cast<float>(real(a[8]));
  int32_t* status = nullptr;
  if (a[9] != Py_None) status = static_cast<int32_t*>(flat(a[9], "status", at::kInt, dev, {1}));
  Call call(dev, a[10]);
  Call::check(cpattn_paged_append_fp4(kr.at, kr.stride, vr.at, vr.stride, c.k, c.v, c.pages, c.size,
                                      c.page_stride, c.table, c.row, c.cu, c.kv, c.seqs, T,
                                      c.heads, c.dim, ks, vs, status, call.stream()),
              "cpattn_paged_append_fp4");
  return keep(Py_None);
}

// k_cache, v_cache, page_table, cu_seqlens, kv_lens, total_tokens, k_scale, v_scale,
// k_out, v_out, status, stream -> (k_out, v_out)
PyObject* paged_gather_fp4(PyObject* const* a) {
  const at::Tensor& cache = tensor(a[0], "k_cache", at::kByte);
  if (!cache.is_cuda())
    raise(PyExc_ValueError, "k_cache must be on a CUDA device, got " + cache.device().str());
  const c10::Device dev = cache.device();
  const Cache c = fp4_args(a, dev, -1, -1);
  const int64_t T = number(a[5], "total_tokens");
  if (T < 0) raise(PyExc_ValueError, "total_tokens must not be negative");
  const float ks = static_cast<float>(real(a[6])), vs = static_cast<float>(real(a[7]));
  int32_t* status = nullptr;
  if (a[10] != Py_None) status = static_cast<int32_t*>(flat(a[10], "status", at::kInt, dev, {1}));
  Call call(dev, a[11]);
  const Output ko = rows_out(call, a[8], "k_out", dev, T, c.heads, c.dim);
  const Output vo = rows_out(call, a[9], "v_out", dev, T, c.heads, c.dim);
  Call::check(cpattn_paged_gather_fp4(c.k, c.v, c.pages, c.size, c.page_stride, c.table, c.row,
                                      c.cu, c.kv, c.seqs, T, c.heads, c.dim, ks, vs, ko.r.at,
                                      ko.r.stride, vo.r.at, vo.r.stride, status, call.stream()),
              "cpattn_paged_gather_fp4");
  return tuple({ko.object(), vo.object()});
}

// q, k_cache, v_cache, page_table, cu_seqlens, kv_lens, max_seqlen, max_kv_len, k_scale,
// v_scale, softmax_scale, causal, out, lse, workspace, stream -> (out, lse)
PyObject* paged_attn_fp4(PyObject* const* a) {
  const at::Tensor& q = leading(a[0], "q");
  const c10::Device dev = q.device();
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
  if (!q.is_contiguous()) raise(PyExc_ValueError, "q must be contiguous");
  const Cache c = fp4_args(a + 1, dev, -1, D);
  const int max_q = as_int(number(a[6], "max_seqlen"), "max_seqlen");
  const int max_kv = as_int(number(a[7], "max_kv_len"), "max_kv_len");
  const float ks = static_cast<float>(real(a[8])), vs = static_cast<float>(real(a[9]));
  const float scale =
      a[10] == Py_None ? 1.f / std::sqrt(static_cast<float>(D)) : static_cast<float>(real(a[10]));
  const bool causal = truth(a[11]);
  Call call(dev, a[15]);
  const Output out = flat_out(call, a[12], "out", at::kBFloat16, dev, {T, H, D});
  const Output lse = flat_out(call, a[13], "lse", at::kFloat, dev, {T, H});
  int64_t bytes;
  if (a[14] != Py_None) {
    bytes = tensor(a[14], "workspace", at::kByte).numel();
  } else {
    bytes = static_cast<int64_t>(cpattn_paged_attn_fp4_workspace_size(
        T, c.seqs, as_int(H, "heads"), c.heads, c.dim, max_q, max_kv));
    // Sizes the call itself will refuse, with its status.
    if (bytes == 0) bytes = 256;
  }
  const Output ws = flat_out(call, a[14], "workspace", at::kByte, dev, {bytes});
  Call::check(cpattn_paged_attn_fp4(q.data_ptr(), c.k, c.v, c.pages, c.size, c.page_stride, c.table,
                                    c.row, c.cu, c.kv, c.seqs, T, max_q, max_kv,
                                    as_int(H, "heads"), c.heads, c.dim, ks, vs, scale, causal,
                                    out.r.at, static_cast<float*>(lse.r.at), ws.r.at,
                                    static_cast<size_t>(bytes), call.stream()),
              "cpattn_paged_attn_fp4");
  return tuple({out.object(), lse.object()});
}

// Every call: its number of arguments, and no C++ exception past this point.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<qk_norm_rope, 12>("qk_norm_rope"),
    method<qk_norm_rope_bwd, 17>("qk_norm_rope_bwd"),
    method<paged_append, 16>("paged_append"),
    method<paged_attn, 14>("paged_attn"),
    method<paged_append_fp4, 11>("paged_append_fp4"),
    method<paged_gather_fp4, 12>("paged_gather_fp4"),
    method<paged_attn_fp4, 16>("paged_attn_fp4"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
