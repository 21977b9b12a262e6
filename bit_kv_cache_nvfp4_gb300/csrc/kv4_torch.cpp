// kv4_torch.cpp -- the PyTorch side of the *_gqa8, *_gqa4 and rotary entry points: a Python
// extension module (_kv4torch) that checks tensors, allocates outputs and
// workspace, and calls the C ABI on the tensors' device and its current
// stream.
//
// A decode step's write or a short attention takes 3 to 12 us on the GPU; the
// same checks and the call written in Python over ctypes took 11 to 17 us of a
// GB300's host core, so such calls waited for their binding.  Written here they
// take 2 to 6.
//
// Bad arguments raise TypeError or ValueError before anything is launched.  A
// nonzero kv4_status is returned as an int, which the Python wrapper
// (gqa8.py, gqa4.py, rotary.py) turns into Kv4Error.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "kv4mla.h"

namespace {

struct BadArg {
  PyObject* type;
  std::string what;
};
[[noreturn]] void type_error(const std::string& s) { throw BadArg{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw BadArg{PyExc_ValueError, s}; }

std::string name_of(at::ScalarType t) {
  switch (t) {
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    default: return c10::toString(t);
  }
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
  return t;
}
void same_device(const at::Tensor& t, const char* name, c10::Device dev) {
  if (t.device() != dev)
    value_error(std::string(name) + " is on " + t.device().str() + ", the pool on " + dev.str());
}
// A contiguous tensor of this type and rank on the pool's device.
const at::Tensor& plain(PyObject* o, const char* name, at::ScalarType type, int dim, c10::Device dev) {
  const at::Tensor& t = cuda_tensor(o, name);
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
  if (t.dim() != dim)
    value_error(std::string(name) + " must have " + std::to_string(dim) + " dimensions, got " +
                std::to_string(t.dim()));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  same_device(t, name, dev);
  return t;
}
int dtype_code(at::ScalarType t, const char* name) {
  if (t == at::kBFloat16) return KV4_BF16;
  if (t == at::kHalf) return KV4_F16;
  type_error(std::string(name) + " must be bfloat16 or float16, got " + name_of(t));
}
// A [T, heads, D] input: last dimension contiguous, the others any multiple of
// 16 bytes.  (The stride of a dimension of one element says nothing: a
// contiguous tensor may have any.)
struct Strided {
  const void* p;
  int64_t token, head;
};
Strided strided(const at::Tensor& t, const char* name) {
  Strided s{t.const_data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
  if (t.stride(2) != 1 || s.token % 8 != 0 || s.head % 8 != 0 || (reinterpret_cast<uintptr_t>(s.p) & 15) != 0)
    value_error(std::string(name) +
                ": the last dimension must be contiguous, the other strides multiples of 8 elements "
                "and the data 16-byte aligned");
  return s;
}

struct Cache {
  c10::Device dev{c10::kCPU};
  uint8_t *pool, *scales;
  const int32_t* table;
  int64_t pages, stride;
  int B, hkv, d;
};
// The cache of 8-bit pages, [.., 64, D] with an exponent a block, or of 4-bit ones,
// [.., 64, D / 2] with a scale for each 16 elements.
template <int BITS>
Cache cache(PyObject* pool_o, PyObject* scales_o, PyObject* table_o) {
  constexpr bool k4 = BITS == 4;
  Cache c;
  const at::Tensor& pool = cuda_tensor(pool_o, "pool");
  if (pool.dim() != 5 || pool.size(2) != 2 || pool.size(3) != KV4_PAGE)
    value_error(k4 ? "pool must be [num_pages, Hkv, 2, 64, D / 2]" : "pool must be [num_pages, Hkv, 2, 64, D]");
  c.dev = pool.device();
  plain(pool_o, "pool", at::kByte, 5, c.dev);
  const at::Tensor& scales = plain(scales_o, "scales", at::kByte, k4 ? 5 : 3, c.dev);
  const at::Tensor& table = plain(table_o, "page_table", at::kInt, 2, c.dev);
  c.pages = pool.size(0);
  if (pool.size(1) < 1 || pool.size(1) > 65535) value_error("pool: no or too many heads");
  c.hkv = static_cast<int>(pool.size(1));
  c.d = static_cast<int>(std::min<int64_t>(pool.size(4), 1 << 20)) * (k4 ? 2 : 1);
  if (scales.size(0) != c.pages || scales.size(1) != c.hkv || scales.size(2) != 2 ||
      (k4 && (scales.size(3) != KV4_PAGE || scales.size(4) != c.d / 16)))
    value_error("scales must be [" + std::to_string(c.pages) + ", " + std::to_string(c.hkv) + ", 2" +
                (k4 ? ", 64, " + std::to_string(c.d / 16) : "") + "]");
  c.pool = pool.mutable_data_ptr<uint8_t>();
  c.scales = scales.mutable_data_ptr<uint8_t>();
  c.table = table.const_data_ptr<int32_t>();
  c.stride = table.size(1);
  c.B = static_cast<int>(std::min<int64_t>(table.size(0), 1 << 30));
  return c;
}
// cu_seqlens [B + 1] and a length or position for each request.
void ragged(const Cache& c, PyObject* cu_o, PyObject* len_o, const char* len_name, const int32_t*& cu,
            const int32_t*& lens) {
  const at::Tensor& t = plain(cu_o, "cu_seqlens", at::kInt, 1, c.dev);
  const at::Tensor& l = plain(len_o, len_name, at::kInt, 1, c.dev);
  if (t.size(0) != static_cast<int64_t>(c.B) + 1 || l.size(0) != c.B)
    value_error(std::string("page_table [B, *], cu_seqlens [B + 1] and ") + len_name + " [B] must agree");
  cu = t.const_data_ptr<int32_t>();
  lens = l.const_data_ptr<int32_t>();
}
int32_t* err_word(PyObject* o, c10::Device dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = plain(o, "dev_err", at::kInt, 1, dev);
  if (t.size(0) < 1) value_error("dev_err must have an element");
  return t.mutable_data_ptr<int32_t>();
}
int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < 0 || v > INT32_MAX) value_error(std::string(name) + " must be in [0, 2^31)");
  return static_cast<int>(v);
}
kv4_stream_t stream_of(c10::Device dev) {
  return reinterpret_cast<kv4_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}
// An output: the caller's, checked, or a new one (past the dispatcher, which
// for a CUDA tensor only leads there).
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  if (o == Py_None) return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
  const at::Tensor& t = plain(o, name, type, static_cast<int>(shape.size()), dev);
  if (t.sizes() != shape) {
    std::string s;
    for (const int64_t n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
    value_error(std::string(name) + " must be [" + s + "]");
  }
  return t;
}

// A tensor of the caller's that a call writes into: autograd has to learn that
// what it may have saved of it is gone.  (Inference tensors count nothing.)
void written(PyObject* o) {
  if (o == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* pair_or_status(kv4_status st, const at::Tensor& a, const at::Tensor& b) {
  if (st != KV4_OK) return PyLong_FromLong(st);
  PyObject* t = PyTuple_New(2);
  if (t == nullptr) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

template <Py_ssize_t N, typename F>
PyObject* guarded(const char* name, Py_ssize_t n, F&& f) {
  HANDLE_TH_ERRORS
  try {
    if (n != N) type_error(std::string(name) + " takes " + std::to_string(N) + " arguments");
    return f();
  } catch (const BadArg& e) {
    PyErr_SetString(e.type, e.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// k, v, cu_seqlens, page_table, seq_lens, pool, scales, dev_err
template <int BITS>
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<8>("append", n, [&]() -> PyObject* {
    const Cache c = cache<BITS>(a[5], a[6], a[3]);
    const at::Tensor &k = cuda_tensor(a[0], "k"), &v = cuda_tensor(a[1], "v");
    const int dt = dtype_code(k.scalar_type(), "k");
    if (v.scalar_type() != k.scalar_type())
      type_error("v must be " + name_of(k.scalar_type()) + ", got " + name_of(v.scalar_type()));
    if (k.dim() != 3 || k.sizes() != v.sizes() || k.size(1) != c.hkv || k.size(2) != c.d)
      value_error("k and v must be [T, " + std::to_string(c.hkv) + ", " + std::to_string(c.d) + "]");
    same_device(k, "k", c.dev);
    same_device(v, "v", c.dev);
    const Strided sk = strided(k, "k"), sv = strided(v, "v");
    const int32_t *cu, *lens;
    ragged(c, a[2], a[4], "seq_lens", cu, lens);
    int32_t* const err = err_word(a[7], c.dev);
    const c10::cuda::CUDAGuard guard(c.dev);
    const kv4_status st =
        (BITS == 8 ? kv4_append_gqa8 : kv4_append_gqa4)(sk.p, sk.token, sk.head, sv.p, sv.token, sv.head, dt, k.size(0), cu, c.table, c.stride,
                        KV4_PAGE, lens, c.B, c.hkv, c.d, c.pool, c.scales, c.pages, err, stream_of(c.dev));
    if (st == KV4_OK)
      for (const int i : {5, 6, 7}) written(a[i]);
    return PyLong_FromLong(st);
  });
}

// pool, scales, page_table, starts, cu_seqlens, total, f16, k_out, v_out, dev_err
template <int BITS>
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>("read", n, [&]() -> PyObject* {
    const Cache c = cache<BITS>(a[0], a[1], a[2]);
    const int32_t *cu, *starts;
    ragged(c, a[4], a[3], "starts", cu, starts);
    const int64_t total = small(a[5], "total");
    const int f16 = PyObject_IsTrue(a[6]);
    int32_t* const err = err_word(a[9], c.dev);
    const c10::cuda::CUDAGuard guard(c.dev);
    const at::ScalarType type = f16 ? at::kHalf : at::kBFloat16;
    const at::Tensor k = output(a[7], "k_out", {total, c.hkv, c.d}, type, c.dev);
    const at::Tensor v = output(a[8], "v_out", {total, c.hkv, c.d}, type, c.dev);
    const kv4_status st =
        (BITS == 8 ? kv4_read_gqa8 : kv4_read_gqa4)(c.pool, c.scales, c.pages, c.table, c.stride, KV4_PAGE, starts, cu, total, c.B, c.hkv, c.d,
                      f16 ? KV4_F16 : KV4_BF16, k.mutable_data_ptr(), v.mutable_data_ptr(), err, stream_of(c.dev));
    if (st == KV4_OK)
      for (const int i : {7, 8, 9}) written(a[i]);
    return pair_or_status(st, k, v);
  });
}

// q, pool, scales, page_table, seq_lens, cu_seqlens, max_new, sm_scale, window, out, lse, workspace, dev_err
template <int BITS>
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<13>("attention", n, [&]() -> PyObject* {
    const Cache c = cache<BITS>(a[1], a[2], a[3]);
    const at::Tensor& q = cuda_tensor(a[0], "q");
    const int dt = dtype_code(q.scalar_type(), "q");
    if (q.dim() != 3 || q.size(2) != c.d || q.size(1) < 1 || q.size(1) % c.hkv != 0 || q.size(1) > (1 << 30))
      value_error("q must be [T, Hq, " + std::to_string(c.d) + "] with Hq a multiple of " + std::to_string(c.hkv));
    same_device(q, "q", c.dev);
    const Strided sq = strided(q, "q");
    const int64_t t = q.size(0);
    const int hq = static_cast<int>(q.size(1));
    const int32_t *cu, *lens;
    ragged(c, a[5], a[4], "seq_lens", cu, lens);
    const int max_new = small(a[6], "max_new"), window = small(a[8], "window");
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      type_error("sm_scale must be a number");
    }
    int32_t* const err = err_word(a[12], c.dev);
    const c10::cuda::CUDAGuard guard(c.dev);
    const at::Tensor out = output(a[9], "out", {t, hq, c.d}, q.scalar_type(), c.dev);
    const at::Tensor lse = output(a[10], "lse", {t, hq}, at::kFloat, c.dev);
    c10::DataPtr own;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[11] == Py_None) {
      const kv4_status st = (BITS == 8 ? kv4_attention_gqa8_plan : kv4_attention_gqa4_plan)(c.B, max_new, t, hq, c.hkv, c.d, &ws_bytes);
      if (st != KV4_OK) return PyLong_FromLong(st);
      if (ws_bytes > 0) {
        own = c10::cuda::CUDACachingAllocator::get()->allocate(ws_bytes);
        ws = own.get();
      }
    } else {
      const at::Tensor& given = plain(a[11], "workspace", at::kByte, 1, c.dev);
      ws = given.mutable_data_ptr();
      ws_bytes = given.numel();
    }
    const kv4_status st =
        (BITS == 8 ? kv4_attention_gqa8 : kv4_attention_gqa4)(sq.p, sq.token, sq.head, dt, t, cu, max_new, c.pool, c.scales, c.pages, c.table, c.stride,
                           KV4_PAGE, lens, c.B, hq, c.hkv, c.d, window, static_cast<float>(scale),
                           out.mutable_data_ptr(), lse.mutable_data_ptr<float>(), ws, ws_bytes, err,
                           stream_of(c.dev));
    if (st == KV4_OK)
      for (const int i : {9, 10, 11, 12}) written(a[i]);
    return pair_or_status(st, out, lse);
  });
}

// One side of a rotary call, q or k: nothing (None), or [T, heads, D] with contiguous
// heads; the output is the caller's (which may be the input itself) or a new one.
struct Side {
  const void* in = nullptr;
  void* out = nullptr;
  int64_t in_token = 0, in_head = 0, out_token = 0, out_head = 0, tokens = 0;
  int heads = 0, d = 0;
  at::Tensor result;
};
// Rows of a side's input or output, strides in elements of 16 bits.
struct Rows {
  const char* p;
  int64_t token, head, tokens;
  int heads, d;
  int64_t row() const { return 2 * ((heads - 1) * head + d); }
  int64_t span() const { return 2 * (tokens - 1) * token + row(); }
};
Rows in_of(const Side& s) { return {static_cast<const char*>(s.in), s.in_token, s.in_head, s.tokens, s.heads, s.d}; }
Rows out_of(const Side& s) { return {static_cast<const char*>(s.out), s.out_token, s.out_head, s.tokens, s.heads, s.d}; }
// Whether no element is both a's and b's: apart as a whole, or in every token (slices of a
// fused projection's rows), or in every head (of a projection [T, heads, parts, D]).
bool lie_apart(const Rows& a, const Rows& b) {
  if (a.tokens == 0 || a.heads == 0 || b.heads == 0) return true;
  if (a.p + a.span() <= b.p || b.p + b.span() <= a.p) return true;
  auto within = [&](int64_t period, int64_t of_a, int64_t of_b) {
    const int64_t at = ((b.p - a.p) % period + period) % period;
    return of_a <= at && at + of_b <= period;
  };
  if (a.tokens > 1 && a.token > 0 && a.token == b.token && within(2 * a.token, a.row(), b.row())) return true;
  const int64_t head = a.heads > 1 ? a.head : b.head;
  return head > 0 && (a.heads == 1 || b.heads == 1 || a.head == b.head) && a.token % head == 0 && b.token % head == 0 &&
         within(2 * head, 2 * a.d, 2 * b.d);
}
Side side_of(PyObject* in_o, PyObject* out_o, const char* name, const at::Tensor& first) {
  Side s;
  const std::string out_name = std::string(name) + "_out";
  if (in_o == Py_None) {
    if (out_o != Py_None) value_error(out_name + " without " + name);
    return s;
  }
  const at::Tensor& t = cuda_tensor(in_o, name);
  if (t.scalar_type() != first.scalar_type())
    type_error(std::string(name) + " must be " + name_of(first.scalar_type()) + ", got " + name_of(t.scalar_type()));
  if (t.dim() != 3 || t.size(0) != first.size(0)) value_error(std::string(name) + " must be [" + std::to_string(first.size(0)) + ", heads, D]");
  same_device(t, name, first.device());
  auto strides = [](const at::Tensor& x, const std::string& what, int64_t& token, int64_t& head) {
    if (x.size(2) > 1 && x.stride(2) != 1) value_error(what + ": the last dimension must be contiguous");
    token = x.size(0) > 1 ? x.stride(0) : 0;
    head = x.size(1) > 1 ? x.stride(1) : 0;
  };
  if (t.size(1) > 65535 || t.size(2) > 65536) value_error(std::string(name) + ": too many heads or elements");
  s.tokens = t.size(0);
  s.heads = static_cast<int>(t.size(1));
  s.d = static_cast<int>(t.size(2));
  strides(t, name, s.in_token, s.in_head);
  s.in = t.const_data_ptr();
  if (out_o == Py_None) {
    s.result = at::Tensor(at::detail::empty_cuda(t.sizes(), t.scalar_type(), t.device(), std::nullopt));
  } else {
    const at::Tensor& o = cuda_tensor(out_o, out_name.c_str());
    if (o.scalar_type() != t.scalar_type())
      type_error(out_name + " must be " + name_of(t.scalar_type()) + ", got " + name_of(o.scalar_type()));
    if (o.sizes() != t.sizes()) value_error(out_name + " must have the shape of " + name);
    same_device(o, out_name.c_str(), t.device());
    s.result = o;
  }
  strides(s.result, out_name, s.out_token, s.out_head);
  s.out = s.result.mutable_data_ptr();
  const bool same = s.in == s.out && s.in_token == s.out_token && s.in_head == s.out_head;
  if (t.numel() > 0 && !same && !lie_apart(in_of(s), out_of(s)))
    value_error(out_name + " must be " + name + " itself or lie apart from it");
  return s;
}

// q, k, positions, inv_freq, interleaved, q_offset, k_offset, factor, q_out, k_out
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>("rotary", n, [&]() -> PyObject* {
    const at::Tensor& first = cuda_tensor(a[0] == Py_None ? a[1] : a[0], a[0] == Py_None ? "k" : "q");
    const int dt = dtype_code(first.scalar_type(), a[0] == Py_None ? "k" : "q");
    if (first.dim() != 3) value_error("q and k must be [T, heads, D]");
    const c10::Device dev = first.device();
    const at::Tensor& pos = cuda_tensor(a[2], "positions");
    if (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong)
      type_error("positions must be torch.int32 or torch.int64, got " + name_of(pos.scalar_type()));
    if (pos.dim() != 1 || pos.size(0) != first.size(0) || !pos.is_contiguous())
      value_error("positions must be [" + std::to_string(first.size(0)) + "], contiguous");
    if (pos.device() != dev) value_error("positions is on " + pos.device().str() + ", the inputs on " + dev.str());
    const at::Tensor& freq = cuda_tensor(a[3], "inv_freq");
    if (freq.scalar_type() != at::kFloat) type_error("inv_freq must be torch.float32, got " + name_of(freq.scalar_type()));
    if (freq.dim() != 1 || !freq.is_contiguous()) value_error("inv_freq must have one dimension, contiguous");
    if (freq.device() != dev) value_error("inv_freq is on " + freq.device().str() + ", the inputs on " + dev.str());
    const int near = PyObject_IsTrue(a[4]);
    if (near < 0) {
      PyErr_Clear();
      type_error("interleaved must be a truth value");
    }
    const int q_at = small(a[5], "q_offset"), k_at = small(a[6], "k_offset");
    const double factor = PyFloat_AsDouble(a[7]);
    if (factor == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      type_error("factor must be a number");
    }
    const c10::cuda::CUDAGuard guard(dev);
    const Side q = side_of(a[0], a[8], "q", first), k = side_of(a[1], a[9], "k", first);
    if (a[0] != Py_None && a[1] != Py_None) {
      if (a[8] != Py_None && !lie_apart(out_of(q), in_of(k))) value_error("q_out must lie apart from k");
      if (a[9] != Py_None && !lie_apart(out_of(k), in_of(q))) value_error("k_out must lie apart from q");
      if (a[8] != Py_None && a[9] != Py_None && !lie_apart(out_of(q), out_of(k)))
        value_error("q_out and k_out must lie apart");
    }
    auto room = [&](const Side& s, const char* name, int at) {
      if (s.heads > 0 && (at > s.d || s.d - at < 2 * freq.size(0)))
        value_error(std::string(name) + ": " + std::to_string(2 * freq.size(0)) + " elements from " + std::to_string(at) +
                    " on do not fit a head of " + std::to_string(s.d));
    };
    room(q, "q", q_at);
    room(k, "k", k_at);
    const kv4_status st =
        kv4_rotary(q.in, q.in_token, q.in_head, q.heads, q.d, q_at, q.out, q.out_token, q.out_head, k.in, k.in_token,
                   k.in_head, k.heads, k.d, k_at, k.out, k.out_token, k.out_head, dt, first.size(0),
                   pos.const_data_ptr(), pos.scalar_type() == at::kLong ? 64 : 32, freq.const_data_ptr<float>(),
                   static_cast<int>(std::min<int64_t>(freq.size(0), 1 << 20)), near, static_cast<float>(factor),
                   stream_of(dev));
    if (st != KV4_OK) return PyLong_FromLong(st);
    written(a[8]);
    written(a[9]);
    PyObject* t = PyTuple_New(2);
    if (t == nullptr) return nullptr;
    auto item = [](PyObject* given, PyObject* in, const at::Tensor& made) -> PyObject* {
      if (in == Py_None || given != Py_None) return Py_NewRef(in == Py_None ? Py_None : given);
      return THPVariable_Wrap(made);
    };
    PyTuple_SET_ITEM(t, 0, item(a[8], a[0], q.result));
    PyTuple_SET_ITEM(t, 1, item(a[9], a[1], k.result));
    return t;
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef methods[] = {{"append", fast(append<8>), METH_FASTCALL, "kv4_append_gqa8"},
                         {"read", fast(read<8>), METH_FASTCALL, "kv4_read_gqa8"},
                         {"attention", fast(attention<8>), METH_FASTCALL, "kv4_attention_gqa8"},
                         {"append4", fast(append<4>), METH_FASTCALL, "kv4_append_gqa4"},
                         {"read4", fast(read<4>), METH_FASTCALL, "kv4_read_gqa4"},
                         {"attention4", fast(attention<4>), METH_FASTCALL, "kv4_attention_gqa4"},
                         {"rotary", fast(rotary), METH_FASTCALL, "kv4_rotary"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv4torch", "PyTorch side of the *_gqa8, *_gqa4 and rotary entry points.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4torch() { return PyModule_Create(&module); }
