// kv4_torch.cpp -- the PyTorch side of the *_gqa8 entry points: a Python
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
// (gqa8.py) turns into Kv4Error.
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
Cache cache(PyObject* pool_o, PyObject* scales_o, PyObject* table_o) {
  Cache c;
  const at::Tensor& pool = cuda_tensor(pool_o, "pool");
  if (pool.dim() != 5 || pool.size(2) != 2 || pool.size(3) != KV4_PAGE)
    value_error("pool must be [num_pages, Hkv, 2, 64, D]");
  c.dev = pool.device();
  plain(pool_o, "pool", at::kByte, 5, c.dev);
  const at::Tensor& scales = plain(scales_o, "scales", at::kByte, 3, c.dev);
  const at::Tensor& table = plain(table_o, "page_table", at::kInt, 2, c.dev);
  c.pages = pool.size(0);
  if (pool.size(1) < 1 || pool.size(1) > 65535) value_error("pool: no or too many heads");
  c.hkv = static_cast<int>(pool.size(1));
  c.d = static_cast<int>(std::min<int64_t>(pool.size(4), 1 << 20));
  if (scales.size(0) != c.pages || scales.size(1) != c.hkv || scales.size(2) != 2)
    value_error("scales must be [" + std::to_string(c.pages) + ", " + std::to_string(c.hkv) + ", 2]");
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
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<8>("append", n, [&]() -> PyObject* {
    const Cache c = cache(a[5], a[6], a[3]);
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
        kv4_append_gqa8(sk.p, sk.token, sk.head, sv.p, sv.token, sv.head, dt, k.size(0), cu, c.table, c.stride,
                        KV4_PAGE, lens, c.B, c.hkv, c.d, c.pool, c.scales, c.pages, err, stream_of(c.dev));
    if (st == KV4_OK)
      for (const int i : {5, 6, 7}) written(a[i]);
    return PyLong_FromLong(st);
  });
}

// pool, scales, page_table, starts, cu_seqlens, total, f16, k_out, v_out, dev_err
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<10>("read", n, [&]() -> PyObject* {
    const Cache c = cache(a[0], a[1], a[2]);
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
        kv4_read_gqa8(c.pool, c.scales, c.pages, c.table, c.stride, KV4_PAGE, starts, cu, total, c.B, c.hkv, c.d,
                      f16 ? KV4_F16 : KV4_BF16, k.mutable_data_ptr(), v.mutable_data_ptr(), err, stream_of(c.dev));
    if (st == KV4_OK)
      for (const int i : {7, 8, 9}) written(a[i]);
    return pair_or_status(st, k, v);
  });
}

// q, pool, scales, page_table, seq_lens, cu_seqlens, max_new, sm_scale, window, out, lse, workspace, dev_err
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<13>("attention", n, [&]() -> PyObject* {
    const Cache c = cache(a[1], a[2], a[3]);
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
      const kv4_status st = kv4_attention_gqa8_plan(c.B, max_new, t, hq, c.hkv, c.d, &ws_bytes);
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
        kv4_attention_gqa8(sq.p, sq.token, sq.head, dt, t, cu, max_new, c.pool, c.scales, c.pages, c.table, c.stride,
                           KV4_PAGE, lens, c.B, hq, c.hkv, c.d, window, static_cast<float>(scale),
                           out.mutable_data_ptr(), lse.mutable_data_ptr<float>(), ws, ws_bytes, err,
                           stream_of(c.dev));
    if (st == KV4_OK)
      for (const int i : {9, 10, 11, 12}) written(a[i]);
    return pair_or_status(st, out, lse);
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef methods[] = {{"append", fast(append), METH_FASTCALL, "kv4_append_gqa8"},
                         {"read", fast(read), METH_FASTCALL, "kv4_read_gqa8"},
                         {"attention", fast(attention), METH_FASTCALL, "kv4_attention_gqa8"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv4torch", "PyTorch side of the *_gqa8 entry points.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4torch() { return PyModule_Create(&module); }
