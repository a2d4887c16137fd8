// CPython module _serving: argument marshalling of the serving calls, which run many times per token.
// A decode step's kernels take 3 to 10 us, and reading the arguments' tensors from Python and passing
// two dozen of them through ctypes took 8 to 14 us a call.  Every function takes the positional
// arguments of the batq.py function of its name (with the stream as None or an integer), checks them,
// calls the C ABI and returns its status; what does not fit raises ValueError or TypeError.  A call without
// rows (a layer whose router sent it none, a step without new tokens) has nothing to do and is not passed on.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "../../include/batq.h"

namespace {

// A Python error to raise: ValueError, or TypeError.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

std::string describe(const at::Tensor& t) {
  std::ostringstream s;
  s << t.scalar_type() << " " << t.sizes() << " on " << t.device();
  return s.str();
}

struct Call {
  int dev;
  void* stream;
  // (the first tensor decides whether there is a device to ask)
  Call(PyObject* stream_arg, PyObject* first, const char* name) {
    if (!THPVariable_Check(first) || !THPVariable_Unpack(first).is_cuda())
      throw Refused{PyExc_TypeError, std::string(name) + " must be a CUDA tensor (libbatq has no CPU path)"};
    dev = c10::cuda::current_device();
    if (stream_arg == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    } else {
      stream = PyLong_AsVoidPtr(stream_arg);
      if (PyErr_Occurred()) throw Refused{nullptr, ""};
    }
  }

  const at::Tensor& tensor(PyObject* o, const char* name) const {
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a CUDA tensor"};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev)
      refuse(std::string(name) + " must be on the current device, cuda:" + std::to_string(dev) + ", got " + describe(t));
    return t;
  }

  // A contiguous tensor of `type` with `numel` elements at least; None gives a null pointer where it may.
  template <class P>
  P* array(PyObject* o, at::ScalarType type, const char* name, int64_t numel = 0, bool optional = false) const {
    if (optional && o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_contiguous() || t.numel() < numel) {
      std::ostringstream s;
      s << name << " must be a contiguous " << type << " tensor of at least " << numel << " elements, got " << describe(t);
      refuse(s.str());
    }
    return static_cast<P*>(t.data_ptr());
  }
  uint8_t* bytes(PyObject* o, const char* name, int64_t numel = 0) const {
    return array<uint8_t>(o, at::kByte, name, numel);
  }
  int* ints(PyObject* o, const char* name, bool optional = false) const {
    return array<int>(o, at::kInt, name, 0, optional);
  }
  float* floats(PyObject* o, const char* name, int64_t numel, bool optional = false) const {
    return array<float>(o, at::kFloat, name, numel, optional);
  }
};

int integer(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  if (v != static_cast<int>(v)) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}
int size32(int64_t v, const char* name) {
  if (v != static_cast<int>(v)) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

// A bf16 or fp32 matrix whose rows hold `cols` consecutive elements.
struct Matrix {
  void* p;
  batq_dtype type;
  int rows, ld;
};
Matrix matrix(const Call& c, PyObject* o, int64_t cols, const char* name) {
  const at::Tensor& t = c.tensor(o, name);
  const bool bf16 = t.scalar_type() == at::kBFloat16;
  if ((!bf16 && t.scalar_type() != at::kFloat) || t.dim() != 2 || t.size(1) != cols || t.stride(1) != 1)
    refuse(std::string(name) + " must be a bf16 or fp32 matrix of rows of " + std::to_string(cols) +
           " consecutive elements, got " + describe(t));
  const int64_t ld = t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.stride(0), cols);
  return Matrix{t.data_ptr(), bf16 ? BATQ_BF16 : BATQ_F32, size32(t.size(0), name), size32(ld, name)};
}
int64_t columns(const Call& c, PyObject* o, const char* name) {
  const at::Tensor& t = c.tensor(o, name);
  if (t.dim() != 2) refuse(std::string(name) + " must be a matrix, got " + describe(t));
  return t.size(1);
}

// 64 host floats (a contiguous fp32 array).  False: it is something else, and the caller converts it.
struct HostFloats {
  Py_buffer view = {};
  bool held = false;
  bool get(PyObject* o, Py_ssize_t count) {
    if (PyObject_GetBuffer(o, &view, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) != 0) {
      PyErr_Clear();
      return false;
    }
    held = true;
    return view.format && std::string(view.format) == "f" && view.len == count * 4;
  }
  const float* data() const { return static_cast<const float*>(view.buf); }
  ~HostFloats() {
    if (held) PyBuffer_Release(&view);
  }
};

// Without the interpreter's lock: a launch may wait (for a full queue, for its module to load), and a host function
// queued ahead of it may need the lock.
class Unlocked {
  PyThreadState* const state_ = PyEval_SaveThread();

 public:
  ~Unlocked() { PyEval_RestoreThread(state_); }
};
template <class F, class... Args>
int call(F f, Args... args) {
  const Unlocked unlocked;
  return f(args...);
}

int64_t mma_scale_bytes(int64_t M, int64_t columns) { return (M + 127) / 128 * 128 * ((columns + 3) / 4 * 4); }

// The arrays of a ragged batch.
struct Batch {
  int *cu, *lens, *table;
  int count, max_pages;
};
Batch batch(const Call& c, PyObject* cu, PyObject* lens, PyObject* table, int64_t rows, const char* cu_name) {
  Batch b;
  const at::Tensor& t = c.tensor(table, "page_table");
  const at::Tensor& l = c.tensor(lens, "seq_lens");
  b.cu = c.ints(cu, cu_name, true);
  b.lens = c.ints(lens, "seq_lens");
  b.table = c.ints(table, "page_table");
  b.count = size32(l.numel(), "batch");
  if (t.dim() != 2 || t.size(0) != b.count) refuse("page_table must be batch x max_pages");
  b.max_pages = size32(t.size(1), "max_pages");
  if (b.cu ? THPVariable_Unpack(cu).numel() != (int64_t)b.count + 1 : rows < b.count)
    refuse(std::string(cu_name) + " must hold batch + 1 entries (without it there must be a row for each sequence)");
  return b;
}

// The four tensors of an 8-bit paged cache.
struct Cache {
  uint8_t *k, *ks, *v, *vs;
  int pages, heads, page, dim;
};
Cache cache(const Call& c, PyObject* k, PyObject* ks, PyObject* v, PyObject* vs) {
  Cache r;
  const at::Tensor& kt = c.tensor(k, "k_codes");
  const at::Tensor& vt = c.tensor(v, "v_codes");
  if (kt.dim() != 4 || vt.sizes() != kt.sizes())
    refuse("cache codes must be num_pages x kv_heads x page_size x head_dim, the same for K and V");
  r.pages = size32(kt.size(0), "num_pages");
  r.heads = size32(kt.size(1), "kv_heads");
  r.page = size32(kt.size(2), "page_size");
  r.dim = size32(kt.size(3), "head_dim");
  for (PyObject* o : {ks, vs}) {
    const at::Tensor& s = c.tensor(o, "scales");
    if (s.dim() != 2 || s.size(0) != r.pages || s.size(1) != r.heads)
      refuse("k_scales and v_scales must be num_pages x kv_heads");
  }
  r.k = c.bytes(k, "k_codes");
  r.ks = c.bytes(ks, "k_scales");
  r.v = c.bytes(v, "v_codes");
  r.vs = c.bytes(vs, "v_scales");
  return r;
}

// A contiguous device buffer of any type.
std::pair<void*, size_t> buffer(const Call& c, PyObject* o, const char* name) {
  const at::Tensor& t = c.tensor(o, name);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return {t.data_ptr(), t.nbytes()};
}

constexpr int kConvert = -1;  // returned instead of a status: A has to be made a contiguous fp32 array first

// X, A, B, w_codes, w_scales, M, out, w_gs, w_format, stream
int linear_w4a16(PyObject* const* a) {
  const Call c(a[9], a[0], "X");
  const int M = integer(a[5], "M"), format = integer(a[8], "w_format");
  const int64_t N = columns(c, a[0], "X");
  const Matrix x = matrix(c, a[0], N, "X"), o = matrix(c, a[6], M, "out");
  if (o.rows != x.rows) refuse("out must have a row for each row of X");
  if (x.rows == 0) return BATQ_OK;
  HostFloats A;
  if (a[1] != Py_None && !A.get(a[1], 64)) return kConvert;
  return call(batq_linear_w4a16, x.p, x.type, x.rows, size32(N, "N"), x.ld, A.held ? A.data() : nullptr,
              c.floats(a[2], "B", N / 32 * 16, true), static_cast<batq_w4_format>(format),
              c.bytes(a[3], "w_codes", (int64_t)M * N / 2),
              c.bytes(a[4], "w_scales", mma_scale_bytes(M, N / (format == BATQ_W4_NVFP4 ? 16 : 32))),
              c.floats(a[7], "w_gs", 1, true), M, o.type, o.p, o.ld, c.stream);
}

// K, V, cu_new, seq_lens, page_table, k_codes, k_scales, v_codes, v_scales, stream
int kv8_append(PyObject* const* a) {
  const Call c(a[9], a[0], "K");
  const Cache m = cache(c, a[5], a[6], a[7], a[8]);
  const int64_t row = (int64_t)m.heads * m.dim;
  const Matrix k = matrix(c, a[0], row, "K"), v = matrix(c, a[1], row, "V");
  if (k.type != v.type || k.rows != v.rows) refuse("K and V must have the same shape and type");
  const Batch b = batch(c, a[2], a[3], a[4], k.rows, "cu_new");
  if (k.rows == 0) return BATQ_OK;
  return call(batq_kv8_append, k.p, v.p, k.type, k.rows, m.heads, m.dim, k.ld, v.ld, b.cu, b.lens, b.table, b.count,
              b.max_pages, m.pages, m.page, m.k, m.ks, m.v, m.vs, c.stream);
}

// Q, cu_q, seq_lens, page_table, k_codes, k_scales, v_codes, v_scales, softmax_scale, max_q_len, workspace, out, lse, stream
int attn_kv8(PyObject* const* a) {
  const Call c(a[13], a[0], "Q");
  const Cache m = cache(c, a[4], a[5], a[6], a[7]);
  const int64_t row = columns(c, a[0], "Q");
  const Matrix q = matrix(c, a[0], row, "Q"), o = matrix(c, a[11], row, "out");
  if (o.rows != q.rows || m.dim < 1 || row % m.dim != 0) refuse("Q and out must be T x q_heads * head_dim");
  const int heads = size32(row / m.dim, "q_heads");
  const Batch b = batch(c, a[1], a[2], a[3], q.rows, "cu_q");
  if (q.rows == 0) return BATQ_OK;
  const double scale = PyFloat_AsDouble(a[8]);
  if (scale == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  const auto ws = buffer(c, a[10], "workspace");
  if (a[12] != Py_None) {
    const at::Tensor& l = c.tensor(a[12], "lse");
    if (l.dim() != 2 || l.size(0) != q.rows || l.size(1) != heads) refuse("lse must be T x q_heads");
  }
  return call(batq_attn_kv8, q.p, q.type, q.rows, q.ld, heads, m.heads, m.dim, b.cu, b.lens, b.table, b.count, b.max_pages,
              m.pages, m.page, m.k, m.ks, m.v, m.vs, static_cast<float>(scale), integer(a[9], "max_q_len"),
              ws.first, ws.second, o.type, o.p, o.ld, c.floats(a[12], "lse", 0, true), c.stream);
}

// a_codes, a_scales, w_codes, w_scales, expert_offsets, M, N, out, stream
int gemm_mxfp4_experts(PyObject* const* a) {
  const Call c(a[8], a[0], "a_codes");
  const int M = integer(a[5], "M"), N = integer(a[6], "N");
  const int E = size32(c.tensor(a[4], "expert_offsets").numel() - 1, "experts");
  const Matrix o = matrix(c, a[7], M, "out");
  if (o.rows == 0) return BATQ_OK;
  return call(batq_gemm_mxfp4_experts, c.bytes(a[0], "a_codes", (int64_t)o.rows * N / 2),
              c.bytes(a[1], "a_scales", (int64_t)o.rows * (N / 32)),
              c.bytes(a[2], "w_codes", (int64_t)E * M * N / 2),
              c.bytes(a[3], "w_scales", E * mma_scale_bytes(M, N / 32)),
              c.ints(a[4], "expert_offsets"), E, o.rows, M, N, o.type, o.p, o.ld, c.stream);
}

// X, A, B, ratios, w_codes, w_scales, expert_offsets, M, workspace, out, stream
int linear_experts(PyObject* const* a) {
  const Call c(a[10], a[0], "X");
  const int M = integer(a[7], "M");
  const int64_t N = columns(c, a[0], "X");
  const int E = size32(c.tensor(a[6], "expert_offsets").numel() - 1, "experts");
  const Matrix x = matrix(c, a[0], N, "X"), o = matrix(c, a[9], M, "out");
  if (o.rows != x.rows) refuse("out must have a row for each row of X");
  if (x.rows == 0) return BATQ_OK;
  HostFloats A;
  if (!A.get(a[1], 64)) return kConvert;
  const auto ws = buffer(c, a[8], "workspace");
  return call(batq_linear_experts, x.p, x.type, x.rows, size32(N, "N"), x.ld, A.data(), c.floats(a[2], "B", N / 32 * 16),
              c.floats(a[3], "ratios", N / 32 * 2, true), c.bytes(a[4], "w_codes", (int64_t)E * M * N / 2),
              c.bytes(a[5], "w_scales", E * mma_scale_bytes(M, N / 32)),
              c.ints(a[6], "expert_offsets"), E, M, ws.first, ws.second, o.type, o.p, o.ld, c.stream);
}

template <int (*kF)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", kArgs, n);
  try {
    return PyLong_FromLong(kF(args));
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());  // otherwise Python has the error already
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define BATQ_ENTRY(name, count) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, count>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {BATQ_ENTRY(linear_w4a16, 10), BATQ_ENTRY(kv8_append, 10), BATQ_ENTRY(attn_kv8, 14),
                         BATQ_ENTRY(gemm_mxfp4_experts, 9), BATQ_ENTRY(linear_experts, 11), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module_def); }
