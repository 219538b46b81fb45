// The Python binding of the few-token entry points, as a compiled module.
//
// A call for one token spends 3 to 10 us on the GPU; checking its tensors and marshalling up to twenty
// arguments one attribute at a time from Python costs more than that (13 us for w8a8_w4_linear and 22 us for
// w8a8_kv_attention on a 298-token sequence, measured back to back, against 3 and 10 us of GPU time).  The
// functions here make the same checks with the same errors, allocate outputs and workspaces as torch tensors,
// and call the C entry points; they return the output, or a status that the Python side raises as W8A8Error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "w8a8.h"

namespace {

struct PythonError {};   // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw PythonError{};
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + ": expected a torch.Tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

void check_device(const at::Tensor& t, const char* name, int device) {
  if (!t.is_cuda()) fail(PyExc_ValueError, std::string(name) + ": must be a device tensor");
  if (t.get_device() != device)
    fail(PyExc_ValueError, std::string(name) + ": is on cuda:" + std::to_string(t.get_device()) +
                               ", but the current device is cuda:" + std::to_string(device));
}

void check_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, std::string(name) + ": expected " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
}

const at::Tensor& want(PyObject* o, at::ScalarType type, const char* name, int64_t dims, int device) {
  const at::Tensor& t = tensor(o, name);
  check_type(t, type, name);
  if (t.dim() != dims)
    fail(PyExc_ValueError, std::string(name) + ": expected " + std::to_string(dims) + " dims, got " + shape_text(t.sizes()));
  check_device(t, name, device);
  if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + ": must be contiguous");
  return t;
}

int64_t whole(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    fail(PyExc_TypeError, std::string(name) + ": expected a whole number");
  }
  return v;
}

at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, int device) {
  if (o == Py_None)
    return at::empty(shape, at::TensorOptions().dtype(at::kBFloat16).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
  const at::Tensor& t = want(o, at::kBFloat16, name, (int64_t)shape.size(), device);
  if (t.sizes() != shape) fail(PyExc_ValueError, std::string(name) + ": expected shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  return t;
}

hipStream_t stream_of(PyObject* o) { return reinterpret_cast<hipStream_t>(PyLong_AsVoidPtr(o)); }

uint16_t* bf16(const at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }

PyObject* result(w8a8_status st, const at::Tensor& y) {
  return st == W8A8_OK ? THPVariable_Wrap(y) : PyLong_FromLong(st);
}

// The C entry points take 16-byte aligned pointers; a table or lengths that begin elsewhere (table[1:], lens[1:])
// are copied, a few bytes per sequence, on the current stream.
at::Tensor aligned(const at::Tensor& t) { return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 ? t.clone() : t; }

// A cache with its page table and lengths.
struct Cache {
  const at::Tensor *k, *v, *ks, *vs;
  at::Tensor table, lens;
  int64_t pages, heads, page, dim, seqs, width;
  int device;

  Cache(PyObject* cache, PyObject* table_, PyObject* lens_) : device(c10::hip::current_device()) {
    if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 4) fail(PyExc_TypeError, "cache: expected a KVCache");
    k = &want(PyTuple_GET_ITEM(cache, 0), at::kChar, "cache.k_codes", 4, device);
    v = &want(PyTuple_GET_ITEM(cache, 1), at::kChar, "cache.v_codes", 4, device);
    ks = &want(PyTuple_GET_ITEM(cache, 2), at::kFloat, "cache.k_scale", 2, device);
    vs = &want(PyTuple_GET_ITEM(cache, 3), at::kFloat, "cache.v_scale", 2, device);
    table = aligned(want(table_, at::kInt, "table", 2, device));
    lens = aligned(want(lens_, at::kInt, "lens", 1, device));
    const auto shape = k->sizes();
    if (v->sizes() != shape || ks->sizes() != shape.slice(0, 2) || vs->sizes() != shape.slice(0, 2))
      fail(PyExc_ValueError, "the cache's tensors disagree on pages, heads, page or dim");
    if (table.size(0) != lens.size(0)) fail(PyExc_ValueError, "table and lens disagree on the number of sequences");
    pages = shape[0], heads = shape[1], page = shape[2], dim = shape[3];
    seqs = table.size(0), width = table.size(1);
  }
  int8_t* k_codes() const { return static_cast<int8_t*>(k->data_ptr()); }
  int8_t* v_codes() const { return static_cast<int8_t*>(v->data_ptr()); }
  float* k_scale() const { return static_cast<float*>(ks->data_ptr()); }
  float* v_scale() const { return static_cast<float*>(vs->data_ptr()); }
  const int32_t* table_ptr() const { return static_cast<const int32_t*>(table.data_ptr()); }
  const int32_t* lens_ptr() const { return static_cast<const int32_t*>(lens.data_ptr()); }
};

// bf16 [seqs, tokens, heads, dim] whose tokens are rows a fixed distance apart (a slice of a wider projection
// is fine), heads and dim dense within a row: that distance.
const at::Tensor& token_rows(PyObject* o, const char* name, const Cache& c, int64_t* ld) {
  const at::Tensor& t = tensor(o, name);
  check_type(t, at::kBFloat16, name);
  if (t.dim() != 4 || t.size(0) != c.seqs || t.size(3) != c.dim)
    fail(PyExc_ValueError, std::string(name) + ": expected [" + std::to_string(c.seqs) + ", tokens, heads, " +
                               std::to_string(c.dim) + "], got " + shape_text(t.sizes()));
  check_device(t, name, c.device);
  const auto s = t.strides();
  const int64_t tokens = t.size(1), heads = t.size(2);
  if (s[3] != 1 || (heads > 1 && s[2] != c.dim))
    fail(PyExc_ValueError, std::string(name) + ": heads and dim must be dense within a token's row");
  if (tokens > 1 && c.seqs > 1 && s[0] != tokens * s[1])
    fail(PyExc_ValueError, std::string(name) + ": tokens must be a fixed distance apart across sequences");
  *ld = tokens > 1 ? s[1] : c.seqs > 1 ? s[0] : heads * c.dim;
  return t;
}

bool expect(Py_ssize_t got, Py_ssize_t wanted) {
  if (got != wanted) PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return got == wanted;
}

// The caller's workspace of at least `need` bytes, or a new one if any is needed.
at::Tensor workspace(PyObject* o, size_t need, int device) {
  if (o == Py_None) {
    if (!need) return at::Tensor();
    return at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
  }
  const at::Tensor& t = tensor(o, "workspace");
  check_device(t, "workspace", device);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "workspace: must be contiguous");
  if (t.nbytes() < need)
    fail(PyExc_ValueError, "workspace: needs " + std::to_string(need) + " bytes, has " + std::to_string(t.nbytes()));
  return t;
}
void* ptr_of(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes_of(const at::Tensor& t) { return t.defined() ? t.nbytes() : 0; }

// (x, codes_packed, scales_packed, N, group, bias, workspace, out, stream)
PyObject* w4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!expect(n, 9)) return nullptr;
  try {
    const int device = c10::hip::current_device();
    const at::Tensor& x = want(a[0], at::kBFloat16, "x", 2, device);
    const at::Tensor& w = want(a[1], at::kByte, "codes_packed", 1, device);
    const at::Tensor& s = want(a[2], at::kBFloat16, "scales_packed", 1, device);
    const int64_t N = whole(a[3], "N"), group = whole(a[4], "group"), M = x.size(0), K = x.size(1);
    if (group != 32 && group != 64 && group != 128)
      fail(PyExc_ValueError, "group: expected 32, 64 or 128, got " + std::to_string(group));
    if (N < 0 || N > ((int64_t)1 << 30)) fail(PyExc_ValueError, "N: outside 0 .. 2^30");
    const int64_t rows = (N + 15) / 16 * 16;
    if (K > W8A8_MAX_K || w.numel() < rows * (K / 2) || s.numel() < rows * (K / group))
      fail(PyExc_ValueError, "packed weight is smaller than [N, K] needs");
    uint16_t* bias = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& b = want(a[5], at::kBFloat16, "bias", 1, device);
      if (b.size(0) != N) fail(PyExc_ValueError, "bias length must equal N");
      bias = bf16(b);
    }
    const at::Tensor ws = workspace(a[6], w8a8_w4_workspace_bytes(M, N, K), device);
    const at::Tensor y = output(a[7], "out", {M, N}, device);
    w8a8_status st;
    Py_BEGIN_ALLOW_THREADS
    st = w8a8_w4_linear(bf16(x), static_cast<const uint8_t*>(w.data_ptr()), bf16(s), bias, bf16(y), M, N, K, (int)group, ptr_of(ws),
                        bytes_of(ws), stream_of(a[8]));
    Py_END_ALLOW_THREADS
    return result(st, y);
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (k, v, cache, table, lens, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!expect(n, 6)) return nullptr;
  try {
    const Cache c(a[2], a[3], a[4]);
    int64_t ldk, ldv;
    const at::Tensor &k = token_rows(a[0], "k", c, &ldk), &v = token_rows(a[1], "v", c, &ldv);
    if (k.sizes() != v.sizes() || k.size(2) != c.heads)
      fail(PyExc_ValueError, "k, v and the cache disagree on tokens or heads");
    w8a8_status st;
    Py_BEGIN_ALLOW_THREADS
    st = w8a8_kv_append(bf16(k), ldk, bf16(v), ldv, c.k_codes(), c.k_scale(), c.v_codes(), c.v_scale(), c.pages, c.table_ptr(),
                        c.width, c.lens_ptr(), c.seqs, k.size(1), c.heads, c.dim, c.page, stream_of(a[5]));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (cache, table, lens, length, k_out, v_out, stream) -> (k, v)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!expect(n, 7)) return nullptr;
  try {
    const Cache c(a[0], a[1], a[2]);
    const int64_t length = whole(a[3], "length");
    if (length < 0) fail(PyExc_ValueError, "length: must not be negative");
    const at::Tensor k = output(a[4], "k", {c.seqs, length, c.heads, c.dim}, c.device);
    const at::Tensor v = output(a[5], "v", {c.seqs, length, c.heads, c.dim}, c.device);
    w8a8_status st;
    Py_BEGIN_ALLOW_THREADS
    st = w8a8_kv_read(c.k_codes(), c.k_scale(), c.v_codes(), c.v_scale(), c.pages, c.table_ptr(), c.width, c.lens_ptr(), c.seqs,
                      length, c.heads, c.dim, c.page, bf16(k), bf16(v), stream_of(a[6]));
    Py_END_ALLOW_THREADS
    if (st != W8A8_OK) return PyLong_FromLong(st);
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(v));
    return both;
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (q, cache, table, lens, scale, workspace, out, stream)
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!expect(n, 8)) return nullptr;
  try {
    const Cache c(a[1], a[2], a[3]);
    int64_t ldq;
    const at::Tensor& q = token_rows(a[0], "q", c, &ldq);
    const int64_t tokens = q.size(1), q_heads = q.size(2);
    double scale = 1.0 / std::sqrt((double)c.dim);
    if (a[4] != Py_None) {
      scale = PyFloat_AsDouble(a[4]);
      if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    const size_t need = w8a8_kv_attention_workspace_bytes(c.seqs, tokens, q_heads, c.heads, c.dim, c.page, c.width);
    const at::Tensor ws = workspace(a[5], need, c.device);
    const at::Tensor y = output(a[6], "out", {c.seqs, tokens, q_heads, c.dim}, c.device);
    w8a8_status st;
    Py_BEGIN_ALLOW_THREADS
    st = w8a8_kv_attention(bf16(q), ldq, c.k_codes(), c.k_scale(), c.v_codes(), c.v_scale(), c.pages, c.table_ptr(), c.width,
                           c.lens_ptr(), c.seqs, tokens, q_heads, c.heads, c.dim, c.page, (float)scale, bf16(y),
                           ptr_of(ws), bytes_of(ws), stream_of(a[7]));
    Py_END_ALLOW_THREADS
    return result(st, y);
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(w4_linear), ENTRY(kv_append), ENTRY(kv_read), ENTRY(kv_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
