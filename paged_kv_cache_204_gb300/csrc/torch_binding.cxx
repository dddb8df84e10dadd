// Python extension: the bounded-cache entry points of pkv.h called with torch
// tensors. Argument checks and marshalling only. A call from Python spends about
// as long on reading ten tensors' attributes, one by one, as the smallest of these
// operators on the GPU (15 us against 7); here that is about 1 us.
//
// Every function takes its arguments by position, raises ValueError for a tensor
// of the wrong type, shape, layout or device, and returns the pkv_status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "pkv.h"

namespace {

struct PyError {};  // a Python exception is already set

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": need a tensor");
  return THPVariable_Unpack(o);
}

[[noreturn]] void refuse_tensor(const at::Tensor& t, const char* name, const char* need) {
  std::ostringstream s;
  s << name << ": need " << need << ", got " << t.dtype().name() << " " << t.sizes() << " on " << t.device()
    << (t.is_contiguous() ? "" : ", not contiguous");
  refuse(s.str());
}

// A contiguous tensor of the given type and shape on the pools' device.
void* want(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device dev,
           const char* need) {
  if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous())
    refuse_tensor(t, name, need);
  return t.data_ptr();
}

int as_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit in 32 bits");
  return (int)v;
}

float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError();
  return (float)v;
}

pkv_dtype code_of(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kFloat: return PKV_F32;
    case at::kHalf: return PKV_F16;
    case at::kBFloat16: return PKV_BF16;
    case at::kByte: return PKV_FP8_E4M3;
    default: refuse(std::string(name) + ": not a type of this library");
  }
}

// The pools, block tables and lengths, which every operator takes.
struct Cache {
  const at::Tensor &k, &v, &tables;
  at::Device dev;
  int nb, Hkv, bs, D, B, MB;
  const int32_t* lens;

  Cache(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo)
      : k(tensor(ko, "k_cache")), v(tensor(vo, "v_cache")), tables(tensor(to, "block_tables")), dev(k.device()) {
    if (!dev.is_cuda()) refuse("k_cache: need a CUDA tensor");
    if (k.dim() != 4 || !k.is_contiguous())
      refuse_tensor(k, "k_cache", "a contiguous [num_blocks, Hkv, block_size, D] tensor");
    want(v, "v_cache", k.scalar_type(), k.sizes(), dev, "a tensor like k_cache");
    if (tables.dim() != 2) refuse_tensor(tables, "block_tables", "int32 [num_seqs, max_blocks_per_seq]");
    nb = size(k, 0), Hkv = size(k, 1), bs = size(k, 2), D = size(k, 3);
    B = size(tables, 0), MB = size(tables, 1);
    want(tables, "block_tables", at::kInt, tables.sizes(), dev, "contiguous int32 [num_seqs, max_blocks_per_seq]");
    lens = static_cast<const int32_t*>(lengths(lo, "context_lens"));
  }
  static int size(const at::Tensor& t, int d) {
    if (t.size(d) > INT32_MAX) refuse("a dimension does not fit in 32 bits");
    return (int)t.size(d);
  }
  void* lengths(PyObject* o, const char* name) const {
    return want(tensor(o, name), name, at::kInt, {B}, dev, "contiguous int32 [num_seqs] on the pools' device");
  }
  const int32_t* table() const { return tables.data_ptr<int32_t>(); }
  // q and out: [rows, H, D] of the pools' type; rows < 0: any number
  int queries(PyObject* qo, PyObject* oo, int64_t rows, const void** q, void** out) const {
    const at::Tensor &qt = tensor(qo, "q"), &ot = tensor(oo, "out");
    if (qt.dim() != 3) refuse_tensor(qt, "q", "[rows, num_heads, head_dim]");
    const char* need = "a contiguous [rows, num_heads, head_dim] tensor of the pools' type on their device";
    *q = want(qt, "q", k.scalar_type(), {rows < 0 ? qt.size(0) : rows, qt.size(1), D}, dev, need);
    *out = want(ot, "out", k.scalar_type(), qt.sizes(), dev, need);
    return size(qt, 1);
  }
  float* scores(PyObject* o, const char* name, int64_t* stride) const {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 3) refuse_tensor(t, name, "float32 [num_seqs, Hkv, n]");
    *stride = t.size(2);
    return static_cast<float*>(want(t, name, at::kFloat, {B, Hkv, t.size(2)}, dev,
                                    "contiguous float32 [num_seqs, Hkv, n] on the pools' device"));
  }
  void* workspace(PyObject* o, size_t* bytes) const {
    const at::Tensor& t = tensor(o, "workspace");
    if (t.device() != dev || !t.is_contiguous()) refuse_tensor(t, "workspace", "a contiguous tensor on the pools' device");
    *bytes = t.nbytes();
    return t.data_ptr();
  }
  int32_t* error_word(PyObject* o) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, "dev_err");
    if (t.scalar_type() != at::kInt || t.numel() < 1 || t.device() != dev)
      refuse_tensor(t, "dev_err", "an int32 tensor on the pools' device");
    return t.data_ptr<int32_t>();
  }
  // `o`: None (the device's current stream) or a torch stream
  pkv_stream_t stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    PyObject* a = PyObject_GetAttrString(o, "cuda_stream");
    if (a == nullptr) throw PyError();
    void* s = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    if (s == nullptr && PyErr_Occurred()) throw PyError();
    return static_cast<pkv_stream_t>(s);
  }
};

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t expected, F f) {
  try {
    if (got != expected) refuse("wrong number of arguments");
    return PyLong_FromLong(f());
  } catch (const PyError&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// out, q, k_cache, v_cache, block_tables, context_lens, scale, window, num_sinks,
// max_context_len, workspace, dev_err, stream
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Cache c(a[2], a[3], a[4], a[5]);
    const void* q;
    void* out;
    size_t bytes;
    const int H = c.queries(a[1], a[0], c.B, &q, &out);
    void* ws = c.workspace(a[10], &bytes);
    const float scale = as_float(a[6]);
    const int window = as_int(a[7], "window"), sinks = as_int(a[8], "num_sinks");
    const int longest = as_int(a[9], "max_context_len");
    int32_t* err = c.error_word(a[11]);
    const c10::cuda::CUDAGuard guard(c.dev);
    return pkv_paged_attention_decode_window(out, q, c.k.data_ptr(), c.v.data_ptr(), c.table(), c.lens, scale, window,
                                             sinks, H, c.Hkv, c.D, c.bs, c.B, c.MB, c.nb, longest,
                                             code_of(c.k.scalar_type(), "k_cache"), ws, bytes, err, c.stream(a[12]));
  });
}

// out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, window,
// num_sinks, max_query_len, dev_err, stream
PyObject* prefill_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Cache c(a[2], a[3], a[4], a[5]);
    const void* q;
    void* out;
    const int H = c.queries(a[1], a[0], -1, &q, &out);
    const void* start = want(tensor(a[6], "query_start"), "query_start", at::kInt, {c.B + 1}, c.dev,
                             "contiguous int32 [num_seqs + 1] on the pools' device");
    const float scale = as_float(a[7]);
    const int window = as_int(a[8], "window"), sinks = as_int(a[9], "num_sinks");
    const int longest = as_int(a[10], "max_query_len");
    int32_t* err = c.error_word(a[11]);
    const c10::cuda::CUDAGuard guard(c.dev);
    return pkv_paged_attention_prefill_window(out, q, c.k.data_ptr(), c.v.data_ptr(), c.table(), c.lens,
                                              static_cast<const int32_t*>(start), scale, window, sinks, H, c.Hkv, c.D,
                                              c.bs, c.B, c.MB, c.nb, longest,
                                              code_of(c.k.scalar_type(), "k_cache"), err, c.stream(a[12]));
  });
}

// out, scores_out, q, k_cache, v_cache, block_tables, context_lens, scale,
// max_context_len, workspace, scores, dev_err, stream
PyObject* decode_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Cache c(a[3], a[4], a[5], a[6]);
    const void* q;
    void* out;
    size_t bytes;
    int64_t stride, stride_in;
    const int H = c.queries(a[2], a[0], c.B, &q, &out);
    float* to = c.scores(a[1], "scores_out", &stride);
    const float* from = nullptr;
    if (a[10] != Py_None) {
      from = c.scores(a[10], "scores", &stride_in);
      if (stride_in != stride) refuse_tensor(tensor(a[10], "scores"), "scores", "the shape of scores_out");
    }
    void* ws = c.workspace(a[9], &bytes);
    const float scale = as_float(a[7]);
    const int longest = as_int(a[8], "max_context_len");
    int32_t* err = c.error_word(a[11]);
    const c10::cuda::CUDAGuard guard(c.dev);
    return pkv_paged_attention_decode_scores(out, to, from, stride, q, c.k.data_ptr(), c.v.data_ptr(), c.table(),
                                             c.lens, scale, H, c.Hkv, c.D, c.bs, c.B, c.MB, c.nb, longest,
                                             code_of(c.k.scalar_type(), "k_cache"), ws, bytes, err, c.stream(a[12]));
  });
}

// k_cache, v_cache, scores, scores_out, block_tables, dst_block_tables, context_lens,
// new_context_lens, kept, num_sinks, num_recent, max_context_len, head_dim (None: the
// pools' last dimension), dev_err, stream
PyObject* evict_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const Cache c(a[0], a[1], a[4], a[6]);
    int64_t s_in, s_out;
    const float* from = c.scores(a[2], "scores", &s_in);
    float* to = c.scores(a[3], "scores_out", &s_out);
    const at::Tensor &dst = tensor(a[5], "dst_block_tables"), &kt = tensor(a[8], "kept");
    want(dst, "dst_block_tables", at::kInt, c.tables.sizes(), c.dev, "an int32 tensor like block_tables");
    void* lens = c.lengths(a[7], "new_context_lens");
    if (kt.dim() != 3) refuse_tensor(kt, "kept", "int32 [num_seqs, Hkv, budget]");
    void* kept = want(kt, "kept", at::kInt, {c.B, c.Hkv, kt.size(2)}, c.dev,
                      "contiguous int32 [num_seqs, Hkv, budget] on the pools' device");
    const int budget = Cache::size(kt, 2);
    const int sinks = as_int(a[9], "num_sinks"), recent = as_int(a[10], "num_recent");
    const int longest = as_int(a[11], "max_context_len");
    pkv_dtype code = code_of(c.k.scalar_type(), "k_cache");
    int D = c.D;
    if (a[12] != Py_None) {
      D = as_int(a[12], "head_dim");
      if (D != c.D) {  // a pool of q4_0 rows: 9 head_dim / 16 bytes
        if (code != PKV_FP8_E4M3 || D <= 0 || D / 16 * 9 != c.D) refuse("the pools' rows are no rows of this head_dim");
        code = PKV_Q4_0;
      }
    }
    int32_t* err = c.error_word(a[13]);
    const c10::cuda::CUDAGuard guard(c.dev);
    return pkv_evict_tokens(c.k.data_ptr(), c.v.data_ptr(), from, s_in, to, s_out, c.table(), dst.data_ptr<int32_t>(),
                            c.lens, static_cast<int32_t*>(lens), static_cast<int32_t*>(kept), budget, sinks, recent,
                            c.Hkv, D, c.bs, c.B, c.MB, c.nb, longest, code, err, c.stream(a[14]));
  });
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(decode_window), ENTRY(prefill_window), ENTRY(decode_scores), ENTRY(evict_tokens),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_torch", "Bounded-cache calls with torch tensors", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&module); }
