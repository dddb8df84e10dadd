// Python extension: the bounded-cache entry points of pkv.h, the rotating cache
// writes and prefill over quantised caches, called with torch tensors. Argument
// checks and marshalling only. A call from Python spends about as long on reading
// ten tensors' attributes, one by one, as the smallest of these operators on the
// GPU (15 us against 7); here that is about 1 us.
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

// The two pools, which every operator takes.
struct Pools {
  const at::Tensor &k, &v;
  at::Device dev;
  int nb, Hkv, bs, D;

  Pools(PyObject* ko, PyObject* vo) : k(tensor(ko, "k_cache")), v(tensor(vo, "v_cache")), dev(k.device()) {
    if (!dev.is_cuda()) refuse("k_cache: need a CUDA tensor");
    if (k.dim() != 4 || !k.is_contiguous())
      refuse_tensor(k, "k_cache", "a contiguous [num_blocks, Hkv, block_size, D] tensor");
    want(v, "v_cache", k.scalar_type(), k.sizes(), dev, "a tensor like k_cache");
    nb = size(k, 0), Hkv = size(k, 1), bs = size(k, 2), D = size(k, 3);
  }
  static int size(const at::Tensor& t, int d) {
    if (t.size(d) > INT32_MAX) refuse("a dimension does not fit in 32 bits");
    return (int)t.size(d);
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

// The pools, block tables and lengths of the attention operators.
struct Cache : Pools {
  const at::Tensor& tables;
  int B, MB;
  const int32_t* lens;

  Cache(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo) : Pools(ko, vo), tables(tensor(to, "block_tables")) {
    if (tables.dim() != 2) refuse_tensor(tables, "block_tables", "int32 [num_seqs, max_blocks_per_seq]");
    B = size(tables, 0), MB = size(tables, 1);
    want(tables, "block_tables", at::kInt, tables.sizes(), dev, "contiguous int32 [num_seqs, max_blocks_per_seq]");
    lens = static_cast<const int32_t*>(lengths(lo, "context_lens"));
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

// A step's rows [tokens, heads, head_dim], each token's together; *stride: from token to token.
void* step_rows(const at::Tensor& t, const char* name, at::ScalarType type, int64_t tokens, int64_t D, at::Device dev,
                int64_t* stride) {
  if (t.dim() != 3 || t.scalar_type() != type || t.size(0) != tokens || t.size(2) != D || t.device() != dev ||
      (t.numel() > 0 && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != D))))
    refuse_tensor(t, name, "[tokens, heads, head_dim], a token's rows together, on the pools' device");
  *stride = t.stride(0);
  return t.data_ptr();
}

// q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, kind (0: caches of q's type,
// 1: e4m3, 2: q4_0), k_scale, v_scale, pair_axis (None or bytes), interleaved, dev_err, stream
PyObject* rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const Pools c(a[4], a[5]);
    const at::Tensor &qt = tensor(a[1], "q"), &kt = tensor(a[2], "k"), &vt = tensor(a[3], "v");
    const at::Tensor &ot = tensor(a[0], "q_out"), &st = tensor(a[6], "slot_mapping"), &pt = tensor(a[7], "positions");
    const at::Tensor& ct = tensor(a[8], "cos_sin");
    const int kind = as_int(a[9], "kind");
    if (qt.dim() != 3) refuse_tensor(qt, "q", "[tokens, num_heads, head_dim]");
    const int T = Pools::size(qt, 0), H = Pools::size(qt, 1), D = Pools::size(qt, 2);
    const at::ScalarType type = qt.scalar_type();
    const pkv_dtype code = code_of(type, "q");
    if (c.k.scalar_type() != (kind == 0 ? type : at::kByte) || c.D != (kind == 2 ? D / 16 * 9 : D))
      refuse_tensor(c.k, "k_cache", kind == 0 ? "rows of q's type" : kind == 1 ? "e4m3 rows of head_dim bytes" : "q4_0 rows of 9 head_dim / 16 bytes");
    int64_t so, sq, sk, sv;
    void* out = step_rows(ot, "q_out", type, T, D, c.dev, &so);
    if (ot.size(1) != H) refuse_tensor(ot, "q_out", "a tensor of q's shape");
    const void* q = step_rows(qt, "q", type, T, D, c.dev, &sq);
    const void* k = step_rows(kt, "k", type, T, D, c.dev, &sk);
    const void* v = step_rows(vt, "v", type, T, D, c.dev, &sv);
    if (kt.size(1) != c.Hkv || vt.size(1) != c.Hkv) refuse("k, v: need the pools' number of kv heads");
    const void* slots = want(st, "slot_mapping", at::kLong, {T}, c.dev, "contiguous int64 [tokens] on the pools' device");
    if (pt.dim() != 1 && pt.dim() != 2) refuse_tensor(pt, "positions", "int32 [tokens] or [axes, tokens]");
    const int axes = pt.dim() == 2 ? Pools::size(pt, 0) : 1;
    const char* need = "contiguous int32 [tokens] or [axes, tokens] on the pools' device";
    const void* positions = pt.dim() == 2 ? want(pt, "positions", at::kInt, {axes, T}, c.dev, need)
                                          : want(pt, "positions", at::kInt, {T}, c.dev, need);
    if (ct.dim() != 2) refuse_tensor(ct, "cos_sin", "float32 [max_position, rotary_dim]");
    const void* table = want(ct, "cos_sin", at::kFloat, ct.sizes(), c.dev,
                             "contiguous float32 [max_position, rotary_dim] on the pools' device");
    const int most = Pools::size(ct, 0), R = Pools::size(ct, 1);
    const float k_scale = as_float(a[10]), v_scale = as_float(a[11]);
    const uint8_t* axis = nullptr;
    if (a[12] != Py_None) {
      if (!PyBytes_Check(a[12]) || PyBytes_GET_SIZE(a[12]) != R / 2) refuse("pair_axis: need bytes, one of each pair");
      axis = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[12]));
    }
    const int interleaved = PyObject_IsTrue(a[13]);
    if (interleaved < 0) throw PyError();
    int32_t* err = c.error_word(a[14]);
    const c10::cuda::CUDAGuard guard(c.dev);
    const pkv_stream_t stream = c.stream(a[15]);
    const auto slot_ids = static_cast<const int64_t*>(slots);
    const auto at_positions = static_cast<const int32_t*>(positions);
    const auto cos_sin = static_cast<const float*>(table);
    void *kc = c.k.data_ptr(), *vc = c.v.data_ptr();
    if (kind == 1)
      return pkv_rope_and_cache_fp8(out, so, q, sq, k, sk, v, sv, kc, vc, slot_ids, at_positions, cos_sin, most, R,
                                    axis, axes, interleaved, T, H, c.Hkv, D, c.bs, c.nb, code, k_scale, v_scale, err,
                                    stream);
    return (kind == 2 ? pkv_rope_and_cache_q4_0 : pkv_rope_and_cache)(out, so, q, sq, k, sk, v, sv, kc, vc, slot_ids,
                                                                      at_positions, cos_sin, most, R, axis, axes,
                                                                      interleaved, T, H, c.Hkv, D, c.bs, c.nb, code,
                                                                      err, stream);
  });
}

// out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, k_scale and
// v_scale (both None: q4_0 pools), max_query_len, workspace, dev_err, stream
PyObject* prefill_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const Cache c(a[2], a[3], a[4], a[5]);
    const bool q4 = a[8] == Py_None;
    const at::Tensor &qt = tensor(a[1], "q"), &ot = tensor(a[0], "out");
    if (qt.dim() != 3) refuse_tensor(qt, "q", "[rows, num_heads, head_dim]");
    if (c.k.scalar_type() != at::kByte) refuse_tensor(c.k, "k_cache", "a uint8 pool");
    const char* need = "a contiguous [rows, num_heads, head_dim] tensor on the pools' device, out of q's type";
    const void* q = want(qt, "q", qt.scalar_type(), qt.sizes(), c.dev, need);
    void* out = want(ot, "out", qt.scalar_type(), qt.sizes(), c.dev, need);
    const char *q0 = static_cast<const char*>(q), *o0 = static_cast<const char*>(out);
    if (qt.nbytes() > 0 && q0 < o0 + ot.nbytes() && o0 < q0 + qt.nbytes()) refuse("out: must not overlap q");
    const int H = Pools::size(qt, 1), D = Pools::size(qt, 2);
    if (c.D != (q4 ? D / 16 * 9 : D))
      refuse_tensor(c.k, "k_cache", q4 ? "q4_0 rows of 9 head_dim / 16 bytes" : "e4m3 rows of head_dim bytes");
    const auto start = static_cast<const int32_t*>(want(tensor(a[6], "query_start"), "query_start", at::kInt, {c.B + 1},
                                                        c.dev, "contiguous int32 [num_seqs + 1] on the pools' device"));
    const float scale = as_float(a[7]);
    const int longest = as_int(a[10], "max_query_len");
    size_t bytes;
    void* ws = c.workspace(a[11], &bytes);
    int32_t* err = c.error_word(a[12]);
    const pkv_dtype code = code_of(qt.scalar_type(), "q");
    const float k_scale = q4 ? 1.f : as_float(a[8]), v_scale = q4 ? 1.f : as_float(a[9]);
    const c10::cuda::CUDAGuard guard(c.dev);
    const pkv_stream_t stream = c.stream(a[13]);
    if (q4)
      return pkv_paged_attention_prefill_q4_0(out, q, c.k.data_ptr(), c.v.data_ptr(), c.table(), c.lens, start, scale,
                                              H, c.Hkv, D, c.bs, c.B, c.MB, c.nb, longest, code, ws, bytes, err,
                                              stream);
    return pkv_paged_attention_prefill_fp8(out, q, c.k.data_ptr(), c.v.data_ptr(), c.table(), c.lens, start, scale,
                                           k_scale, v_scale, H, c.Hkv, D, c.bs, c.B, c.MB, c.nb, longest, code, ws,
                                           bytes, err, stream);
  });
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(decode_window), ENTRY(prefill_window), ENTRY(decode_scores), ENTRY(evict_tokens),
                         ENTRY(rope_and_cache), ENTRY(prefill_quant),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_torch", "Calls with torch tensors", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&module); }
