// marshal.cpp -- torch tensors to the plain pointers and sizes of include/pda.h, for calls whose
// kernels are shorter than a Python function that looks at a dozen tensors: each call here checks
// its tensors (device, type, shape, layout) and makes the C call, 2 us on the host where the same
// checks in Python and the conversion of 30 arguments took 8.
//
// Every function takes (device index, stream, the call's arguments ...) and returns the C call's
// status; the caller has made the device current. A tensor that does not fit raises ValueError
// before anything is launched. The C functions come from the library that the package has loaded
// (bind).
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "pda.h"

namespace {

decltype(&pda_qk_norm_rope_append) rope_append_fn;
decltype(&pda_qk_norm_rope) rope_fn;
decltype(&pda_paged_window_attention) window_fn;
decltype(&pda_paged_window_chunk_attention) window_chunk_fn;
decltype(&pda_verify_drafts) verify_fn;

using at::ScalarType;
using Sizes = std::initializer_list<int64_t>;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, int dev, const char* name) {
  if (t.is_cuda() && t.get_device() == dev) return;
  std::ostringstream s;
  s << name << " is on " << t.device() << "; all tensors must live on one CUDA device";
  refuse(s.str());
}

void fits(const at::Tensor& t, const char* name, ScalarType type, at::IntArrayRef sizes) {
  if (t.scalar_type() == type && t.sizes() == sizes) return;
  std::ostringstream s;
  s << name << " must be " << type << " of shape " << sizes << ", not " << t.scalar_type() << " "
    << t.sizes();
  refuse(s.str());
}

// The address of a dense tensor (None: NULL).
void* dense(PyObject* o, int dev, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  on_device(t, dev, name);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}
void* dense(PyObject* o, int dev, const char* name, ScalarType type, Sizes sizes) {
  void* p = dense(o, dev, name);
  if (o != Py_None) fits(THPVariable_Unpack(o), name, type, sizes);
  return p;
}
int32_t* ints(PyObject* o, int dev, const char* name, Sizes sizes) {
  return static_cast<int32_t*>(dense(o, dev, name, ScalarType::Int, sizes));
}
int32_t* error_word(PyObject* o, int dev) {
  return static_cast<int32_t*>(dense(o, dev, "error_word"));
}

int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a whole number");
  }
  return v;
}
int in_31_bits(PyObject* o, const char* name) {
  const int64_t v = whole(o, name);
  if (v < -0x7fffffff || v > 0x7fffffff) refuse(std::string(name) + " passes 31 bits");
  return static_cast<int>(v);
}
float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return static_cast<float>(v);
}
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(std::string(name) + " must be true or false");
  }
  return v != 0;
}

pda_dtype dtype(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case ScalarType::Float: return PDA_F32;
    case ScalarType::BFloat16: return PDA_BF16;
    case ScalarType::Half: return PDA_F16;
    case ScalarType::Byte:
    case ScalarType::Float8_e4m3fn: return PDA_FP8_E4M3;
    default: refuse(std::string(name) + " must be float32, bfloat16, float16 or FP8 E4M3 codes");
  }
}

// Dimensions must fit the C call's ints.
int size(const at::Tensor& t, int dim) {
  const int64_t n = t.size(dim);
  if (n > 0x7fffffff) refuse("a dimension passes 31 bits");
  return static_cast<int>(n);
}
void ranked(const at::Tensor& t, int64_t rank, const char* what) {
  if (t.dim() != rank) refuse(what);
}

// Rows [T, ...] whose tokens are any distance apart and dense in themselves.
struct Rows {
  void* at;
  long long stride;
  const char* begin;
  const char* end;
};
Rows rows(PyObject* o, int dev, const char* name, ScalarType type, Sizes sizes) {
  const at::Tensor& t = tensor(o, name);
  on_device(t, dev, name);
  fits(t, name, type, sizes);
  int64_t row = 1;
  for (int64_t d = t.dim() - 1; d > 0; --d) {
    if (t.size(d) != 1 && t.size(0) > 0 && t.stride(d) != row)
      refuse(std::string(name) + ": a row must be dense");
    row *= t.size(d);
  }
  const int64_t T = t.size(0), stride = T > 1 ? t.stride(0) : row;
  char* at = static_cast<char*>(t.data_ptr());
  return Rows{at, stride, at, T > 0 ? at + ((T - 1) * stride + row) * t.element_size() : at};
}
// Refuses an output that overlaps `x`, unless it is the same dense memory where that is allowed.
void apart(const Rows& out, const Rows& x, bool may_be_same, const char* name) {
  if (out.begin >= x.end || x.begin >= out.end) return;
  if (may_be_same && out.begin == x.begin && out.stride == x.stride) return;
  refuse(std::string("an output overlaps ") + name);
}
Rows dense_rows(PyObject* o, int dev, const char* name, ScalarType type, Sizes sizes) {
  const Rows r = rows(o, dev, name, type, sizes);
  if (!THPVariable_Unpack(o).is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return r;
}

cudaStream_t stream_of(PyObject* o) {
  return reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(o)));
}

// Makes the C call without the interpreter's lock (a launch may wait for room in its queue).
template <typename F, typename... Args>
int released(F f, Args... args) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = f(args...);
  PyEval_RestoreThread(state);
  return status;
}

// ---------------------------------------------------------------- the calls
int rope_append(PyObject* const* a) {
  const int dev = static_cast<int>(whole(a[0], "device"));
  const at::Tensor &q = tensor(a[3], "q"), &kc = tensor(a[6], "k_cache"),
                   &freqs = tensor(a[10], "freqs");
  ranked(q, 3, "q must be [T, H, D]");
  ranked(kc, 4, "the caches must be [NB, bs, H_kv, D]");
  ranked(freqs, 1, "freqs must be [rope_dim / 2]");
  const int T = size(q, 0), H = size(q, 1), D = size(q, 2);
  const int NB = size(kc, 0), bs = size(kc, 1), H_kv = size(kc, 2);
  if (kc.size(3) != D) refuse("q and the caches must agree in head size");
  const ScalarType type = q.scalar_type();
  const Rows out = dense_rows(a[2], dev, "q_out", type, {T, H, D});
  const Rows qr = rows(a[3], dev, "q", type, {T, H, D});
  const Rows kr = rows(a[4], dev, "k", type, {T, H_kv, D});
  const Rows vr = rows(a[5], dev, "v", type, {T, H_kv, D});
  apart(out, qr, true, "q");
  apart(out, kr, false, "k");
  apart(out, vr, false, "v");
  return released(
      rope_append_fn, out.at, qr.at, kr.at, vr.at, qr.stride, kr.stride, vr.stride,
      dense(a[6], dev, "k_cache"),
      dense(a[7], dev, "v_cache", kc.scalar_type(), {NB, bs, H_kv, D}),
      ints(a[8], dev, "slot_mapping", {T}), ints(a[9], dev, "positions", {T}),
      static_cast<const uint64_t*>(dense(a[10], dev, "freqs", ScalarType::Long, {freqs.size(0)})),
      2 * size(freqs, 0), truth(a[14], "interleaved"), number(a[15], "attention_factor"),
      dense(a[11], dev, "q_weight", type, {D}), dense(a[12], dev, "k_weight", type, {D}),
      number(a[13], "eps"), T, H, H_kv, D, bs, NB, number(a[16], "k_scale"),
      number(a[17], "v_scale"), dtype(q, "q"), dtype(kc, "k_cache"), error_word(a[18], dev),
      stream_of(a[1]));
}

int rope(PyObject* const* a) {
  const int dev = static_cast<int>(whole(a[0], "device"));
  const at::Tensor &q = tensor(a[4], "q"), &k = tensor(a[5], "k"), &freqs = tensor(a[7], "freqs");
  ranked(q, 3, "q must be [T, H, D]");
  ranked(k, 3, "k must be [T, H_kv, D]");
  ranked(freqs, 1, "freqs must be [rope_dim / 2]");
  const int T = size(q, 0), H = size(q, 1), D = size(q, 2), H_kv = size(k, 1);
  const ScalarType type = q.scalar_type();
  const Rows qo = dense_rows(a[2], dev, "q_out", type, {T, H, D});
  const Rows ko = dense_rows(a[3], dev, "k_out", type, {T, H_kv, D});
  const Rows qr = rows(a[4], dev, "q", type, {T, H, D});
  const Rows kr = rows(a[5], dev, "k", type, {T, H_kv, D});
  apart(qo, qr, true, "q");
  apart(qo, kr, false, "k");
  apart(ko, qr, false, "q");
  apart(ko, kr, true, "k");
  apart(qo, ko, false, "the other output");
  return released(
      rope_fn, qo.at, ko.at, qr.at, kr.at, qr.stride, kr.stride, ints(a[6], dev, "positions", {T}),
      static_cast<const uint64_t*>(dense(a[7], dev, "freqs", ScalarType::Long, {freqs.size(0)})),
      2 * size(freqs, 0), truth(a[11], "interleaved"), number(a[12], "attention_factor"),
      dense(a[8], dev, "q_weight", type, {D}), dense(a[9], dev, "k_weight", type, {D}),
      number(a[10], "eps"), T, H, H_kv, D, dtype(q, "q"), stream_of(a[1]));
}

void check_window(int window, int sinks) {
  if (window < 0 || sinks < 0) refuse("window and sinks must not be negative");
  if (window == 0) refuse("sinks are the first tokens beside a window");
}

int window(PyObject* const* a) {
  const int dev = static_cast<int>(whole(a[0], "device"));
  const at::Tensor &out = tensor(a[2], "out"), &q = tensor(a[3], "q"),
                   &kc = tensor(a[4], "k_cache"), &tables = tensor(a[8], "block_tables"),
                   &ws = tensor(a[18], "workspace");
  const int W = in_31_bits(a[11], "window"), S = in_31_bits(a[12], "sinks");
  check_window(W, S);
  ranked(q, 3, "q must be [B, H, D]");
  ranked(kc, 4, "the caches must be [NB, bs, H_kv, D]");
  ranked(tables, 2, "block_tables must be [B, max_blocks]");
  const auto kv = static_cast<pda_dtype>(in_31_bits(a[16], "kv_dtype"));
  const int B = size(q, 0), H = size(q, 1), D = size(q, 2);
  const int NB = size(kc, 0), bs = size(kc, 1), H_kv = size(kc, 2);
  if (kc.size(3) != (kv == PDA_NVFP4 ? D / 2 : D))
    refuse("q and the caches must agree in head size");
  if (dtype(kc, "k_cache") != (kv == PDA_NVFP4 ? PDA_FP8_E4M3 : kv))
    refuse(kv == PDA_FP8_E4M3 || kv == PDA_NVFP4 ? "the caches must hold codes"
                                                 : "an FP8 cache needs its scales: the _fp8 call");
  void *k_bs = nullptr, *v_bs = nullptr;
  if (kv == PDA_NVFP4) {
    const ScalarType type = tensor(a[6], "k_block_scales").scalar_type();
    k_bs = dense(a[6], dev, "k_block_scales", type, {NB, H_kv, bs, D / 16});
    v_bs = dense(a[7], dev, "v_block_scales", type, {NB, H_kv, bs, D / 16});
  }
  return released(
      window_fn, dense(a[2], dev, "out", out.scalar_type(), {B, H, D}), dense(a[3], dev, "q"),
      dense(a[4], dev, "k_cache"),
      dense(a[5], dev, "v_cache", kc.scalar_type(), {NB, bs, H_kv, kc.size(3)}), k_bs, v_bs,
      ints(a[8], dev, "block_tables", {B, tables.size(1)}), size(tables, 1),
      ints(a[9], dev, "context_lens", {B}), in_31_bits(a[10], "max_context_len"), W, S, B, H, H_kv,
      D, bs, NB, number(a[13], "scale"), number(a[14], "k_scale"), number(a[15], "v_scale"),
      dtype(q, "q"), kv, dtype(out, "out"), in_31_bits(a[17], "sm_cap"),
      dense(a[18], dev, "workspace"), ws.nbytes(), error_word(a[19], dev), stream_of(a[1]));
}

int window_chunk(PyObject* const* a) {
  const int dev = static_cast<int>(whole(a[0], "device"));
  const at::Tensor &q = tensor(a[3], "q"), &kc = tensor(a[4], "k_cache"),
                   &tables = tensor(a[6], "block_tables"), &ws = tensor(a[17], "workspace");
  const int W = in_31_bits(a[10], "window"), S = in_31_bits(a[11], "sinks");
  check_window(W, S);
  ranked(q, 3, "q must be [T, H, D]");
  ranked(kc, 4, "the caches must be [NB, bs, H_kv, D]");
  ranked(tables, 2, "block_tables must be [B, max_blocks]");
  const bool codes = truth(a[15], "codes");
  const int T = size(q, 0), H = size(q, 1), D = size(q, 2), B = size(tables, 0);
  const int NB = size(kc, 0), bs = size(kc, 1), H_kv = size(kc, 2);
  if (kc.size(3) != D) refuse("q and the caches must agree in head size");
  const pda_dtype kv = dtype(kc, "k_cache");
  if ((kv == PDA_FP8_E4M3) != codes)
    refuse(codes ? "the caches must hold FP8 E4M3 codes"
                 : "an FP8 cache needs its scales: the _fp8 call");
  return released(
      window_chunk_fn, dense(a[2], dev, "out", q.scalar_type(), {T, H, D}), dense(a[3], dev, "q"),
      dense(a[4], dev, "k_cache"), dense(a[5], dev, "v_cache", kc.scalar_type(), {NB, bs, H_kv, D}),
      ints(a[6], dev, "block_tables", {B, tables.size(1)}), size(tables, 1),
      ints(a[7], dev, "context_lens", {B}), ints(a[8], dev, "query_start", {B + 1}),
      in_31_bits(a[9], "max_context_len"), W, S, B, T, H, H_kv, D, bs, NB, number(a[12], "scale"),
      number(a[13], "k_scale"), number(a[14], "v_scale"), dtype(q, "q"), kv,
      in_31_bits(a[16], "sm_cap"), dense(a[17], dev, "workspace"), ws.nbytes(),
      error_word(a[18], dev), stream_of(a[1]));
}

int verify(PyObject* const* a) {
  const int dev = static_cast<int>(whole(a[0], "device"));
  const at::Tensor &p = tensor(a[4], "target_probs"), &accepted = tensor(a[2], "accepted");
  ranked(p, 2, "target_probs must be [T, V]");
  ranked(accepted, 1, "accepted must be [B]");
  const int T = size(p, 0), V = size(p, 1), B = size(accepted, 0);
  const ScalarType type = p.scalar_type();
  const Rows target = rows(a[4], dev, "target_probs", type, {T, V});
  Rows draft{};
  if (a[5] != Py_None) draft = rows(a[5], dev, "draft_probs", type, {T, V});
  return released(
      verify_fn, ints(a[2], dev, "accepted", {B}), ints(a[3], dev, "next_tokens", {B}), target.at,
      draft.at, target.stride, draft.stride, ints(a[6], dev, "tokens", {T}),
      ints(a[7], dev, "query_start", {B + 1}),
      static_cast<float*>(dense(a[8], dev, "accept_u", ScalarType::Float, {T})),
      static_cast<float*>(dense(a[9], dev, "sample_u", ScalarType::Float, {B})), T, B, V,
      dtype(p, "target_probs"), error_word(a[10], dev), stream_of(a[1]));
}

// ---------------------------------------------------------------- the module
template <int (*call)(PyObject* const*), Py_ssize_t count>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "takes %zd arguments, got %zd", count, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(call(args));
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(addresses of the C functions, in this order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "takes the five functions' addresses");
    return nullptr;
  }
  uintptr_t at[5];
  for (int i = 0; i < 5; ++i) at[i] = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(a[i]));
  if (PyErr_Occurred()) return nullptr;
  rope_append_fn = reinterpret_cast<decltype(rope_append_fn)>(at[0]);
  rope_fn = reinterpret_cast<decltype(rope_fn)>(at[1]);
  window_fn = reinterpret_cast<decltype(window_fn)>(at[2]);
  window_chunk_fn = reinterpret_cast<decltype(window_chunk_fn)>(at[3]);
  verify_fn = reinterpret_cast<decltype(verify_fn)>(at[4]);
  Py_RETURN_NONE;
}

#define PDA_ENTRY(name, fn, count) \
  {name, reinterpret_cast<PyCFunction>(entry<fn, count>), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    PDA_ENTRY("qk_norm_rope_append", rope_append, 19),
    PDA_ENTRY("qk_norm_rope", rope, 13),
    PDA_ENTRY("paged_window_attention", window, 20),
    PDA_ENTRY("paged_window_chunk_attention", window_chunk, 19),
    PDA_ENTRY("verify_drafts", verify, 11),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
