// pa_torch.cpp -- the torch side of the cache operators and of a prompt's way into the cache: checks of the tensors (the library sees only
// pointers), allocation of the outputs that are not given, and the call into libpagedfp8.
//
// These calls come several times per decode step, and their kernels take a few microseconds.  Checked
// and marshalled in Python they cost 11 to 23 us each on the host, more than most of the kernels;
// here 3 to 9.  The functions take their arguments by position, as binding.py passes them; None stands
// for what is absent.  Tensors have to be dense (queries, keys and values of a prompt may be views of one projection's
// output), of the documented type and shape, and all on one CUDA device, on which the call runs whatever the current
// device is.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <exception>
#include <optional>
#include <sstream>
#include <string>

#include "pa.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// The library's entry points and the error class, handed over by bind().
struct Library {
  pa_status_t (*attn_mass)(const pa_attn_mass_args_t *, void *) = nullptr;
  pa_status_t (*evict_select)(const pa_evict_select_args_t *, void *) = nullptr;
  pa_status_t (*kv_compact)(const pa_kv_compact_args_t *, void *) = nullptr;
  pa_status_t (*beam_select)(const pa_beam_select_args_t *, void *) = nullptr;
  pa_status_t (*beam_reorder)(const pa_beam_reorder_args_t *, void *) = nullptr;
  pa_status_t (*page_assign)(const pa_page_assign_args_t *, void *) = nullptr;
  pa_status_t (*page_release)(const pa_page_release_args_t *, void *) = nullptr;
  pa_status_t (*rope)(const pa_rope_args_t *, void *) = nullptr;
  pa_status_t (*prompt_attn)(const pa_prompt_attn_args_t *, void *) = nullptr;
  PyObject *error = nullptr;
} g_lib;

// A refused argument: a Python exception of this type.  With type NULL one is already set.
struct Refusal : std::exception {
  PyObject *type;
  std::string text;
  Refusal(PyObject *t, std::string s) : type(t), text(std::move(s)) {}
};
[[noreturn]] void type_error(const std::string &s) { throw Refusal(PyExc_TypeError, s); }
[[noreturn]] void value_error(const std::string &s) { throw Refusal(PyExc_ValueError, s); }

std::string shape_text(IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << ")";
  return o.str();
}

// ------------------------------------------------------------------------- arguments

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

int32_t int_arg(PyObject *o, const char *name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refusal(nullptr, "");
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + ": beyond 32 bits");
  return (int32_t)v;
}

int32_t int_of(int64_t v, const char *name) {
  if (v > INT32_MAX) value_error(std::string(name) + ": beyond 32 bits");
  return (int32_t)v;
}

float float_arg(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refusal(nullptr, "");
  return (float)v;
}

IntArrayRef rank(const Tensor &t, int64_t dims, const char *name) {
  if (t.dim() != dims)
    value_error(std::string(name) + ": " + std::to_string(t.dim()) + " dimensions, expected " + std::to_string(dims));
  return t.sizes();
}

// The pointer of a dense tensor of this type and shape on CUDA device dev.
void *need(const Tensor &t, const char *name, ScalarType type, IntArrayRef shape, int dev) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + ": " + toString(t.scalar_type()) + ", expected " + toString(type));
  if (t.sizes() != shape) value_error(std::string(name) + ": shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
  if (!t.is_contiguous()) value_error(std::string(name) + ": must be contiguous");
  if (!t.is_cuda() || t.get_device() != dev)
    value_error(std::string(name) + ": on " + t.device().str() + ", expected cuda:" + std::to_string(dev) + " like the rest of the call");
  return t.data_ptr();
}
void *need(PyObject *o, const char *name, ScalarType type, IntArrayRef shape, int dev) {
  return need(tensor(o, name), name, type, shape, dev);
}
void *need_or_null(PyObject *o, const char *name, ScalarType type, IntArrayRef shape, int dev) {
  return o == Py_None ? nullptr : need(o, name, type, shape, dev);
}

// The pointer of a [tokens, heads, head_dim] tensor whose tokens may lie apart (a view of a projection's output), and the
// elements between tokens.
void *token_rows(const Tensor &t, const char *name, ScalarType type, IntArrayRef shape, int dev, int64_t &stride) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + ": " + toString(t.scalar_type()) + ", expected " + toString(type));
  if (t.sizes() != shape) value_error(std::string(name) + ": shape " + shape_text(t.sizes()) + ", expected " + shape_text(shape));
  const IntArrayRef st = t.strides();
  const int64_t row = shape[1] * shape[2];
  stride = shape[0] > 1 ? st[0] : row;  // the stride of a dimension of size 1 means nothing
  if ((shape[2] > 1 && st[2] != 1) || (shape[1] > 1 && st[1] != shape[2]) || stride < row)
    value_error(std::string(name) + ": a token's heads must lie one behind the other, and its tokens apart");
  if (!t.is_cuda() || t.get_device() != dev)
    value_error(std::string(name) + ": on " + t.device().str() + ", expected cuda:" + std::to_string(dev) + " like the rest of the call");
  return t.data_ptr();
}

int cuda_device(const Tensor &t) {
  if (!t.is_cuda()) value_error("tensors on " + t.device().str() + ", expected a CUDA device");
  return t.get_device();
}

uint32_t *status_word(PyObject *o, int dev) {
  if (o == Py_None) return nullptr;
  const Tensor &t = tensor(o, "status");
  if (t.element_size() != 4 || t.numel() < 1 || !t.is_cuda() || t.get_device() != dev)
    value_error("status: a 4-byte word on the call's device");
  return static_cast<uint32_t *>(t.data_ptr());
}

// A cache tensor's mode: its type, and whether per-token scales come with it.
int32_t kv_dtype(const Tensor &k) {
  const ScalarType t = k.scalar_type();
  if (t == ScalarType::Byte || t == ScalarType::Float8_e4m3fn) return PA_KV_FP8_E4M3;
  if (t != ScalarType::BFloat16) type_error(std::string("k_cache: ") + toString(t) + ", expected uint8, float8_e4m3fn or bfloat16");
  return PA_KV_BF16;
}
int32_t scale_mode(int32_t kv, bool scales) {
  if (kv == PA_KV_FP8_E4M3) return scales ? PA_SCALE_PER_TOKEN : PA_SCALE_SCALAR;
  if (scales) value_error("k_scale: a bf16 cache has no scales");
  return PA_SCALE_NONE;
}

// The K and V caches and scales of a call, into the fields all its structures share.
template <typename Args>
void caches(Args &a, PyObject *ko, PyObject *vo, PyObject *kso, PyObject *vso, int dev) {
  const Tensor &k = tensor(ko, "k_cache");
  const IntArrayRef s = rank(k, 4, "k_cache");
  a.k_cache = need(k, "k_cache", k.scalar_type(), s, dev);
  a.v_cache = need(vo, "v_cache", k.scalar_type(), s, dev);
  if ((kso == Py_None) != (vso == Py_None)) value_error("k_scale and v_scale: both or neither");
  a.k_scale = static_cast<float *>(need_or_null(kso, "k_scale", ScalarType::Float, s.slice(0, 3), dev));
  a.v_scale = static_cast<float *>(need_or_null(vso, "v_scale", ScalarType::Float, s.slice(0, 3), dev));
  a.kv_dtype = kv_dtype(k);
  a.scale_mode = scale_mode(a.kv_dtype, kso != Py_None);
  a.num_pages = s[0];
  a.num_kv_heads = int_of(s[1], "k_cache");
  a.page_size = int_of(s[2], "k_cache");
  a.head_dim = int_of(s[3], "k_cache");
}

// The launching stream: a handle, or torch's current one on the device.
c10::cuda::CUDAStream stream_arg(PyObject *o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
  const unsigned long long h = PyLong_AsUnsignedLongLong(o);
  if (PyErr_Occurred()) throw Refusal(nullptr, "");
  return c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(h), (c10::DeviceIndex)dev);
}

// A new tensor from torch's allocator, on the launching stream (the allocator reuses a block in the order of the stream
// it was allocated on).  Each output has storage of its own: tensors cut from one allocation would cost less, but a
// caller's resize_ of one runs into its neighbour.  Without the dispatcher, which takes as long as the allocation.
Tensor make(ScalarType type, IntArrayRef shape, int dev, const c10::cuda::CUDAStream &stream, bool own_stream) {
  std::optional<c10::cuda::CUDAStreamGuard> on;
  std::optional<c10::cuda::CUDAGuard> at_dev;
  if (own_stream)
    on.emplace(stream);
  else if (c10::cuda::current_device() != dev)
    at_dev.emplace((c10::DeviceIndex)dev);
  return Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                          type, std::nullopt));
}

// A given output, or a new one.  Owns a reference to the Python object.
class Output {
 public:
  Output() = default;
  Output(PyObject *given, const char *name, ScalarType type, IntArrayRef shape, int dev, const c10::cuda::CUDAStream &stream,
         bool own_stream) {
    if (given != Py_None) {
      ptr_ = need(given, name, type, shape, dev);
      Py_INCREF(given);
      obj_ = given;
      return;
    }
    Tensor t = make(type, shape, dev, stream, own_stream);
    ptr_ = t.data_ptr();
    obj_ = THPVariable_Wrap(std::move(t));
    if (obj_ == nullptr) throw Refusal(nullptr, "");
  }
  ~Output() { Py_XDECREF(obj_); }
  Output(const Output &) = delete;
  Output &operator=(const Output &) = delete;
  template <typename T>
  T *as() const {
    return static_cast<T *>(ptr_);
  }
  PyObject *release() {  // None where there is no output
    PyObject *o = obj_;
    obj_ = nullptr;
    if (o == nullptr) Py_RETURN_NONE;
    return o;
  }

 private:
  void *ptr_ = nullptr;
  PyObject *obj_ = nullptr;
};

// Calls an entry point on the device and stream; a status other than PA_OK becomes the error class.
// An empty batch enqueues nothing (torch's empty tensors have no pointer that the library could check).
template <typename Args>
void enqueue(const char *name, pa_status_t (*entry)(const Args *, void *), const Args &a, bool empty, int dev,
             const c10::cuda::CUDAStream &stream) {
  if (empty) return;
  if (entry == nullptr) throw Refusal(PyExc_RuntimeError, "the library is not bound");
  pa_status_t st;
  if (c10::cuda::current_device() == dev) {
    st = entry(&a, stream.stream());
  } else {
    const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
    st = entry(&a, stream.stream());
  }
  if (st == PA_OK) return;
  PyObject *e = PyObject_CallFunction(g_lib.error, "is", (int)st, name);
  if (e != nullptr) {
    PyErr_SetObject(g_lib.error, e);
    Py_DECREF(e);
  }
  throw Refusal(nullptr, "");
}

// Runs a call's body; exceptions become Python ones.
template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t expected, F &&body) {
  if (got != expected) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refusal &r) {
    if (r.type != nullptr) PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception &e) {  // from torch: an allocation that failed, a CUDA error
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// ------------------------------------------------------------------------------ calls

// q, k_cache, block_table, context_lens, cu_seqlens_q, lse, mass, out, k_scale, status, stream, max_q_len,
// sm_scale or None, decay, k_scale_scalar -> the updated mass
PyObject *attn_mass(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject * {
    const Tensor &q = tensor(x[0], "q"), &k = tensor(x[1], "k_cache"), &mass = tensor(x[6], "mass");
    const int dev = cuda_device(k);
    const IntArrayRef c = rank(k, 4, "k_cache"), qs = rank(q, 3, "q"), ms = rank(mass, 3, "mass");
    const IntArrayRef ts = rank(tensor(x[2], "block_table"), 2, "block_table");
    if (c[1] < 1 || qs[1] % c[1] != 0 || ms[1] != c[1] || ts[0] != ms[0])
      value_error("q " + shape_text(qs) + ", mass " + shape_text(ms) + " and block_table " + shape_text(ts) + " for " +
                  std::to_string(c[1]) + " KV heads");
    const int64_t B = ms[0], B1 = B + 1;
    pa_attn_mass_args_t a = {};
    a.q = need(q, "q", ScalarType::BFloat16, {qs[0], qs[1], c[3]}, dev);
    a.k_cache = need(k, "k_cache", k.scalar_type(), c, dev);
    a.k_scale = static_cast<float *>(need_or_null(x[8], "k_scale", ScalarType::Float, c.slice(0, 3), dev));
    a.block_table = static_cast<int32_t *>(need(x[2], "block_table", ScalarType::Int, ts, dev));
    a.context_lens = static_cast<int32_t *>(need(x[3], "context_lens", ScalarType::Int, B, dev));
    a.cu_seqlens_q = static_cast<int32_t *>(need(x[4], "cu_seqlens_q", ScalarType::Int, B1, dev));
    a.lse = static_cast<float *>(need(x[5], "lse", ScalarType::Float, qs.slice(0, 2), dev));
    a.mass = static_cast<float *>(need(mass, "mass", ScalarType::Float, ms, dev));
    PyObject *out = x[7] == Py_None ? x[6] : x[7];
    a.mass_out = static_cast<float *>(need(out, "out", ScalarType::Float, ms, dev));
    a.status = status_word(x[9], dev);
    a.num_pages = c[0];
    a.num_seqs = int_of(B, "mass");
    a.num_rows = int_of(qs[0], "q");
    a.num_kv_heads = int_of(c[1], "k_cache");
    a.group_size = int_of(qs[1] / c[1], "q");
    a.head_dim = int_of(c[3], "k_cache");
    a.page_size = int_of(c[2], "k_cache");
    a.kv_dtype = kv_dtype(k);
    a.scale_mode = scale_mode(a.kv_dtype, x[8] != Py_None);
    a.block_table_stride = int_of(ts[1], "block_table");
    a.mass_stride = int_of(ms[2], "mass");
    a.max_q_len = int_arg(x[11], "max_q_len");
    a.sm_scale = x[12] == Py_None ? (float)(1.0 / std::sqrt((double)c[3])) : float_arg(x[12]);
    a.decay = float_arg(x[13]);
    a.k_scale_scalar = float_arg(x[14]);
    enqueue("pa_attn_mass", g_lib.attn_mass, a, B == 0 || qs[0] == 0, dev, stream_arg(x[10], dev));
    Py_INCREF(out);
    return out;
  });
}

// mass, context_lens, keep, new_lens, status, stream, budget, first, recent -> (keep, new_lens)
PyObject *evict_select(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const Tensor &mass = tensor(x[0], "mass");
    const int dev = cuda_device(mass);
    const IntArrayRef s = rank(mass, 3, "mass");
    const auto stream = stream_arg(x[5], dev);
    pa_evict_select_args_t a = {};
    a.mass = static_cast<float *>(need(mass, "mass", ScalarType::Float, s, dev));
    a.context_lens = static_cast<int32_t *>(need(x[1], "context_lens", ScalarType::Int, s[0], dev));
    a.status = status_word(x[4], dev);
    a.num_seqs = int_of(s[0], "mass");
    a.num_kv_heads = int_of(s[1], "mass");
    a.mass_stride = int_of(s[2], "mass");
    a.budget = int_arg(x[6], "budget");
    a.keep_first = int_arg(x[7], "first");
    a.keep_recent = int_arg(x[8], "recent");
    const int64_t width = a.budget > 0 ? a.budget : 1;  // (the library refuses a budget below 1)
    const bool own_stream = x[5] != Py_None;
    Output keep(x[2], "keep", ScalarType::Int, {s[0], s[1], width}, dev, stream, own_stream);
    Output lens(x[3], "new_lens", ScalarType::Int, s[0], dev, stream, own_stream);
    a.keep = keep.as<int32_t>();
    a.new_lens = lens.as<int32_t>();
    enqueue("pa_evict_select", g_lib.evict_select, a, s[0] == 0, dev, stream);
    return Py_BuildValue("(NN)", keep.release(), lens.release());
  });
}

// keep, new_lens, block_table, dst_block_table, k_cache, v_cache, k_scale, v_scale, mass, mass_out, status,
// stream -> None
PyObject *kv_compact(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    const int dev = cuda_device(tensor(x[4], "k_cache"));
    pa_kv_compact_args_t a = {};
    caches(a, x[4], x[5], x[6], x[7], dev);
    const IntArrayRef ks = rank(tensor(x[0], "keep"), 3, "keep"), ts = rank(tensor(x[2], "block_table"), 2, "block_table");
    const int64_t B = ks[0], H = a.num_kv_heads;
    a.keep = static_cast<int32_t *>(need(x[0], "keep", ScalarType::Int, {B, H, ks[2]}, dev));
    a.new_lens = static_cast<int32_t *>(need(x[1], "new_lens", ScalarType::Int, B, dev));
    a.block_table = static_cast<int32_t *>(need(x[2], "block_table", ScalarType::Int, {B, ts[1]}, dev));
    if (x[3] != Py_None) {
      const IntArrayRef ds = rank(tensor(x[3], "dst_block_table"), 2, "dst_block_table");
      a.dst_block_table = static_cast<int32_t *>(need(x[3], "dst_block_table", ScalarType::Int, {B, ds[1]}, dev));
      a.dst_block_table_stride = int_of(ds[1], "dst_block_table");
    }
    PyObject *mo = x[9] == Py_None && x[3] == Py_None ? x[8] : x[9];
    if ((x[8] == Py_None) != (mo == Py_None)) value_error("mass and mass_out: both or neither (in place mass alone)");
    if (x[8] != Py_None) {
      const IntArrayRef m = rank(tensor(x[8], "mass"), 3, "mass"), o = rank(tensor(mo, "mass_out"), 3, "mass_out");
      a.mass = static_cast<float *>(need(x[8], "mass", ScalarType::Float, {B, H, m[2]}, dev));
      a.mass_out = static_cast<float *>(need(mo, "mass_out", ScalarType::Float, {B, H, o[2]}, dev));
      a.mass_stride = int_of(m[2], "mass");
      a.mass_out_stride = int_of(o[2], "mass_out");
    }
    a.status = status_word(x[10], dev);
    a.num_seqs = int_of(B, "keep");
    a.keep_stride = int_of(ks[2], "keep");
    a.block_table_stride = int_of(ts[1], "block_table");
    enqueue("pa_kv_compact", g_lib.kv_compact, a, B == 0, dev, stream_arg(x[11], dev));
    Py_RETURN_NONE;
  });
}

// logits, scores, finished, lengths, tokens, parents, scores_out, finished_out, lengths_out, stream, eos,
// length_penalty -> (tokens, parents, scores, finished or None, lengths or None)
PyObject *beam_select(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    const Tensor &logits = tensor(x[0], "logits"), &scores = tensor(x[1], "scores");
    const int dev = cuda_device(logits);
    const bool own = x[9] != Py_None;
    const auto stream = stream_arg(x[9], dev);
    const IntArrayRef s = rank(scores, 2, "scores"), l = logits.sizes();
    const int64_t N = s[0], W = s[1];
    const ScalarType t = logits.scalar_type();
    if (t != ScalarType::BFloat16 && t != ScalarType::Float)
      type_error(std::string("logits: ") + toString(t) + ", expected bfloat16 or float32");
    if (!((l.size() == 3 && l[0] == N && l[1] == W) || (l.size() == 2 && l[0] == N * W)))
      value_error("logits: shape " + shape_text(l) + " for " + std::to_string(N) + " x " + std::to_string(W) + " beams");
    const int64_t V = l.back();
    int64_t stride = V;
    if (!logits.is_contiguous()) {
      const IntArrayRef st = logits.strides();
      bool even = true;
      if (l.size() == 3) {  // the stride of a dimension of size 1 means nothing
        stride = W > 1 ? st[1] : N > 1 ? st[0] : V;
        even = N == 1 || st[0] == W * stride;
      } else if (N * W > 1) {
        stride = st[0];
      }
      if ((V > 1 && st.back() != 1) || stride < V || !even) value_error("logits: rows must be dense and evenly spaced");
    }
    pa_beam_select_args_t a = {};
    a.logits = logits.data_ptr();
    a.scores = static_cast<float *>(need(scores, "scores", ScalarType::Float, s, dev));
    a.finished = static_cast<uint8_t *>(need_or_null(x[2], "finished", ScalarType::Byte, s, dev));
    a.lengths = static_cast<int32_t *>(need_or_null(x[3], "lengths", ScalarType::Int, s, dev));
    a.logits_stride = stride;
    a.num_reqs = int_of(N, "scores");
    a.num_beams = int_of(W, "scores");
    a.vocab = int_of(V, "logits");
    a.logits_dtype = t == ScalarType::Float ? PA_LOGITS_F32 : PA_LOGITS_BF16;
    a.eos_token = int_arg(x[10], "eos");
    a.length_penalty = float_arg(x[11]);
    const bool ends = x[2] != Py_None || x[7] != Py_None, lasts = x[3] != Py_None || x[8] != Py_None;
    Output tokens(x[4], "tokens", ScalarType::Int, s, dev, stream, own), parents(x[5], "parents", ScalarType::Int, s, dev, stream, own);
    Output totals(x[6], "scores_out", ScalarType::Float, s, dev, stream, own);
    std::optional<Output> ended, lens;
    if (ends) ended.emplace(x[7], "finished_out", ScalarType::Byte, s, dev, stream, own);
    if (lasts) lens.emplace(x[8], "lengths_out", ScalarType::Int, s, dev, stream, own);
    a.tokens = tokens.as<int32_t>();
    a.parents = parents.as<int32_t>();
    a.scores_out = totals.as<float>();
    if (ends) a.finished_out = ended->as<uint8_t>();
    if (lasts) a.lengths_out = lens->as<int32_t>();
    enqueue("pa_beam_select", g_lib.beam_select, a, N == 0, dev, stream);
    Output none;
    return Py_BuildValue("(NNNNN)", tokens.release(), parents.release(), totals.release(),
                         ended ? ended->release() : none.release(), lens ? lens->release() : none.release());
  });
}

// parents, context_lens, block_table, block_table_out, k_cache, v_cache, k_scale, v_scale, states, status,
// stream -> None
PyObject *beam_reorder(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const int dev = cuda_device(tensor(x[4], "k_cache"));
    pa_beam_reorder_args_t a = {};
    caches(a, x[4], x[5], x[6], x[7], dev);
    const IntArrayRef s = rank(tensor(x[0], "parents"), 2, "parents"), ts = rank(tensor(x[2], "block_table"), 2, "block_table");
    const int64_t R = s[0] * s[1];
    a.parents = static_cast<int32_t *>(need(x[0], "parents", ScalarType::Int, s, dev));
    a.context_lens = static_cast<int32_t *>(need(x[1], "context_lens", ScalarType::Int, R, dev));
    a.block_table = static_cast<int32_t *>(need(x[2], "block_table", ScalarType::Int, {R, ts[1]}, dev));
    a.block_table_out = static_cast<int32_t *>(need(x[3], "block_table_out", ScalarType::Int, {R, ts[1]}, dev));
    PyObject *pairs = PySequence_Fast(x[8], "states: expected a sequence of (in, out) pairs");
    if (pairs == nullptr) throw Refusal(nullptr, "");
    struct Owned {
      PyObject *o;
      ~Owned() { Py_DECREF(o); }
    } owned{pairs};
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(pairs);
    if (count > PA_MAX_BEAM_STATES) value_error("states: at most " + std::to_string(PA_MAX_BEAM_STATES));
    for (Py_ssize_t i = 0; i < count; ++i) {
      PyObject *pair = PySequence_Fast_GET_ITEM(pairs, i);
      if (!(PyTuple_Check(pair) || PyList_Check(pair)) || PySequence_Fast_GET_SIZE(pair) != 2)
        value_error("states: expected (in, out) pairs");
      const Tensor &in = tensor(PySequence_Fast_GET_ITEM(pair, 0), "states' input");
      if (in.dim() < 1 || in.size(0) != R)
        value_error("states: shape " + shape_text(in.sizes()) + ", expected " + std::to_string(R) + " rows");
      a.state_in[i] = need(in, "states' input", in.scalar_type(), in.sizes(), dev);
      a.state_out[i] = need(PySequence_Fast_GET_ITEM(pair, 1), "states' output", in.scalar_type(), in.sizes(), dev);
      a.state_bytes[i] = R > 0 ? in.numel() / R * (int64_t)in.element_size() : (int64_t)in.element_size();
    }
    a.status = status_word(x[9], dev);
    a.num_states = (int32_t)count;
    a.num_reqs = int_of(s[0], "parents");
    a.num_beams = int_of(s[1], "parents");
    a.block_table_stride = int_of(ts[1], "block_table");
    enqueue("pa_beam_reorder", g_lib.beam_reorder, a, s[0] == 0, dev, stream_arg(x[10], dev));
    Py_RETURN_NONE;
  });
}

// context_lens, cu_seqlens_q, block_table, free_pages, num_free, num_free_out, new_lens, slot_mapping, positions, status,
// stream, page_size, num_pages, num_rows or None -> (new_lens, slot_mapping, positions)
PyObject *page_assign(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject * {
    const Tensor &table = tensor(x[2], "block_table");
    const int dev = cuda_device(table);
    const IntArrayRef ts = rank(table, 2, "block_table"), fs = rank(tensor(x[3], "free_pages"), 1, "free_pages");
    const auto stream = stream_arg(x[10], dev);
    const bool own = x[10] != Py_None;
    const int64_t B = ts[0], B1 = B + 1, one = 1;
    pa_page_assign_args_t a = {};
    a.context_lens = static_cast<int32_t *>(need(x[0], "context_lens", ScalarType::Int, B, dev));
    a.cu_seqlens_q = static_cast<int32_t *>(need(x[1], "cu_seqlens_q", ScalarType::Int, B1, dev));
    a.block_table = static_cast<int32_t *>(need(table, "block_table", ScalarType::Int, ts, dev));
    a.free_pages = static_cast<int32_t *>(need(x[3], "free_pages", ScalarType::Int, fs, dev));
    a.num_free = static_cast<int32_t *>(need(x[4], "num_free", ScalarType::Int, one, dev));
    a.num_free_out = static_cast<int32_t *>(need(x[5] == Py_None ? x[4] : x[5], "num_free_out", ScalarType::Int, one, dev));
    a.status = status_word(x[9], dev);
    a.page_size = int_arg(x[11], "page_size");
    a.num_pages = int_arg(x[12], "num_pages");
    int64_t rows = 0;
    if (x[13] != Py_None)
      rows = int_arg(x[13], "num_rows");
    else if (x[7] != Py_None)
      rows = rank(tensor(x[7], "slot_mapping"), 1, "slot_mapping")[0];
    else
      type_error("num_rows: needed without slot_mapping");
    if (rows < 0) value_error("num_rows: negative");
    a.num_seqs = int_of(B, "block_table");
    a.num_rows = int_of(rows, "slot_mapping");
    a.block_table_stride = int_of(ts[1], "block_table");
    a.free_capacity = int_of(fs[0], "free_pages");
    Output lens(x[6], "new_lens", ScalarType::Int, B, dev, stream, own), slots(x[7], "slot_mapping", ScalarType::Long, rows, dev, stream, own),
        pos(x[8], "positions", ScalarType::Int, rows, dev, stream, own);
    a.new_lens = lens.as<int32_t>();
    a.slot_mapping = slots.as<int64_t>();
    a.positions = pos.as<int32_t>();
    enqueue("pa_page_assign", g_lib.page_assign, a, false, dev, stream);
    return Py_BuildValue("(NNN)", lens.release(), slots.release(), pos.release());
  });
}

// context_lens, new_lens, block_table, free_pages, num_free, num_free_out, status, stream, page_size, num_pages -> None
PyObject *page_release(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const Tensor &table = tensor(x[2], "block_table");
    const int dev = cuda_device(table);
    const IntArrayRef ts = rank(table, 2, "block_table"), fs = rank(tensor(x[3], "free_pages"), 1, "free_pages");
    const int64_t B = ts[0], one = 1;
    pa_page_release_args_t a = {};
    a.context_lens = static_cast<int32_t *>(need(x[0], "context_lens", ScalarType::Int, B, dev));
    a.new_lens = static_cast<int32_t *>(need(x[1], "new_lens", ScalarType::Int, B, dev));
    a.block_table = static_cast<int32_t *>(need(table, "block_table", ScalarType::Int, ts, dev));
    a.free_pages = static_cast<int32_t *>(need(x[3], "free_pages", ScalarType::Int, fs, dev));
    a.num_free = static_cast<int32_t *>(need(x[4], "num_free", ScalarType::Int, one, dev));
    a.num_free_out = static_cast<int32_t *>(need(x[5] == Py_None ? x[4] : x[5], "num_free_out", ScalarType::Int, one, dev));
    a.status = status_word(x[6], dev);
    a.page_size = int_arg(x[8], "page_size");
    a.num_pages = int_arg(x[9], "num_pages");
    a.num_seqs = int_of(B, "block_table");
    a.block_table_stride = int_of(ts[1], "block_table");
    a.free_capacity = int_of(fs[0], "free_pages");
    enqueue("pa_page_release", g_lib.page_release, a, false, dev, stream_arg(x[7], dev));
    Py_RETURN_NONE;
  });
}

// q, k or None, positions, freqs, q_out, k_out, stream, layout, inverse, scale -> (q_out, k_out or None); without an
// output its input is turned in place
PyObject *rope(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const Tensor &q = tensor(x[0], "q");
    const int dev = cuda_device(q);
    const IntArrayRef qs = rank(q, 3, "q"), fs = rank(tensor(x[3], "freqs"), 1, "freqs");
    const ScalarType t = q.scalar_type();
    if (t != ScalarType::BFloat16 && t != ScalarType::Float)
      type_error(std::string("q: ") + toString(t) + ", expected bfloat16 or float32");
    pa_rope_args_t a = {};
    a.q = token_rows(q, "q", t, qs, dev, a.q_stride);
    PyObject *qo = x[4] == Py_None ? x[0] : x[4], *ko = x[5] == Py_None ? x[1] : x[5];
    a.q_out = token_rows(tensor(qo, "q_out"), "q_out", t, qs, dev, a.q_out_stride);
    a.num_tokens = int_of(qs[0], "q");
    a.num_q_heads = int_of(qs[1], "q");
    a.head_dim = int_of(qs[2], "q");
    if (x[1] != Py_None) {
      const Tensor &k = tensor(x[1], "k");
      const IntArrayRef ks = rank(k, 3, "k");
      if (ks[0] != qs[0] || ks[2] != qs[2] || ks[1] < 1) value_error("k " + shape_text(ks) + " for q " + shape_text(qs));
      a.k = token_rows(k, "k", t, ks, dev, a.k_stride);
      a.k_out = token_rows(tensor(ko, "k_out"), "k_out", t, ks, dev, a.k_out_stride);
      a.num_kv_heads = int_of(ks[1], "k");
    } else if (x[5] != Py_None) {
      value_error("k_out: without k");
    }
    a.positions = static_cast<int32_t *>(need(x[2], "positions", ScalarType::Int, qs[0], dev));
    a.freqs = static_cast<int64_t *>(need(x[3], "freqs", ScalarType::Long, fs, dev));
    if (fs[0] > 64) value_error("freqs: more than 64 pairs");
    a.rot_dim = (int32_t)(2 * fs[0]);
    a.dtype = t == ScalarType::Float ? PA_ROPE_F32 : PA_ROPE_BF16;
    a.layout = int_arg(x[7], "layout");
    a.inverse = int_arg(x[8], "inverse");
    a.scale = float_arg(x[9]);
    enqueue("pa_rope", g_lib.rope, a, qs[0] == 0, dev, stream_arg(x[6], dev));
    return Py_BuildValue("(OO)", qo, x[1] == Py_None ? Py_None : ko);
  });
}

// q, k, v, cu_seqlens, out, lse, status, stream, sm_scale or None, out_f32, want_lse -> (out, lse or None)
PyObject *prompt_attn(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const Tensor &q = tensor(x[0], "q"), &k = tensor(x[1], "k"), &v = tensor(x[2], "v");
    const int dev = cuda_device(q);
    const IntArrayRef qs = rank(q, 3, "q"), ks = rank(k, 3, "k"), cs = rank(tensor(x[3], "cu_seqlens"), 1, "cu_seqlens");
    if (ks[0] != qs[0] || ks[2] != qs[2] || ks[1] < 1 || qs[1] < 1 || qs[1] % ks[1] != 0 || cs[0] < 1)
      value_error("q " + shape_text(qs) + ", k " + shape_text(ks) + " and cu_seqlens " + shape_text(cs));
    const auto stream = stream_arg(x[7], dev);
    const bool own = x[7] != Py_None;
    const ScalarType bf = ScalarType::BFloat16;
    pa_prompt_attn_args_t a = {};
    a.q = token_rows(q, "q", bf, qs, dev, a.q_stride);
    a.k = token_rows(k, "k", bf, ks, dev, a.k_stride);
    a.v = token_rows(v, "v", bf, ks, dev, a.v_stride);
    a.cu_seqlens = static_cast<int32_t *>(need(x[3], "cu_seqlens", ScalarType::Int, cs, dev));
    a.status = status_word(x[6], dev);
    const ScalarType ot = x[4] != Py_None ? tensor(x[4], "out").scalar_type() : int_arg(x[9], "out_dtype") != 0 ? ScalarType::Float : bf;
    if (ot != bf && ot != ScalarType::Float) type_error(std::string("out: ") + toString(ot) + ", expected bfloat16 or float32");
    Output out(x[4], "out", ot, qs, dev, stream, own);
    std::optional<Output> lse;
    if (x[5] != Py_None || int_arg(x[10], "want_lse") != 0) lse.emplace(x[5], "lse", ScalarType::Float, qs.slice(0, 2), dev, stream, own);
    a.out = out.as<void>();
    if (lse) a.lse = lse->as<float>();
    a.num_seqs = int_of(cs[0] - 1, "cu_seqlens");
    a.num_rows = int_of(qs[0], "q");
    a.num_kv_heads = int_of(ks[1], "k");
    a.group_size = int_of(qs[1] / ks[1], "q");
    a.head_dim = int_of(qs[2], "q");
    a.out_dtype = ot == ScalarType::Float ? PA_OUT_F32 : PA_OUT_BF16;
    a.sm_scale = x[8] == Py_None ? (float)(1.0 / std::sqrt((double)qs[2])) : float_arg(x[8]);
    enqueue("pa_prompt_attn", g_lib.prompt_attn, a, qs[0] == 0, dev, stream);
    Output none;
    return Py_BuildValue("(NN)", out.release(), lse ? lse->release() : none.release());
  });
}

// error class, then the addresses of the entry points in the order of the calls above
PyObject *bind(PyObject *, PyObject *const *x, Py_ssize_t n) {
  constexpr int kEntries = 9;
  return guarded(n, 1 + kEntries, [&]() -> PyObject * {
    void *at[kEntries];
    for (int i = 0; i < kEntries; ++i) {
      at[i] = PyLong_AsVoidPtr(x[i + 1]);
      if (at[i] == nullptr) throw Refusal(PyErr_Occurred() ? nullptr : PyExc_ValueError, "a null entry point");
    }
    g_lib.attn_mass = reinterpret_cast<decltype(g_lib.attn_mass)>(at[0]);
    g_lib.evict_select = reinterpret_cast<decltype(g_lib.evict_select)>(at[1]);
    g_lib.kv_compact = reinterpret_cast<decltype(g_lib.kv_compact)>(at[2]);
    g_lib.beam_select = reinterpret_cast<decltype(g_lib.beam_select)>(at[3]);
    g_lib.beam_reorder = reinterpret_cast<decltype(g_lib.beam_reorder)>(at[4]);
    g_lib.page_assign = reinterpret_cast<decltype(g_lib.page_assign)>(at[5]);
    g_lib.page_release = reinterpret_cast<decltype(g_lib.page_release)>(at[6]);
    g_lib.rope = reinterpret_cast<decltype(g_lib.rope)>(at[7]);
    g_lib.prompt_attn = reinterpret_cast<decltype(g_lib.prompt_attn)>(at[8]);
    Py_INCREF(x[0]);
    Py_XDECREF(g_lib.error);
    g_lib.error = x[0];
    Py_RETURN_NONE;
  });
}

#define PA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {PA_METHOD(bind),        PA_METHOD(attn_mass),   PA_METHOD(evict_select), PA_METHOD(kv_compact), PA_METHOD(beam_select),
                           PA_METHOD(beam_reorder), PA_METHOD(page_assign), PA_METHOD(page_release), PA_METHOD(rope),       PA_METHOD(prompt_attn),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "pa_torch", "Torch side of the cache operators.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_torch() { return PyModule_Create(&g_module); }
