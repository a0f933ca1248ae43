// Marshalling of the tree, rotation and page entry points for Python: torch tensors in, their
// checks, the call into the C ABI, torch tensors out.  The same work in Python (as for the
// other entry points) took most of such a call: their kernels run for a few microseconds, and
// an engine's step waits for the host (a release 18 us a call, of which 4 are the launch).
//
// The entry points' addresses come from the library that the package has loaded, so this
// module links to torch alone.  Every failure is a Python exception; nothing is kept
// between calls but the addresses.  Other Python threads run while a call is in the library or the
// allocator: either may wait for the GPU (a full launch queue, a workspace that grows), and
// the GPU may be waiting for a host function that needs the interpreter.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "paged_attn.h"

namespace {

using at::Tensor;
using c10::IntArrayRef;
using c10::ScalarType;

struct Entries {
  decltype(&paged_attn_decode_tree) tree;
  decltype(&paged_kv_rope_append_slots) rope;
  decltype(&paged_kv_compact) compact;
  decltype(&paged_kv_fork) fork;
  decltype(&paged_kv_release) release;
} entry = {};
PyObject* on_error = nullptr;  // called with a status that is not 0; raises

// A Python exception is set.
struct Raised {};
[[noreturn]] void refuse(const std::string& why) {
  PyErr_SetString(PyExc_ValueError, why.c_str());
  throw Raised();
}

// The interpreter's lock, let go of in a scope that touches no Python object.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

std::string dtype_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    default: return c10::toString(t);
  }
}
std::string shape_text(IntArrayRef s) {
  std::string x = "(";
  for (size_t i = 0; i < s.size(); ++i) x += (i ? ", " : "") + std::to_string(s[i]);
  return x + (s.size() == 1 ? ",)" : ")");
}

// The tensors of a call: each checked once, all on the current device or pinned; and its stream,
// the one given or the device's current one.
class Call {
 public:
  explicit Call(PyObject* s) {
    if (s == Py_None) return;
    PyObject* h = PyObject_GetAttrString(s, "cuda_stream");
    if (!h) throw Raised();
    stream_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
    Py_DECREF(h);
    if (!stream_ && PyErr_Occurred()) throw Raised();
    given_ = true;
  }
  const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  const Tensor* optional(PyObject* o, const char* name) {
    return o == Py_None ? nullptr : &tensor(o, name);
  }
  void need(const Tensor& t, const char* name, ScalarType dtype, IntArrayRef shape) {
    if (t.scalar_type() != dtype || t.sizes() != shape || !t.is_contiguous())
      refuse(std::string(name) + " must be a contiguous " + dtype_name(dtype) +
             " tensor of shape " + shape_text(shape) + ", got " + dtype_name(t.scalar_type()) +
             " " + shape_text(t.sizes()));
  }
  // Rows [rows, heads, D] of bf16, each contiguous; their stride.
  int64_t strided_rows(const Tensor& t, const char* name, int64_t rows, int64_t heads, int64_t D) {
    if (t.scalar_type() != ScalarType::BFloat16 || t.sizes() != IntArrayRef({rows, heads, D}))
      refuse(std::string(name) + " must be bfloat16 " + shape_text({rows, heads, D}));
    if (rows == 0) return heads * D;
    if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D))
      refuse("the rows of " + std::string(name) + " must be contiguous [heads, head_dim]");
    return rows > 1 ? t.stride(0) : heads * D;
  }
  void* at(const Tensor& t) {
    if (t.is_cuda()) {
      if (device_ < 0) device_ = c10::cuda::current_device();
      if (t.get_device() != device_) refuse("every tensor must be on the current CUDA device");
    } else if (!t.is_pinned()) {
      refuse("host tensors must be pinned");
    }
    return t.data_ptr();
  }
  void* at(const Tensor* t) { return t ? at(*t) : nullptr; }
  // What tensor copies and atomics reach lies in device memory.
  void* on_device(const Tensor& t, const char* name) {
    void* x = at(t);
    if (!t.is_cuda()) refuse(std::string(name) + " must be in device memory");
    return x;
  }
  template <typename T>
  T* as(const Tensor& t) {
    return static_cast<T*>(at(t));
  }
  template <typename T>
  T* as(const Tensor* t) {
    return static_cast<T*>(at(t));
  }
  void* stream() const {
    return given_ ? stream_
                  : c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
  }
  // An output of the call (its inputs have been seen), in device memory even where it is made like a
  // pinned tensor.  With a stream given it is that stream's memory: the allocator may give a
  // block of the current stream's whose last use there is still to come, and may give it
  // away again before the call's kernels have run.
  Tensor make(const Tensor& like) {
    if (device_ < 0) device_ = c10::cuda::current_device();
    const auto device = static_cast<c10::DeviceIndex>(device_);
    const auto options = like.options().device(c10::Device(c10::DeviceType::CUDA, device));
    if (!given_ || c10::cuda::getCurrentCUDAStream(device).stream() == stream_)
      return at::empty(like.sizes(), options);
    c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(stream_, device));
    return at::empty(like.sizes(), options);
  }

 private:
  int device_ = -1;  // the current one, once a CUDA tensor has been seen
  cudaStream_t stream_ = nullptr;
  bool given_ = false;
};

int int32_of(PyObject* o, const char* name) {
  PyObject* x = PyNumber_Long(o);
  if (!x) throw Raised();
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(x, &over);
  Py_DECREF(x);
  if (over || v < INT32_MIN || v > INT32_MAX)
    refuse(std::string(name) + " must fit 32 bits");
  return static_cast<int>(v);
}
int int32_size(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + " must fit 32 bits, got " + std::to_string(v));
  return static_cast<int>(v);
}
float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}
// The cap as the C ABI takes it: one below float32's range is not taken for none.
float softcap_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  if (v != 0.0 && static_cast<float>(v) == 0.f)
    refuse("softcap must be 0 or in [1e-30, 1e30], got " + std::to_string(v));
  return static_cast<float>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
// A call into the library, with the outputs that it makes, and its status as an exception.
template <typename... P, typename... A>
void run(int (*f)(P...), A... a) {
  int status;
  {
    const Unlocked others;
    status = f(a...);
  }
  if (status == 0) return;
  PyObject* r = PyObject_CallFunction(on_error, "i", status);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "paged_attn status %d", status);
  throw Raised();
}

// The caches [num_blocks, H_kv, block_size, D]: bf16, or e4m3 bytes with both floats.
struct Caches {
  const Tensor &k, &v;
  const Tensor *k_scale, *v_scale;
  int64_t nb;
  int H, BS, D;
  Caches(Call& c, PyObject* pk, PyObject* pv, PyObject* pks, PyObject* pvs)
      : k(c.tensor(pk, "k_cache")), v(c.tensor(pv, "v_cache")),
        k_scale(c.optional(pks, "k_scale")), v_scale(c.optional(pvs, "v_scale")) {
    if (k.dim() != 4) refuse("the caches must be [num_blocks, H_kv, block_size, D]");
    if (!k_scale != !v_scale)
      refuse("k_scale and v_scale come together (FP8 caches) or not at all");
    const ScalarType dtype = k_scale ? ScalarType::Byte : ScalarType::BFloat16;
    const IntArrayRef s = k.sizes();
    c.need(k, "k_cache", dtype, s);
    c.need(v, "v_cache", dtype, s);
    if (k_scale) {
      c.need(*k_scale, "k_scale", ScalarType::Float, s.slice(0, 3));
      c.need(*v_scale, "v_scale", ScalarType::Float, s.slice(0, 3));
    }
    nb = s[0];
    H = int32_size(s[1], "H_kv");
    BS = int32_size(s[2], "block_size");
    D = int32_size(s[3], "head_dim");
  }
};

constexpr ScalarType kI32 = ScalarType::Int;

// An output: the tensor given, checked, or one like an input that is made when the library is called.
struct Output {
  PyObject* object;
  const Tensor* given;
  Tensor made;
  Output(Call& c, PyObject* o, const char* name, ScalarType dtype, IntArrayRef shape)
      : object(o), given(c.optional(o, name)) {
    if (given) c.need(*given, name, dtype, shape);
  }
  // An argument of `run`, which turns it into the pointer.
  struct Pointer {
    Output& output;
    Call& call;
    const Tensor& like;
    void* known;
    template <typename T>
    operator T*() const {
      if (!output.given) output.made = call.make(like);
      return static_cast<T*>(output.given ? known : output.made.data_ptr());
    }
  };
  Pointer at(Call& c, const Tensor& like) {
    return {*this, c, like, given ? c.at(*given) : nullptr};
  }
  PyObject* result() const {  // a new reference
    if (!given) return THPVariable_Wrap(made);
    Py_INCREF(object);
    return object;
  }
};
void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    throw Raised();
  }
}

PyObject* decode_tree(PyObject* const* a, Py_ssize_t n) {
  expect(n, 15);
  const float scale = float_of(a[7]), softcap = softcap_of(a[8]);
  const int window = int32_of(a[10], "window");
  Call c(a[14]);
  const Tensor &q = c.tensor(a[0], "q"), &k = c.tensor(a[1], "k_cache"),
               &v = c.tensor(a[2], "v_cache"), &qo = c.tensor(a[3], "qo_indptr"),
               &mask = c.tensor(a[4], "tree_mask"), &bt = c.tensor(a[5], "block_tables"),
               &lens = c.tensor(a[6], "seq_lens");
  const Tensor *slopes = c.optional(a[9], "alibi_slopes"),
               *prefix = c.optional(a[11], "prefix_lens"), *ws = c.optional(a[13], "workspace");
  if (q.dim() != 3 || k.dim() != 4 || bt.dim() != 2 || lens.dim() != 1)
    refuse("q must be [rows, H_q, D], the caches [num_blocks, H_kv, block_size, D], "
           "block_tables [num_seqs, max_blocks] and seq_lens [num_seqs]");
  if (k.size(3) != q.size(2)) refuse("q and the caches disagree on head_dim");
  if (mask.dim() != 2) refuse("tree_mask must be [total_q, words]");
  const int64_t seqs = lens.size(0), rows = q.size(0), H = q.size(1);
  c.need(q, "q", ScalarType::BFloat16, q.sizes());
  c.need(k, "k_cache", ScalarType::BFloat16, k.sizes());
  c.need(v, "v_cache", ScalarType::BFloat16, k.sizes());
  c.need(bt, "block_tables", kI32, {seqs, bt.size(1)});
  c.need(lens, "seq_lens", kI32, {seqs});
  c.need(qo, "qo_indptr", kI32, {seqs + 1});
  c.need(mask, "tree_mask", kI32, {rows, mask.size(1)});
  if (slopes) c.need(*slopes, "alibi_slopes", ScalarType::Float, {H});
  if (prefix) c.need(*prefix, "prefix_lens", kI32, {seqs});
  if (ws && !ws->is_contiguous()) refuse("workspace must be contiguous");
  Output made(c, a[12], "out", ScalarType::BFloat16, q.sizes());
  const void *pq = c.at(q), *pk = c.on_device(k, "k_cache"), *pv = c.on_device(v, "v_cache");
  run(entry.tree, pq, pk, pv, made.at(c, q), c.as<int32_t>(qo), c.as<int32_t>(mask),
      int32_size(mask.size(1), "tree_mask's words"), c.as<int32_t>(bt), c.as<int32_t>(lens),
      int32_size(seqs, "num_seqs"), int32_size(rows, "total_q"), int32_size(H, "H_q"),
      int32_size(k.size(1), "H_kv"), int32_size(q.size(2), "head_dim"),
      int32_size(bt.size(1), "max_blocks"), int32_size(k.size(2), "block_size"), scale, softcap,
      c.as<float>(slopes), window, c.as<int32_t>(prefix), c.at(ws), ws ? ws->nbytes() : 0, c.stream());
  return made.result();
}

PyObject* rope_append_slots(PyObject* const* a, Py_ssize_t n) {
  expect(n, 17);
  Call c(a[16]);
  const Caches cache(c, a[3], a[4], a[13], a[14]);
  const Tensor &q = c.tensor(a[0], "q"), &kn = c.tensor(a[1], "k_new"),
               &vn = c.tensor(a[2], "v_new"), &slots = c.tensor(a[5], "slot_map"),
               &pos = c.tensor(a[6], "positions"), &cs = c.tensor(a[7], "cos_sin");
  const bool interleaved = truth(a[8]);
  const Tensor *axis = c.optional(a[9], "freq_axis"), *qw = c.optional(a[10], "q_norm"),
               *kw = c.optional(a[11], "k_norm");
  const float eps = float_of(a[12]);
  if (q.dim() != 3) refuse("q must be [rows, H_q, D]");
  const int64_t rows = q.size(0), H = q.size(1), D = cache.D;
  const int64_t qs = c.strided_rows(q, "q", rows, H, D);
  const int64_t ks = c.strided_rows(kn, "k_new", rows, cache.H, D);
  const int64_t vs = c.strided_rows(vn, "v_new", rows, cache.H, D);
  c.need(slots, "slot_map", ScalarType::Long, {rows});
  int64_t axes = 1;
  if (pos.dim() == 2) {
    axes = pos.size(0);
    c.need(pos, "positions", kI32, {axes, rows});
  } else {
    c.need(pos, "positions", kI32, {rows});
  }
  if (cs.dim() != 2) refuse("cos_sin must be [max_positions, rotary_dim]");
  c.need(cs, "cos_sin", ScalarType::Float, cs.sizes());
  if (axis) c.need(*axis, "freq_axis", kI32, {cs.size(1) / 2});
  if (qw) c.need(*qw, "q_norm", ScalarType::Float, {D});
  if (kw) c.need(*kw, "k_norm", ScalarType::Float, {D});
  Output made(c, a[15], "out", ScalarType::BFloat16, q.sizes());
  const void *pq = c.on_device(q, "q"), *pk = c.on_device(kn, "k_new"),
             *pv = c.on_device(vn, "v_new");
  run(entry.rope, pq, pk, pv, qs, ks, vs, made.at(c, q), c.on_device(cache.k, "k_cache"),
      c.on_device(cache.v, "v_cache"), c.as<float>(cache.k_scale), c.as<float>(cache.v_scale),
      c.as<int64_t>(slots), c.as<int32_t>(pos), int32_size(axes, "axes"), c.as<int32_t>(axis),
      c.as<float>(cs), int32_size(cs.size(0), "max_positions"),
      int32_size(cs.size(1), "rotary_dim"), interleaved, c.as<float>(qw), c.as<float>(kw), eps,
      int32_size(rows, "rows"), int32_size(H, "H_q"), cache.H, cache.D, cache.BS, cache.nb, c.stream());
  return made.result();
}

PyObject* compact(PyObject* const* a, Py_ssize_t n) {
  expect(n, 10);
  Call c(a[9]);
  const Caches cache(c, a[0], a[1], a[6], a[7]);
  const Tensor &qo = c.tensor(a[2], "qo_indptr"), &acc = c.tensor(a[3], "accepted"),
               &bt = c.tensor(a[4], "block_tables"), &lens = c.tensor(a[5], "seq_lens");
  if (acc.dim() != 2 || bt.dim() != 2 || lens.dim() != 1)
    refuse("accepted must be [num_seqs, max_accept], block_tables [num_seqs, max_blocks], "
           "seq_lens [num_seqs]");
  const int64_t seqs = lens.size(0);
  c.need(lens, "seq_lens", kI32, {seqs});
  c.need(qo, "qo_indptr", kI32, {seqs + 1});
  c.need(acc, "accepted", kI32, {seqs, acc.size(1)});
  c.need(bt, "block_tables", kI32, {seqs, bt.size(1)});
  Output made(c, a[8], "seq_lens_out", kI32, {seqs});
  int32_t* plens = c.as<int32_t>(lens);
  run(entry.compact, c.on_device(cache.k, "k_cache"), c.on_device(cache.v, "v_cache"),
      c.as<float>(cache.k_scale), c.as<float>(cache.v_scale), c.as<int32_t>(qo),
      c.as<int32_t>(acc), c.as<int32_t>(bt), plens, made.at(c, lens),
      int32_size(seqs, "num_seqs"), int32_size(acc.size(1), "max_accept"), cache.H, cache.D,
      int32_size(bt.size(1), "max_blocks"), cache.BS, cache.nb, c.stream());
  return made.result();
}

PyObject* fork(PyObject* const* a, Py_ssize_t n) {
  expect(n, 14);
  Call c(a[13]);
  const Caches cache(c, a[0], a[1], a[9], a[10]);
  const Tensor &bt = c.tensor(a[2], "block_tables"), &lens = c.tensor(a[3], "seq_lens"),
               &parents = c.tensor(a[4], "parents"), &children = c.tensor(a[5], "children"),
               &refs = c.tensor(a[6], "block_refs"), &free_blocks = c.tensor(a[7], "free_blocks"),
               &count = c.tensor(a[8], "free_count");
  const Tensor* refused = c.optional(a[12], "refused");
  if (bt.dim() != 2 || parents.dim() != 1)
    refuse("block_tables must be [rows, max_blocks], parents [forks]");
  const int64_t rows = bt.size(0), forks = parents.size(0), n_free = free_blocks.numel();
  c.need(bt, "block_tables", kI32, bt.sizes());
  c.need(lens, "seq_lens", kI32, {rows});
  c.need(parents, "parents", kI32, {forks});
  c.need(children, "children", kI32, {forks});
  c.need(refs, "block_refs", kI32, {cache.nb});
  c.need(free_blocks, "free_blocks", kI32, {n_free});
  c.need(count, "free_count", kI32, {1});
  if (refused) c.need(*refused, "refused", kI32, {1});
  Output made(c, a[11], "free_count_out", kI32, {1});
  int32_t* pcount = c.as<int32_t>(count);
  c.on_device(refs, "block_refs");
  run(entry.fork, c.on_device(cache.k, "k_cache"), c.on_device(cache.v, "v_cache"),
      c.as<float>(cache.k_scale), c.as<float>(cache.v_scale), c.as<int32_t>(bt),
      c.as<int32_t>(lens), c.as<int32_t>(parents), c.as<int32_t>(children), c.as<int32_t>(refs),
      c.as<int32_t>(free_blocks), pcount, made.at(c, count), c.as<int32_t>(refused),
      int32_size(forks, "forks"), int32_size(rows, "rows"), cache.H, cache.D,
      int32_size(bt.size(1), "max_blocks"), cache.BS, int32_size(n_free, "free_blocks' length"),
      cache.nb, c.stream());
  return made.result();
}

PyObject* release(PyObject* const* a, Py_ssize_t n) {
  expect(n, 10);
  const int BS = int32_of(a[5], "block_size");
  Call c(a[9]);
  const Tensor &bt = c.tensor(a[0], "block_tables"), &lens = c.tensor(a[1], "seq_lens"),
               &keep = c.tensor(a[2], "keep_lens"), &free_blocks = c.tensor(a[3], "free_blocks"),
               &count = c.tensor(a[4], "free_count");
  const Tensor* refs = c.optional(a[6], "block_refs");
  if (bt.dim() != 2 || lens.dim() != 1)
    refuse("block_tables must be [num_seqs, max_blocks], seq_lens [num_seqs]");
  const int64_t seqs = lens.size(0), n_free = free_blocks.numel();
  c.need(bt, "block_tables", kI32, {seqs, bt.size(1)});
  c.need(lens, "seq_lens", kI32, {seqs});
  c.need(keep, "keep_lens", kI32, {seqs});
  c.need(free_blocks, "free_blocks", kI32, {n_free});
  c.need(count, "free_count", kI32, {1});
  if (refs) c.need(*refs, "block_refs", kI32, {refs->numel()});
  Output made_lens(c, a[7], "seq_lens_out", kI32, {seqs});
  Output made_count(c, a[8], "free_count_out", kI32, {1});
  int32_t *plens = c.as<int32_t>(lens), *pcount = c.as<int32_t>(count);
  if (refs) c.on_device(*refs, "block_refs");
  run(entry.release, c.as<int32_t>(bt), plens, c.as<int32_t>(keep), c.as<int32_t>(refs),
      refs ? refs->numel() : 0, c.as<int32_t>(free_blocks), pcount, made_lens.at(c, lens),
      made_count.at(c, count), int32_size(seqs, "num_seqs"), int32_size(bt.size(1), "max_blocks"), BS,
      int32_size(n_free, "free_blocks' length"), c.stream());
  PyObject* x = made_lens.result();
  if (!x) return nullptr;
  PyObject* y = made_count.result();
  if (!y) {
    Py_DECREF(x);
    return nullptr;
  }
  PyObject* pair = PyTuple_New(2);
  if (!pair) {
    Py_DECREF(x);
    Py_DECREF(y);
    return nullptr;
  }
  PyTuple_SET_ITEM(pair, 0, x);
  PyTuple_SET_ITEM(pair, 1, y);
  return pair;
}

// No C++ exception leaves a function that Python calls.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// init(on_error, addresses of the five entry points in the order of Entries)
PyObject* init(PyObject* const* a, Py_ssize_t n) {
  expect(n, 6);
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point has no address");
      throw Raised();
    }
  }
  entry.tree = reinterpret_cast<decltype(entry.tree)>(p[0]);
  entry.rope = reinterpret_cast<decltype(entry.rope)>(p[1]);
  entry.compact = reinterpret_cast<decltype(entry.compact)>(p[2]);
  entry.fork = reinterpret_cast<decltype(entry.fork)>(p[3]);
  entry.release = reinterpret_cast<decltype(entry.release)>(p[4]);
  Py_INCREF(a[0]);
  Py_XSETREF(on_error, a[0]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {
    {"init", fast(guarded<init>), METH_FASTCALL, nullptr},
    {"decode_tree", fast(guarded<decode_tree>), METH_FASTCALL, nullptr},
    {"rope_append_slots", fast(guarded<rope_append_slots>), METH_FASTCALL, nullptr},
    {"compact", fast(guarded<compact>), METH_FASTCALL, nullptr},
    {"fork", fast(guarded<fork>), METH_FASTCALL, nullptr},
    {"release", fast(guarded<release>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_native() { return PyModule_Create(&module); }
